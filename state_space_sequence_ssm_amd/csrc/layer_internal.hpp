// Launchers and shared device helpers of the layer operators (causal
// convolution, selective scan, gated and residual norms).  The argument blocks
// are the public ones of m3ssm.h, validated and with every `*_ld` filled in.
#pragma once
#include "common.hpp"
#include "m3ssm.h"

namespace m3 {

// Column sums of partial results, part [P][ncols] (row-major fp32), in a fixed
// order.  Columns go, in order, to the n[i] elements at dst[i] (null: dropped);
// with `taps` > 0 the first n[0] = taps * D columns are [taps][D] and go to
// dst[0] transposed, [D][taps].
struct ColSum {
  const float* part;
  int64_t P;
  int64_t ncols;
  float* dst[4];
  int64_t n[4];
  int taps;
  int D;
};
hipError_t launch_colsum(const ColSum& c, hipStream_t s);

// Whether a launch's work items, blocks times threads, stay within the 32 bits in which
// they are counted.  The *_fits functions, and for the backwards of convolution and scan a
// workspace size other than 0, say so for all launches of a call; the calls without either
// stay within it by the limits of their sizes.
inline bool launchable(int64_t blocks, int threads) { return blocks * threads < (int64_t(1) << 32); }

hipError_t launch_conv(const m3_conv_args& a, hipStream_t s);
hipError_t launch_conv_step(const m3_conv_step_args& a, hipStream_t s);
size_t conv_backward_workspace(const m3_conv_backward_args& a);
hipError_t launch_conv_backward(const m3_conv_backward_args& a, hipStream_t s);

bool scan_fits(const m3_scan_args& a);
size_t scan_workspace(const m3_scan_args& a);
hipError_t launch_scan(const m3_scan_args& a, hipStream_t s);
bool scan_step_fits(const m3_scan_step_args& a);
hipError_t launch_scan_step(const m3_scan_step_args& a, hipStream_t s);
size_t scan_backward_workspace(const m3_scan_backward_args& a);
hipError_t launch_scan_backward(const m3_scan_backward_args& a, hipStream_t s);

hipError_t launch_gated_norm(const m3_gated_norm_args& a, hipStream_t s);
bool gated_norm_backward_fits(const m3_gated_norm_backward_args& a);
size_t gated_norm_backward_workspace(const m3_gated_norm_backward_args& a);
hipError_t launch_gated_norm_backward(const m3_gated_norm_backward_args& a, hipStream_t s);
hipError_t launch_residual_norm(const m3_residual_norm_args& a, hipStream_t s);
bool residual_norm_backward_fits(const m3_residual_norm_backward_args& a);
size_t residual_norm_backward_workspace(const m3_residual_norm_backward_args& a);
hipError_t launch_residual_norm_backward(const m3_residual_norm_backward_args& a, hipStream_t s);

// ---------------------------------------------------------------- device helpers
// V consecutive elements, moved as whole words (16 bytes at most per access).
template <typename T, int V>
struct alignas(V & (V - 1) ? sizeof(T) : sizeof(T) * V < 16 ? sizeof(T) * V : 16) Pack {
  T e[V];
};
__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(bf16_t v) { return bf16_to_f32(v.bits); }
__device__ __forceinline__ void from_f32(float v, float& o) { o = v; }
__device__ __forceinline__ void from_f32(float v, bf16_t& o) { o.bits = f32_to_bf16(v); }

template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_pack(const T* p) {
  return *reinterpret_cast<const Pack<T, V>*>(p);
}
template <typename T, int V>
__device__ __forceinline__ void store_pack(T* p, const float* v) {
  Pack<T, V> o;
  if constexpr (sizeof(T) == 2 && V % 2 == 0) {
    uint32_t w[V / 2];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) w[i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
    __builtin_memcpy(&o, w, sizeof(o));
  } else {
#pragma unroll
    for (int i = 0; i < V; ++i) from_f32(v[i], o.e[i]);
  }
  *reinterpret_cast<Pack<T, V>*>(p) = o;
}
// The same with the alignment of T only, in the widest accesses all the same (vector
// types, which the compiler keeps whole, unlike a struct).
template <int BYTES>
struct Loose {
  typedef uint32_t whole __attribute__((ext_vector_type(BYTES / 4)));
  typedef whole type __attribute__((aligned(2), may_alias));
};
template <>
struct Loose<4> {
  typedef uint32_t whole;
  typedef whole type __attribute__((aligned(2), may_alias));
};
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_loose(const T* p) {
  constexpr int kBytes = int(sizeof(T)) * V, kStep = kBytes < 16 ? kBytes : 16;
  static_assert(kBytes >= 4, "a dword at least");
  Pack<T, V> q;
#pragma unroll
  for (int i = 0; i < kBytes / kStep; ++i) {
    const typename Loose<kStep>::whole w = reinterpret_cast<const typename Loose<kStep>::type*>(p)[i];
    __builtin_memcpy(reinterpret_cast<char*>(&q) + kStep * i, &w, kStep);
  }
  return q;
}
template <typename T, int V>
__device__ __forceinline__ void put_loose(T* p, const Pack<T, V>& q) {
  constexpr int kBytes = int(sizeof(T)) * V, kStep = kBytes < 16 ? kBytes : 16;
#pragma unroll
  for (int i = 0; i < kBytes / kStep; ++i) {
    typename Loose<kStep>::whole w;
    __builtin_memcpy(&w, reinterpret_cast<const char*>(&q) + kStep * i, kStep);
    reinterpret_cast<typename Loose<kStep>::type*>(p)[i] = w;
  }
}
template <typename T, int V>
__device__ __forceinline__ void store_loose(T* p, const float* v) {
  Pack<T, V> q;
  store_pack<T, V>(q.e, v);
  put_loose<T, V>(p, q);
}
// A word, aligned or (RAG) with the alignment of its elements.
template <typename T, int V, bool RAG>
__device__ __forceinline__ Pack<T, V> load_word(const T* p) {
  if constexpr (RAG) return load_loose<T, V>(p);
  else return load_pack<T, V>(p);
}
template <typename T, int V, bool RAG>
__device__ __forceinline__ void store_word(T* p, const float* v) {
  if constexpr (RAG) store_loose<T, V>(p, v);
  else store_pack<T, V>(p, v);
}
template <typename T, int V>
__device__ __forceinline__ void unpack(const Pack<T, V>& q, float* v) {
#pragma unroll
  for (int i = 0; i < V; ++i) v[i] = to_f32(q.e[i]);
}
// The first n (0..V) of V elements one at a time, the others zero: rows whose
// width or address does not allow whole words.
template <typename T, int V>
__device__ __forceinline__ Pack<T, V> load_some(const T* p, int n) {
  Pack<T, V> q;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    if (i < n) q.e[i] = p[i];
    else q.e[i] = T{};
  }
  return q;
}
template <typename T, int V>
__device__ __forceinline__ void store_some(T* p, const float* v, int n) {
#pragma unroll
  for (int i = 0; i < V; ++i)
    if (i < n) from_f32(v[i], p[i]);
}

// sigmoid and SiLU from the hardware exponential and reciprocal (1 ulp each).
// At v <= -88.8 the exponential overflows to infinity and the sigmoid is 0.
__device__ __forceinline__ float sigmoid_f(float v) { return __builtin_amdgcn_rcpf(1.f + __expf(-v)); }
__device__ __forceinline__ float silu_f(float v) { return v * sigmoid_f(v); }
// silu'(v) = g (1 + v (1 - g)), g = sigmoid(v)
__device__ __forceinline__ float dsilu_f(float v, float g) { return g * (1.f + v * (1.f - g)); }

// The block's index with neighbours on one XCD (workgroups are dealt to the 8
// XCDs in turn), so that lines that neighbours share are fetched into one L2.
__device__ __forceinline__ int block_on_xcd() {
  const int n = gridDim.x, i = blockIdx.x;
  return n % 8 == 0 ? (i & 7) * (n >> 3) + (i >> 3) : i;
}

__device__ __forceinline__ int item_length(const int32_t* lengths, int b, int L) {
  if (lengths == nullptr) return L;
  const int n = lengths[b];
  return n < 0 ? 0 : (n > L ? L : n);
}

// ---------------------------------------------------------------- host helpers
inline bool rows_aligned(const void* p, int64_t ld, size_t elem, size_t bytes) {
  return reinterpret_cast<uintptr_t>(p) % bytes == 0 && (size_t(ld) * elem) % bytes == 0;
}
inline size_t round256(size_t v) { return (v + 255) & ~size_t(255); }


// Column sums: a block of 1024 threads takes COLS columns, its 1024 / COLS row groups
// every so many-th partial row, joined in LDS.  Few columns per block for many rows, so
// that a narrow matrix still fills the card (64-byte pieces of a row).
inline int colsum_cols(int64_t P) { return P > 32 ? 16 : 128; }
inline int64_t colsum_blocks(int64_t P, int64_t ncols) { return (ncols + colsum_cols(P) - 1) / colsum_cols(P); }
template <int COLS>
__device__ __forceinline__ void colsum_block(const ColSum& c, uint32_t block, float* red) {
  constexpr int RG = 1024 / COLS;
  const int lane = threadIdx.x % COLS, rg = threadIdx.x / COLS;
  const int64_t col = int64_t(block) * COLS + lane;
  float s = 0.f;
  if (col < c.ncols) {
#pragma unroll 4
    for (int64_t r = rg; r < c.P; r += RG) s += c.part[r * c.ncols + col];
  }
  red[threadIdx.x] = s;
  for (int n = RG / 2; n > 0; n /= 2) {
    __syncthreads();
    if (rg < n) red[threadIdx.x] += red[threadIdx.x + n * COLS];
  }
  if (rg != 0 || col >= c.ncols) return;
  s = red[lane];
  int64_t k = col;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (k < c.n[i]) {
      if (c.dst[i] != nullptr) c.dst[i][i == 0 && c.taps > 0 ? (k % c.D) * c.taps + k / c.D : k] = s;
      return;
    }
    k -= c.n[i];
  }
}

}  // namespace m3
