// Shared parts of the selective scan's kernels (scan.hip, scan_backward.hip):
// tile geometry, staging of a tile in LDS, sums over a channel's lanes.
//
//   h_t[d,n] = exp(delta_t[d] A[d,n]) h_{t-1}[d,n] + u_t[d] B_t[n],  u = delta x
//
// With a decay of its own for every (channel, state) pair the recurrence has no
// matrix-product form: per (token, channel, state) it is a multiply, an
// exponential and a multiply-add, and one more multiply-add for the readout.  So
// the vector ALUs bound it, the exponentials (half rate) for two fifths.
//
// A wave holds 16 channels, lane = 16 s + channel, with the states 16 i + 4 s ..
// + 3 (i < NB) of its channel in registers: a token's sum over the states of
// four tokens takes three lane swaps and three additions.  What is shared by a
// channel's lanes (delta, u, the gate) or by all channels (B, C) is computed or
// converted once per tile and passed on in LDS.  (This is also the layout of a
// 16 x 16 fp32 matrix product's result; forming u_t B_t^T on the matrix cores
// saved a ninth of the vector instructions and made the scan a quarter slower.)
#pragma once
#include "layer_internal.hpp"

namespace m3 {
namespace scan {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 256;

// exp(delta A) from A log2(e): the hardware exponential, 1 ulp.
__device__ __forceinline__ float decay(float delta, float a2) { return __builtin_amdgcn_exp2f(delta * a2); }

// softplus(v) = max(v, 0) + log1p(u), u = exp(-|v|), in 9 instructions.  With
// w = fl(1 + u), log1p(u) = log(w) + log1p((u - (w - 1)) / w); the last term is
// at most 2^-24 and matters against log(w) for small u only, where w is near 1:
// so it enters as u - (w - 1), which costs at most 1.5 2^-24 of the value and
// leaves log1p(u) = u where w rounds to 1.
__device__ __forceinline__ float softplus_fast(float v) {
  const float u = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e);
  const float w = 1.f + u;
  return fmaxf(v, 0.f) + fmaf(__builtin_amdgcn_logf(w), kLn2, u - (w - 1.f));
}
// delta of one token: 0 behind the end.
__device__ __forceinline__ float step_of(float raw, bool softplus, float bias, bool valid) {
  return !valid ? 0.f : softplus ? softplus_fast(raw + bias) : raw;
}

// Blocks of neighbouring channels on one XCD (workgroups are dealt to the 8 XCDs
// in turn), so that the lines they share are fetched into one L2.
__device__ __forceinline__ int block_on_xcd() {
  const int n = gridDim.x, i = blockIdx.x;
  return n % 8 == 0 ? (i & 7) * (n >> 3) + (i >> 3) : i;
}

// Sums over the four lanes of a channel of four values, one left in each lane:
// row q of 16 lanes ends with the sum of v[row_value(q)].
__device__ __forceinline__ int row_value(int q) { return (q & 1) << 1 | q >> 1; }  // 0, 2, 1, 3
__device__ __forceinline__ float rows_sum4(const float* v) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[0]), __float_as_uint(v[1]), false, false);
  const auto b = __builtin_amdgcn_permlane32_swap(__float_as_uint(v[2]), __float_as_uint(v[3]), false, false);
  const float lo = __uint_as_float(a[0]) + __uint_as_float(a[1]), hi = __uint_as_float(b[0]) + __uint_as_float(b[1]);
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(lo), __float_as_uint(hi), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// One tile's share of a row-major [token][channel] tensor: this thread's VE
// neighbouring channels of one token.  The loads have no branch around them (a
// branch makes the compiler wait for the values at its end): rows and columns
// past the edge are read from the nearest ones inside and dropped by the user.
template <typename T, int VE, bool VEC>
__device__ __forceinline__ Pack<T, VE> fetch_cols(const T* p, int ncol) {
  if constexpr (VEC) return load_pack<T, VE>(p);
  Pack<T, VE> q;
#pragma unroll
  for (int v = 0; v < VE; ++v) q.e[v] = p[v < ncol ? v : ncol - 1];
  return q;
}
template <typename T, int VE, bool VEC>
__device__ __forceinline__ Pack<T, VE> load_cols(const T* p, bool row, int ncol) {
  Pack<T, VE> q{};
  if constexpr (VEC) {
    if (row && ncol > 0) q = load_pack<T, VE>(p);
  } else {
    if (row) q = load_some<T, VE>(p, ncol);
  }
  return q;
}
template <typename T, int VE, bool VEC>
__device__ __forceinline__ void store_cols(T* p, const float* v, bool row, int ncol) {
  if constexpr (VEC) {
    if (row && ncol > 0) store_pack<T, VE>(p, v);
  } else {
    if (row) store_some<T, VE>(p, v, ncol);
  }
}

// Blocks of channels never straddle two groups.
constexpr int CH = 64;  // channels of a block: 16 for each of its four scanning waves
inline int state_blocks(int N) { return N <= 16 ? 1 : N <= 32 ? 2 : 4; }  // of 16 states
inline int blocks_per_group(int Dg) { return (Dg + CH - 1) / CH; }

}  // namespace scan
}  // namespace m3
