// Shared parts of the selective scan's kernels (scan.hip, scan_backward.hip):
// tile geometry, staging of a tile in LDS, sums over a channel's lanes.
//
//   h_t[d,n] = exp(delta_t[d] A[d,n]) h_{t-1}[d,n] + u_t[d] B_t[n],  u = delta x
//
// With a decay of its own for every (channel, state) pair the recurrence has no
// matrix-product form: it is one exponential, two multiplies and a multiply-add
// per (token, channel, state), and one more multiply-add for the readout.  So
// the vector ALUs bound it.  A channel's N states lie in S neighbouring lanes,
// K each; a block of 256 lanes owns 256 / S channels of one group and walks the
// token axis in tiles.  What is shared by a channel's lanes (delta, u, the
// gate) or by all channels (B, C) is computed or converted once per tile by the
// block and passed on in LDS.
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

// Sum over the S neighbouring lanes of a channel, in each of them.
template <int S>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (S >= 2) v += dpp<0xB1, 0xF, true>(v);    // lane ^ 1
  if constexpr (S >= 4) v += dpp<0x4E, 0xF, true>(v);    // lane ^ 2
  if constexpr (S >= 8) v += dpp<0x141, 0xF, true>(v);   // mirrored within 8
  if constexpr (S >= 16) v += dpp<0x140, 0xF, true>(v);  // mirrored within 16
  return v;
}

// m ? a : b for an all-ones or all-zeros m, as one bit-field instruction (a
// ternary of sums becomes a branch around them).
__device__ __forceinline__ float pick(uint32_t m, float a, float b) {
  return __uint_as_float((__float_as_uint(a) & m) | (__float_as_uint(b) & ~m));
}
// Sums over a channel's S lanes of four values, one value left in each lane:
// lane s ends with the sum of v[s & 3] (S = 2: v[s] and v[2 + s]).  Halving the
// values with the lanes takes 9 instructions at S = 4 instead of 8 for four
// full sums and the selection after them.  odd, two: all ones where s & 1, s & 2.
template <int S>
__device__ __forceinline__ void lanes_sum4(const float (&v)[4], uint32_t odd, uint32_t two, float& r0, float& r1) {
  float t[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t[i] = v[i];
    if constexpr (S >= 16) t[i] += dpp<0x140, 0xF, true>(t[i]);
    if constexpr (S >= 8) t[i] += dpp<0x141, 0xF, true>(t[i]);
  }
  const float a = pick(odd, t[1], t[0]) + dpp<0xB1, 0xF, true>(pick(odd, t[0], t[1]));
  const float b = pick(odd, t[3], t[2]) + dpp<0xB1, 0xF, true>(pick(odd, t[2], t[3]));
  if constexpr (S >= 4) {
    r0 = pick(two, b, a) + dpp<0x4E, 0xF, true>(pick(two, a, b));
    r1 = 0.f;
  } else {
    r0 = a;
    r1 = b;
  }
}

// One tile's share of a row-major [token][channel] tensor: this thread's VE
// neighbouring channels of one token.
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
inline int lanes_for(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }  // of 4 states each
inline int blocks_per_group(int Dg, int S) { return (Dg + kThreads / S - 1) / (kThreads / S); }

}  // namespace scan
}  // namespace m3
