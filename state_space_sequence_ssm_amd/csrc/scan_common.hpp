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

// Sum over the S neighbouring lanes of a channel, in each of them.
template <int S>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (S >= 2) v += dpp<0xB1, 0xF, true>(v);    // lane ^ 1
  if constexpr (S >= 4) v += dpp<0x4E, 0xF, true>(v);    // lane ^ 2
  if constexpr (S >= 8) v += dpp<0x141, 0xF, true>(v);   // mirrored within 8
  if constexpr (S >= 16) v += dpp<0x140, 0xF, true>(v);  // mirrored within 16
  return v;
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
struct Split {
  int S;      // lanes per channel (4 states each)
  int nblk;   // blocks per group
};
inline int lanes_for(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
inline Split split_of(int D, int N, int G) {
  Split q;
  q.S = lanes_for(N);
  const int CH = kThreads / q.S;
  q.nblk = (D / G + CH - 1) / CH;
  return q;
}

}  // namespace scan
}  // namespace m3
