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
// A wave holds 16 channels and a block of 4 S states (S = 4, fewer where the state size
// needs no more), lane = 16 s + channel with the states S s .. S s + S - 1: the sums over
// the states of four tokens take three lane swaps and three additions.  What is shared by a
// channel's lanes (delta, u, the gate) or by all channels (B, C) is computed or
// converted once per tile and passed on in LDS.  (This is also the layout of a
// 16 x 16 fp32 matrix product's result; forming u_t B_t^T on the matrix cores
// takes four of 29 vector instructions per token away and is slower all the same:
// 341 us against 317 at Bt 8, L 4096, D 2048, N 16.)
#pragma once
#include "layer_internal.hpp"
#include "m3ssm_internal.hpp"

namespace m3 {
namespace scan {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 256;

// A log2(e), kept finite: a token without a step (delta = 0, as behind an item's
// length) leaves the state alone at A = -inf too.
__device__ __forceinline__ float rate(float A) {
  const float v = A * kLog2e;
  return v < -3.402823466e38f ? -3.402823466e38f : v;
}
// exp(delta A) from that: the hardware exponential, 1 ulp.
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
// The same, and sigmoid(v) = d softplus / dv from the same exponential.
__device__ __forceinline__ float softplus_sigmoid(float v, float& sg) {
  const float u = __builtin_amdgcn_exp2f(-fabsf(v) * kLog2e);
  const float w = 1.f + u;
  const float r = __builtin_amdgcn_rcpf(w);
  sg = v >= 0.f ? r : u * r;
  return fmaxf(v, 0.f) + fmaf(__builtin_amdgcn_logf(w), kLn2, u - (w - 1.f));
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
// How VE neighbouring values are moved: in aligned words of four; in words of four
// with the alignment of the type (widths, state sizes or rows that are no multiples);
// or one at a time, where there are fewer than four channels or states.  8192 tokens
// of 2047 channels fp32 take 154 us in loose words, 253 us one at a time; aligned, 2048 take 140 us.
enum Words { kSingle, kLoose, kAligned };
template <int VE, Words WD>
constexpr int word() {
  return WD == kSingle ? 1 : VE < 4 ? VE : 4;
}
// VE neighbouring values, `ncol` of them inside (any number).  The loads have no
// branch around them (a branch makes the compiler wait for the values at its end): words
// past the edge are read from inside and dropped later, and a loose word across the edge
// is moved back to end there, for unpack_cols to turn.
template <typename T, int VE, Words WD>
__device__ __forceinline__ Pack<T, VE> fetch_cols(const T* p, int ncol) {
  constexpr int VW = word<VE, WD>();
  Pack<T, VE> q;
  if constexpr (WD == kLoose && VW > 1) asm volatile("" : "+v"(ncol));
#pragma unroll
  for (int v = 0; v < VE; v += VW) {
    Pack<T, VW> o;
    if constexpr (WD == kLoose && VW > 1) o = load_loose<T, VW>(p + (v + VW <= ncol ? v : ncol > 0 ? ncol - VW : 0));
    else o = load_pack<T, VW>(p + (v < ncol ? v : 0));
#pragma unroll
    for (int i = 0; i < VW; ++i) q.e[v + i] = o.e[i];
  }
  return q;
}
template <typename T, int VE, Words WD>
__device__ __forceinline__ void unpack_cols(const Pack<T, VE>& q, float* f, int ncol) {
  constexpr int VW = word<VE, WD>();
  unpack<T, VE>(q, f);
  if constexpr (WD == kLoose && VW > 1) {
    if (ncol >= VE) return;
    asm volatile("" : "+v"(ncol));  // computed here, not kept in registers over the tiles
#pragma unroll
    for (int v = 0; v < VE; v += VW) {
      const int back = v + VW - ncol;  // values of the word before it, in front
#pragma unroll
      for (int k = 1; k < VW; ++k) {
#pragma unroll
        for (int i = v; i + 1 < v + VW; ++i) f[i] = back >= k && back < VW ? f[i + 1] : f[i];
      }
    }
  }
}
template <typename T, int VE, Words WD>
__device__ __forceinline__ void store_cols(T* p, const float* v, bool row, int ncol) {
  constexpr int VW = word<VE, WD>(), VP = WD == kLoose ? 1 : VW;  // VP: at the edge
  if (row && VE <= ncol) {
    if constexpr (VW > 1 || VE == 1) {
#pragma unroll
      for (int i = 0; i < VE; i += VW) {
        if constexpr (WD == kLoose && VW > 1) store_loose<T, VW>(p + i, v + i);
        else store_pack<T, VW>(p + i, v + i);
      }
      return;
    }
  }
#pragma unroll
  for (int i = 0; i < VE; i += VP)
    if (row && i < ncol) store_pack<T, VP>(p + i, v + i);
}
// The words for widths of Dg and N; `aligned`: every row and width at whole words.
inline Words words_of(int Dg, int N, bool aligned) { return aligned ? kAligned : Dg >= 4 && N >= 4 ? kLoose : kSingle; }
// The tensors of a call as the kernels take them.
struct Inputs {
  const void* x;
  const void* dt;
  const void* z;
  const void* B;
  const void* C;
  const void* dy;
  int64_t xld, dtld, zld, Bld, Cld;
  const float* Dsk;
  const float* dtb;
  int L, D, N, G, Dg;
};

// A staging thread's part of the tiles of one item and one block of CHB channels:
// VE neighbouring channels of token r of each tensor, and quads of B (and C).
// fetch() starts the loads of a tile into registers; the values are used a tile
// later.  Z, DY, CC: whether z, dy and C are wanted.  TAIL: the rows of a tile that is
// partly past the end lie at its end and not at its start; the rows that fill it have no
// step (delta = u = B = C = do = 0) either way, but in front of the tokens they pass on
// the state in front of the tile, behind them the last one.
template <typename T, int TT, int CHB, int NP, Words WD, bool Z, bool DY, bool CC, bool TAIL = false>
struct Stager {
  static constexpr int VE = TT * CHB / kThreads;
  static constexpr int kQuads = (CC ? 2 : 1) * TT * NP / 4, NQ = (kQuads + kThreads - 1) / kThreads;
  const T *x, *dt, *z, *dy, *B, *C;
  int64_t xld, dtld, zld, dyld, Bld, Cld;
  int r, c0, ncol, cin, tend, N;
  int qt[NQ], qn[NQ];
  bool qc[NQ], gated;
  uint32_t ox, odt, oz, ody, oq[NQ];
  Pack<T, VE> qx, qd, qz, qy;
  Pack<T, 4> qb[NQ];

  __device__ __forceinline__ void init(const Inputs& p, int b, int g, int cb, int tid, int end) {
    r = tid / (CHB / VE);
    c0 = (tid % (CHB / VE)) * VE;
    const int left = p.Dg - (cb * CHB + c0);
    ncol = left < VE ? left : VE;  // channels inside: none past the group
    cin = ncol > 0 ? cb * CHB + c0 : 0;
    tend = end;
    N = p.N;
    gated = p.z != nullptr;
    xld = p.xld;
    dtld = p.dtld;
    zld = gated ? p.zld : p.xld;
    dyld = p.D;
    Bld = p.Bld;
    Cld = p.Cld;
    const int64_t row0 = int64_t(b) * p.L;
    x = static_cast<const T*>(p.x) + row0 * xld + g * p.Dg;
    dt = static_cast<const T*>(p.dt) + row0 * dtld + g * p.Dg;
    z = gated ? static_cast<const T*>(p.z) + row0 * zld + g * p.Dg : x;
    dy = DY ? static_cast<const T*>(p.dy) + row0 * dyld + g * p.Dg : x;
    B = static_cast<const T*>(p.B) + row0 * Bld + int64_t(g) * p.N;
    C = static_cast<const T*>(p.C) + row0 * Cld + int64_t(g) * p.N;
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int e = (tid + i * kThreads) % kQuads;
      qt[i] = (e / (NP / 4)) % TT;
      qn[i] = e % (NP / 4) * 4;
      qc[i] = e / (NP / 4 * TT) == 1;
    }
    place(TT - 1, ox, odt, oz, ody, oq);
    qx = qd = qz = qy = Pack<T, VE>{};
  }
  // row r of a full tile in one whose last row is `last`; whether it is a token's
  static __device__ __forceinline__ int row_of(int r, int last) {
    if (TAIL) return r > TT - 1 - last ? r - (TT - 1 - last) : 0;
    return r < last ? r : last;
  }
  __device__ __forceinline__ bool token(int t0, int r) const { return TAIL ? r >= t0 + TT - tend : t0 + r < tend; }
  // this thread's offsets in a tile whose last row is `last`
  __device__ __forceinline__ void place(int last, uint32_t& px, uint32_t& pdt, uint32_t& pz, uint32_t& pdy, uint32_t (&pq)[NQ]) const {
    const uint32_t rr = row_of(r, last);
    px = rr * uint32_t(xld) + cin;
    pdt = rr * uint32_t(dtld) + cin;
    pz = rr * uint32_t(zld) + cin;
    pdy = rr * uint32_t(dyld) + cin;
#pragma unroll
    for (int i = 0; i < NQ; ++i)
      pq[i] = uint32_t(row_of(qt[i], last)) * uint32_t(qc[i] ? Cld : Bld) + (qn[i] < N ? qn[i] : 0);
  }
  // tend > 0; a tile past the end reads its last row
  __device__ __forceinline__ void fetch(int t0) {
    const int64_t tb = t0 < 0 ? 0 : t0 < tend ? t0 : tend - 1;
    uint32_t px = ox, pdt = odt, pz = oz, pdy = ody, pq[NQ];
#pragma unroll
    for (int i = 0; i < NQ; ++i) pq[i] = oq[i];
    if (tend - 1 - tb < TT - 1) place(int(tend - 1 - tb), px, pdt, pz, pdy, pq);
    qx = fetch_cols<T, VE, WD>(x + tb * xld + px, ncol);
    qd = fetch_cols<T, VE, WD>(dt + tb * dtld + pdt, ncol);
    if constexpr (Z) qz = fetch_cols<T, VE, WD>(z + tb * zld + pz, ncol);
    if constexpr (DY) qy = fetch_cols<T, VE, WD>(dy + tb * dyld + pdy, ncol);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      qb[i] = fetch_cols<T, 4, WD>((qc[i] ? C + tb * Cld : B + tb * Bld) + pq[i], N - qn[i]);
    }
  }
  __device__ __forceinline__ void values(const Pack<T, VE>& q, float* f) const { unpack_cols<T, VE, WD>(q, f, ncol); }
  // B and C of the fetched tile to LDS [2][TT][NP]; zeros past the end and past N
  __device__ __forceinline__ void put_bc(int t0, float* bc) const {
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      float f[4];
      unpack_cols<T, 4, WD>(qb[i], f, N - qn[i]);
      if (t0 + TT > tend || N < NP) {
#pragma unroll
        for (int k = 0; k < 4; ++k) f[k] = qn[i] + k < N && token(t0, qt[i]) ? f[k] : 0.f;
      }
      store_pack<float, 4>(bc + ((qc[i] ? TT : 0) + qt[i]) * NP + qn[i], f);
    }
  }
  // whether value v of the fetched tile lies inside
  __device__ __forceinline__ bool edge(int t0) const { return t0 + TT > tend || ncol < VE; }
  __device__ __forceinline__ bool inside(int t0, int v) const { return token(t0, r) && v < ncol; }
};

// Blocks of channels never straddle two groups.
constexpr int CH = 64;  // channels of a block with one state block: 16 for each of its four scanning waves
inline int state_blocks(int N) { return N <= 16 ? 1 : N <= 32 ? 2 : 4; }  // of at most 16 states
// States of a lane, S: as many as make a block's 4 S of a channel's four lanes enough.
// 8192 tokens of 2048 channels bf16 with N = 4, 8, 12, 16, 24, 32 take 75, 93, 115, 125,
// 144, 153 us, the backward 208, 231, 301, 315, 527, 581 us; padded to whole blocks of 16
// states, the first three took what 16 does and the fifth what 32 does.
inline int lane_states(int N) { return (N + 4 * state_blocks(N) - 1) / (4 * state_blocks(N)); }
template <int S>
struct States {
  typedef float type __attribute__((ext_vector_type(S), aligned(S == 3 ? 4 : 4 * S)));
};
template <int S>
__device__ __forceinline__ typename States<S>::type load_states(const float* p) {
  return *reinterpret_cast<const typename States<S>::type*>(p);
}
// The kernels for a state size: CALL(NB, S).
#define M3_SCAN_STATES(N, CALL)     \
  if ((N) <= 4) return CALL(1, 1);  \
  if ((N) <= 8) return CALL(1, 2);  \
  if ((N) <= 12) return CALL(1, 3); \
  if ((N) <= 16) return CALL(1, 4); \
  if ((N) <= 24) return CALL(2, 3); \
  if ((N) <= 32) return CALL(2, 4); \
  if ((N) <= 48) return CALL(4, 3); \
  return CALL(4, 4);
inline int blocks_per_group(int Dg, int NB) { return (Dg + CH / NB - 1) / (CH / NB); }

}  // namespace scan
}  // namespace m3
