// Backward of the selective scan (see scan_common.hpp for the forward's layout).
//
// With do_t = dy_t silu(z_t) and g_t the gradient of the state after token t:
//   g_t = C_t do_t + a_{t+1} g_{t+1},      a_t = exp(delta_t A)
//   dC_t[n] = sum_d do_t h_t,   dB_t[n] = sum_d g_t u_t
//   dx_t = D do_t + delta_t sum_n g_t B_t
//   ddelta_t = x_t sum_n g_t B_t + sum_n g_t (a_t h_{t-1}) A
//   dA = sum_t g_t (a_t h_{t-1}) delta_t,   dz_t = dy_t o_t silu'(z_t)
//
// Two walks.  The first runs forward over the tokens and keeps the state in
// front of every 16th one.  The second walks these 16-token tiles from the last
// to the first: it computes a tile's decays and states again, keeps them in
// registers (2 x 16 x 4 per lane) and runs the reverse recurrence over them, so
// each decay is computed twice in all and no state goes to memory per token.
// dB and dC are summed over a wave's channels by lane swaps, over the block's
// waves in LDS and over the blocks from a workspace in a fixed order.
// The token axis can be cut into segments walked at once: the first walk then
// starts every segment from zero and also forms, in the same forward pass, what
// the segment contributes to the gradient in front of it,
//   sum_t (prod_{r<=t} a_r) C_t do_t,
// and the second walk joins states from the left and gradients from the right.
#include "scan_common.hpp"

namespace m3 {
namespace scan {
namespace {

constexpr int TB = 16;  // tokens per tile of the reverse walk
inline int lanes_for(int N) { return N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }  // of 4 states each
inline int blocks_per_group(int Dg, int S) { return (Dg + kThreads / S - 1) / (kThreads / S); }
template <int S>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (S >= 2) v += dpp<0xB1, 0xF, true>(v);    // lane ^ 1
  if constexpr (S >= 4) v += dpp<0x4E, 0xF, true>(v);    // lane ^ 2
  if constexpr (S >= 8) v += dpp<0x141, 0xF, true>(v);   // mirrored within 8
  if constexpr (S >= 16) v += dpp<0x140, 0xF, true>(v);  // mirrored within 16
  return v;
}

struct BwP {
  const void* x;
  const void* dt;
  const void* z;
  const void* B;
  const void* C;
  const void* dy;
  int64_t xld, dtld, zld, Bld, Cld;
  const float* A;
  const float* Dsk;
  const float* dtb;
  const float* h0;
  const float* dhf;
  const int32_t* lengths;
  void* dx;
  void* ddt;
  void* dz;
  float* dh0;
  float* ck;    // [tiles][blocks][256][4] state in front of each tile (of its segment from zero)
  float* cd;    // [tiles][blocks][CH] sum of delta from the segment's start to the tile
  float* hend;  // [nseg][Bt][D][N] state of a segment from zero (segment 0: from h0)
  float* gsum;  // [nseg][Bt][D][N] a segment's contribution to the gradient in front of it
  float* sdel;  // [nseg][Bt][D] sum of delta
  float* bc;    // [nblk][Bt * L][G][2][NP] sums of dB and dC over a block's channels
  float* part;  // [nseg * Bt][D * N + D + D] sums of dA, dD, ddt_bias
  int Bt, L, D, N, G, Dg, nblk, nseg, seglen, softplus;
};

// First walk: states in front of the tiles, and with SEG the segments' ends.
template <typename T, int S, bool VEC, bool SEG>
__global__ __launch_bounds__(kThreads) void states_kernel(BwP p) {
  constexpr int K = 4, CH = kThreads / S, TT = S >= 4 ? 32 : 16, VE = TT / S, NP = K * S;
  constexpr int NQ = (TT * NP / 2 + kThreads - 1) / kThreads;
  __shared__ __align__(16) float2 du[TT][CH];
  __shared__ __align__(16) float bc[SEG ? 2 : 1][TT][NP];
  __shared__ __align__(16) float dos[SEG ? TT : 1][CH];

  const int tid = threadIdx.x, s = tid % S, chl = tid / S;
  int blk = block_on_xcd();
  const int64_t blocks = int64_t(p.Bt) * p.G * p.nblk;
  const int seg = int(blk / blocks);
  blk = int(blk - seg * blocks);
  const int64_t unit = blk;
  const int cb = blk % p.nblk;
  blk /= p.nblk;
  const int g = blk % p.G, b = blk / p.G;
  const int len = item_length(p.lengths, b, p.L);
  const int tbeg = seg * p.seglen;
  const int tend = tbeg + p.seglen < len ? tbeg + p.seglen : len;

  const int dl = cb * CH + chl;
  const bool live = dl < p.Dg;
  const int d = g * p.Dg + (live ? dl : 0);
  float A2[K], h[K], P[K], gs[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int n = s * K + k;
    const bool on = live && n < p.N;
    A2[k] = on ? p.A[int64_t(d) * p.N + n] * kLog2e : 0.f;
    h[k] = on && p.h0 != nullptr && seg == 0 ? p.h0[(int64_t(b) * p.D + d) * p.N + n] : 0.f;
    P[k] = 1.f;
    gs[k] = 0.f;
  }
  float sum_delta = 0.f;

  const int r = tid / (CH / VE), c0 = (tid % (CH / VE)) * VE;
  const int ncol = p.Dg - (cb * CH + c0) < VE ? p.Dg - (cb * CH + c0) : VE;
  const int dc = g * p.Dg + cb * CH + c0;
  const int64_t row0 = int64_t(b) * p.L;
  const T* xp = static_cast<const T*>(p.x) + row0 * p.xld + dc;
  const T* dtp = static_cast<const T*>(p.dt) + row0 * p.dtld + dc;
  const T* zp = p.z == nullptr ? nullptr : static_cast<const T*>(p.z) + row0 * p.zld + dc;
  const T* dyp = static_cast<const T*>(p.dy) + row0 * p.D + dc;
  float bias[VE];
#pragma unroll
  for (int v = 0; v < VE; ++v) bias[v] = p.dtb != nullptr && v < ncol ? p.dtb[dc + v] : 0.f;
  const bool bcvec = VEC && p.N % 4 == 0;

  Pack<T, VE> qx{}, qd{}, qz{}, qy{};
  Pack<T, 4> qb[NQ];
  auto fetch = [&](int t0) {
    const int t = t0 + r;
    const bool row = t < tend;
    qx = load_cols<T, VE, VEC>(xp + int64_t(t) * p.xld, row, ncol);
    qd = load_cols<T, VE, VEC>(dtp + int64_t(t) * p.dtld, row, ncol);
    if constexpr (SEG) {
      qy = load_cols<T, VE, VEC>(dyp + int64_t(t) * p.D, row, ncol);
      if (zp != nullptr) qz = load_cols<T, VE, VEC>(zp + int64_t(t) * p.zld, row, ncol);
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int e = tid + i * kThreads, q = e % (NP / 4), tt = (e / (NP / 4)) % TT, which = e / (NP / 4 * TT);
      qb[i] = Pack<T, 4>{};
      if (which < (SEG ? 2 : 1) && t0 + tt < tend && 4 * q < p.N) {
        const int64_t ld = which ? p.Cld : p.Bld;
        const T* src = static_cast<const T*>(which ? p.C : p.B) + (row0 + t0 + tt) * ld + int64_t(g) * p.N + 4 * q;
        qb[i] = bcvec ? load_pack<T, 4>(src) : load_some<T, 4>(src, p.N - 4 * q);
      }
    }
  };
  if (tbeg < tend) fetch(tbeg);
  for (int t0 = tbeg; t0 < tend; t0 += TT) {
#pragma unroll
    for (int v = 0; v < VE; ++v) {
      const float dl_ = step_of(to_f32(qd.e[v]), p.softplus != 0, bias[v], t0 + r < tend);
      du[r][c0 + v] = float2{dl_, dl_ * to_f32(qx.e[v])};
      if constexpr (SEG) dos[r][c0 + v] = to_f32(qy.e[v]) * (zp != nullptr ? silu_f(to_f32(qz.e[v])) : 1.f);
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int e = tid + i * kThreads, q = e % (NP / 4), tt = (e / (NP / 4)) % TT, which = e / (NP / 4 * TT);
      if (which < (SEG ? 2 : 1)) {
        float f[4];
        unpack<T, 4>(qb[i], f);
        *reinterpret_cast<f32x4*>(&bc[which][tt][4 * q]) = f32x4{f[0], f[1], f[2], f[3]};
      }
    }
    __syncthreads();
    if (t0 + TT < tend) fetch(t0 + TT);
    const int nt = tend - t0 < TT ? (tend - t0 + 3) & ~3 : TT;
    for (int tq = 0; tq < nt; tq += 4) {
      if (tq % TB == 0) {
        const int64_t at = int64_t((t0 + tq) / TB) * blocks + unit;
        store_pack<float, 4>(p.ck + (at * kThreads + tid) * 4, h);
        if (SEG && s == 0) p.cd[at * CH + chl] = sum_delta;
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int t = tq + i;
        const float2 q = du[t][chl];
        if constexpr (SEG) sum_delta += q.x;
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const float a = decay(q.x, A2[k]);
          h[k] = fmaf(a, h[k], q.y * bc[0][t][s * K + k]);
          if constexpr (SEG) {
            P[k] *= a;
            gs[k] = fmaf(P[k], bc[1][t][s * K + k] * dos[t][chl], gs[k]);
          }
        }
      }
    }
    __syncthreads();
  }
  if constexpr (SEG) {
    if (!live) return;
    const int64_t at = (int64_t(seg) * p.Bt + b) * p.D + d;
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (s * K + k < p.N) {
        p.hend[at * p.N + s * K + k] = h[k];
        p.gsum[at * p.N + s * K + k] = gs[k];
      }
    if (s == 0) p.sdel[at] = sum_delta;
  }
}

// Sum of v[0..3] over a wave's channels (the lanes equal modulo S).  Row q of
// 16 lanes ends with the sums of v[{0, 2, 1, 3}[q]], in every one of its lanes
// of the same state group.
template <int S>
__device__ __forceinline__ float channels_sum(const float* v) {
  auto swap32 = [](float a, float b) {
    const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
    return __uint_as_float(r[0]) + __uint_as_float(r[1]);
  };
  const float lo = swap32(v[0], v[1]), hi = swap32(v[2], v[3]);
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(lo), __float_as_uint(hi), false, false);
  float t = __uint_as_float(r[0]) + __uint_as_float(r[1]);
  if constexpr (S <= 8) t += dpp<0x128, 0xF, true>(t);  // rotated by 8 within 16
  if constexpr (S <= 4) t += dpp<0x124, 0xF, true>(t);  // by 4
  if constexpr (S <= 2) t += dpp<0x122, 0xF, true>(t);  // by 2
  return t;
}

// Second walk.
template <typename T, int S, bool VEC>
__global__ __launch_bounds__(kThreads) void reverse_kernel(BwP p) {
  constexpr int K = 4, CH = kThreads / S, VE = TB / S, NP = K * S;
  constexpr int NQ = (TB * NP / 2 + kThreads - 1) / kThreads;
  constexpr int YS = CH + 64 / S;
  __shared__ __align__(16) float2 du[TB][CH];
  __shared__ __align__(16) float dos[TB][CH];
  __shared__ __align__(16) float bc[2][TB][NP];
  __shared__ __align__(16) float os[TB][YS];
  __shared__ __align__(16) float gb[2][TB][YS];
  __shared__ __align__(16) float wp[4][TB][2][NP];

  const int tid = threadIdx.x, s = tid % S, chl = tid / S, lane = tid & 63, wv = tid >> 6;
  int blk = block_on_xcd();
  const int64_t blocks = int64_t(p.Bt) * p.G * p.nblk;
  const int seg = int(blk / blocks);
  blk = int(blk - seg * blocks);
  const int64_t unit = blk;
  const int cb = blk % p.nblk;
  blk /= p.nblk;
  const int g = blk % p.G, b = blk / p.G;
  const int len = item_length(p.lengths, b, p.L);
  const int tbeg = seg * p.seglen;
  const int tlim = tbeg + p.seglen < p.L ? tbeg + p.seglen : p.L;
  const int tend = tlim < len ? tlim : len;

  const int dl = cb * CH + chl;
  const bool live = dl < p.Dg;
  const int d = g * p.Dg + (live ? dl : 0);
  const int64_t at0 = int64_t(b) * p.D + d;
  float A2[K], gg[K], hin[K], dA[K];
#pragma unroll
  for (int k = 0; k < K; ++k) {
    const int n = s * K + k;
    const bool on = live && n < p.N;
    A2[k] = on ? p.A[int64_t(d) * p.N + n] * kLog2e : 0.f;
    gg[k] = on && p.dhf != nullptr ? p.dhf[at0 * p.N + n] : 0.f;
    hin[k] = 0.f;
    dA[k] = 0.f;
  }
  const int64_t per = int64_t(p.Bt) * p.D;
  for (int q = 0; q < seg; ++q) {  // state in front of the segment
    const float sd = p.sdel[q * per + at0];
#pragma unroll
    for (int k = 0; k < K; ++k)
      hin[k] = fmaf(decay(sd, A2[k]), hin[k], s * K + k < p.N ? p.hend[(q * per + at0) * p.N + s * K + k] : 0.f);
  }
  for (int q = p.nseg - 1; q > seg; --q) {  // gradient behind it
    const float sd = p.sdel[q * per + at0];
#pragma unroll
    for (int k = 0; k < K; ++k)
      gg[k] = fmaf(decay(sd, A2[k]), gg[k], s * K + k < p.N ? p.gsum[(q * per + at0) * p.N + s * K + k] : 0.f);
  }

  const int r = tid / (CH / VE), c0 = (tid % (CH / VE)) * VE;
  const int ncol = p.Dg - (cb * CH + c0) < VE ? p.Dg - (cb * CH + c0) : VE;
  const int dc = g * p.Dg + cb * CH + c0;
  const int64_t row0 = int64_t(b) * p.L;
  const T* xp = static_cast<const T*>(p.x) + row0 * p.xld + dc;
  const T* dtp = static_cast<const T*>(p.dt) + row0 * p.dtld + dc;
  const T* zp = p.z == nullptr ? nullptr : static_cast<const T*>(p.z) + row0 * p.zld + dc;
  const T* dyp = static_cast<const T*>(p.dy) + row0 * p.D + dc;
  T* dxp = static_cast<T*>(p.dx) + row0 * p.D + dc;
  T* ddtp = static_cast<T*>(p.ddt) + row0 * p.D + dc;
  T* dzp = p.dz == nullptr ? nullptr : static_cast<T*>(p.dz) + row0 * p.D + dc;
  float bias[VE], dsk[VE], dD[VE], dbias[VE];
#pragma unroll
  for (int v = 0; v < VE; ++v) {
    bias[v] = p.dtb != nullptr && v < ncol ? p.dtb[dc + v] : 0.f;
    dsk[v] = p.Dsk != nullptr && v < ncol ? p.Dsk[dc + v] : 0.f;
    dD[v] = dbias[v] = 0.f;
  }
  const bool bcvec = VEC && p.N % 4 == 0;
  // rows behind the item's length: zero gradients
  for (int t = (tend > tbeg ? tend : tbeg) + r; t < tlim; t += TB) {
    float zero[VE];
#pragma unroll
    for (int v = 0; v < VE; ++v) zero[v] = 0.f;
    store_cols<T, VE, VEC>(dxp + int64_t(t) * p.D, zero, true, ncol);
    store_cols<T, VE, VEC>(ddtp + int64_t(t) * p.D, zero, true, ncol);
    if (dzp != nullptr) store_cols<T, VE, VEC>(dzp + int64_t(t) * p.D, zero, true, ncol);
  }

  Pack<T, VE> qx{}, qd{}, qz{}, qy{};
  Pack<T, 4> qb[NQ];
  Pack<float, 4> qh{};
  float qcd = 0.f;
  auto fetch = [&](int t0) {
    const int t = t0 + r;
    const bool row = t < tend;
    qx = load_cols<T, VE, VEC>(xp + int64_t(t) * p.xld, row, ncol);
    qd = load_cols<T, VE, VEC>(dtp + int64_t(t) * p.dtld, row, ncol);
    qy = load_cols<T, VE, VEC>(dyp + int64_t(t) * p.D, row, ncol);
    if (zp != nullptr) qz = load_cols<T, VE, VEC>(zp + int64_t(t) * p.zld, row, ncol);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int e = tid + i * kThreads, q = e % (NP / 4), tt = (e / (NP / 4)) % TB, which = e / (NP / 4 * TB);
      qb[i] = Pack<T, 4>{};
      if (which < 2 && t0 + tt < tend && 4 * q < p.N) {
        const int64_t ld = which ? p.Cld : p.Bld;
        const T* src = static_cast<const T*>(which ? p.C : p.B) + (row0 + t0 + tt) * ld + int64_t(g) * p.N + 4 * q;
        qb[i] = bcvec ? load_pack<T, 4>(src) : load_some<T, 4>(src, p.N - 4 * q);
      }
    }
    const int64_t at = int64_t(t0 / TB) * blocks + unit;
    qh = load_pack<float, 4>(p.ck + (at * kThreads + tid) * 4);
    if (seg > 0) qcd = p.cd[at * CH + chl];
  };
  const int tlast = tend > tbeg ? tbeg + (tend - tbeg - 1) / TB * TB : tbeg - TB;
  if (tlast >= tbeg) fetch(tlast);
  for (int t0 = tlast; t0 >= tbeg; t0 -= TB) {
    // ---- stage the tile
    const bool row = t0 + r < tend;
    float xv[VE], raw[VE], dov[VE], yv[VE], zv[VE];
    unpack<T, VE>(qx, xv);
    unpack<T, VE>(qd, raw);
    unpack<T, VE>(qy, yv);
    unpack<T, VE>(qz, zv);
#pragma unroll
    for (int v = 0; v < VE; ++v) {
      const float dl_ = step_of(raw[v], p.softplus != 0, bias[v], row);
      du[r][c0 + v] = float2{dl_, dl_ * xv[v]};
      dov[v] = yv[v] * (zp != nullptr ? silu_f(zv[v]) : 1.f);
      dos[r][c0 + v] = dov[v];
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int e = tid + i * kThreads, q = e % (NP / 4), tt = (e / (NP / 4)) % TB, which = e / (NP / 4 * TB);
      if (which < 2) {
        float f[4];
        unpack<T, 4>(qb[i], f);
        *reinterpret_cast<f32x4*>(&bc[which][tt][4 * q]) = f32x4{f[0], f[1], f[2], f[3]};
      }
    }
    float h[K];
#pragma unroll
    for (int k = 0; k < K; ++k) h[k] = seg > 0 ? fmaf(decay(qcd, A2[k]), hin[k], qh.e[k]) : qh.e[k];
    __syncthreads();
    if (t0 - TB >= tbeg) fetch(t0 - TB);
    // ---- decays and states of the tile, forward
    float a[TB][K], ah[TB][K];
    float keep = 0.f;
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      const float2 q = du[t][chl];
      float o = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        a[t][k] = decay(q.x, A2[k]);
        ah[t][k] = a[t][k] * h[k];
        h[k] = fmaf(q.y, bc[0][t][s * K + k], ah[t][k]);
        o = fmaf(bc[1][t][s * K + k], h[k], o);
      }
      o = lanes_sum<S>(o);
      if (s == (S >= 4 ? t & 3 : t & 1)) keep = o;
      if (S >= 4 ? (t & 3) == 3 : (t & 1)) {
        if (s < 4) os[S >= 4 ? t - 3 + s : t - 1 + s][chl] = keep;
      }
    }
    // ---- gradients, backward
    float dAt[K] = {0.f, 0.f, 0.f, 0.f};
    float keepB = 0.f, keepA = 0.f;
#pragma unroll
    for (int t = TB - 1; t >= 0; --t) {
      const float2 q = du[t][chl];
      const float dot = dos[t][chl];
      float gu[K], dh[K], sB = 0.f, sA = 0.f;
#pragma unroll
      for (int k = 0; k < K; ++k) {
        const float Bv = bc[0][t][s * K + k], Cv = bc[1][t][s * K + k];
        const float gk = fmaf(Cv, dot, gg[k]);
        const float hk = fmaf(q.y, Bv, ah[t][k]);
        dh[k] = dot * hk;
        gu[k] = gk * q.y;
        sB = fmaf(gk, Bv, sB);
        const float w = gk * ah[t][k];
        sA = fmaf(w, A2[k], sA);
        dAt[k] = fmaf(w, q.x, dAt[k]);
        gg[k] = gk * a[t][k];
      }
      sB = lanes_sum<S>(sB);
      sA = lanes_sum<S>(sA);
      if (s == (S >= 4 ? t & 3 : t & 1)) {
        keepB = sB;
        keepA = sA;
      }
      if (S >= 4 ? (t & 3) == 0 : (t & 1) == 0) {
        if (s < 4) {
          gb[0][t + s][chl] = keepB;
          gb[1][t + s][chl] = keepA;
        }
      }
      const float rB = channels_sum<S>(gu), rC = channels_sum<S>(dh);
      const int rowq = lane >> 4, n = s * 4 + ((rowq & 1) << 1 | rowq >> 1);
      if constexpr (S <= 8) {
        const int which = (lane & 15) / S;
        if (which < 2) wp[wv][t][which][n] = which ? rC : rB;
      } else {
        wp[wv][t][0][n] = rB;
        wp[wv][t][1][n] = rC;
      }
    }
#pragma unroll
    for (int k = 0; k < K; ++k) dA[k] += dAt[k];
    __syncthreads();
    // ---- outputs of the tile
    float ox[VE], od[VE], oz[VE];
#pragma unroll
    for (int v = 0; v < VE; ++v) {
      const float gB = gb[0][r][c0 + v], gA = gb[1][r][c0 + v];
      const float dl_ = du[r][c0 + v].x;
      ox[v] = fmaf(dsk[v], dov[v], dl_ * gB);
      od[v] = fmaf(xv[v], gB, gA * kLn2);
      if (p.softplus) od[v] *= sigmoid_f(raw[v] + bias[v]);
      if (row) {
        dD[v] = fmaf(dov[v], xv[v], dD[v]);
        dbias[v] += od[v];
      }
      oz[v] = zp != nullptr ? yv[v] * fmaf(dsk[v], xv[v], os[r][c0 + v]) * dsilu_f(zv[v], sigmoid_f(zv[v])) : 0.f;
    }
    store_cols<T, VE, VEC>(dxp + int64_t(t0 + r) * p.D, ox, row, ncol);
    store_cols<T, VE, VEC>(ddtp + int64_t(t0 + r) * p.D, od, row, ncol);
    if (dzp != nullptr) store_cols<T, VE, VEC>(dzp + int64_t(t0 + r) * p.D, oz, row, ncol);
    for (int i = tid; i < TB * 2 * NP; i += kThreads) {
      const int t = i / (2 * NP), e = i % (2 * NP);
      const float* w0 = &wp[0][t][0][0] + e;
      const float v = (w0[0] + w0[TB * 2 * NP]) + (w0[2 * TB * 2 * NP] + w0[3 * TB * 2 * NP]);
      if (t0 + t < tend)
        p.bc[((int64_t(cb) * p.Bt * p.L + row0 + t0 + t) * p.G + g) * (2 * NP) + e] = v;
    }
    __syncthreads();  // du is read above and written by the next tile
  }
  // ---- sums over the tokens
  const int64_t ncols = int64_t(p.D) * (p.N + 2);
  float* part = p.part + (int64_t(seg) * p.Bt + b) * ncols;
  if (live) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int n = s * K + k;
      if (n < p.N) {
        part[int64_t(d) * p.N + n] = dA[k];
        if (seg == 0 && p.dh0 != nullptr) p.dh0[at0 * p.N + n] = gg[k];
      }
    }
  }
  __syncthreads();
#pragma unroll
  for (int v = 0; v < VE; ++v) {
    os[r][c0 + v] = dD[v];
    gb[0][r][c0 + v] = dbias[v];
  }
  __syncthreads();
  if (tid < CH && cb * CH + tid < p.Dg) {
    float sd = 0.f, sb = 0.f;
#pragma unroll
    for (int q = 0; q < TB; ++q) {
      sd += os[q][tid];
      sb += gb[0][q][tid];
    }
    const int dd = g * p.Dg + cb * CH + tid;
    part[int64_t(p.D) * p.N + dd] = sd;
    part[int64_t(p.D) * (p.N + 1) + dd] = sb;
  }
}

// dB and dC: sums of the blocks' parts, rounded once; zeros behind the lengths.
template <typename T, int NP>
__global__ __launch_bounds__(256) void join_bc_kernel(const float* bc, T* dB, T* dC, const int32_t* lengths, int64_t rows,
                                                      int L, int G, int N, int nblk) {
  const int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t total = rows * G * 2 * NP;
  if (i >= total) return;
  const int n = int(i % NP), which = int(i / NP) & 1;
  const int64_t rg = i / (2 * NP), row = rg / G;
  if (n >= N) return;
  float v = 0.f;
  const int64_t b = row / L;
  if (lengths == nullptr || row - b * L < item_length(lengths, int(b), L)) {
#pragma unroll 8
    for (int q = 0; q < nblk; ++q) v += bc[q * total + i];
  }
  from_f32(v, (which ? dC : dB)[rg * N + n]);
}

struct Plan {
  int S, nblk, nseg, seglen;
  int64_t tiles, blocks;
  size_t oCk, oCd, oHe, oGs, oSd, oBc, oPart, bytes;
};
// Segments as in the forward, at least 128 tokens each, multiples of the tiles.
Plan plan_of(const m3_scan_args& f) {
  Plan p;
  p.S = lanes_for(f.N);
  p.nblk = blocks_per_group(f.D / f.G, p.S);
  p.blocks = int64_t(f.Bt) * f.G * p.nblk;
  p.nseg = 1;
  p.seglen = (f.L + 31) / 32 * 32;
  if (p.blocks < 512) {
    int64_t n = (512 + p.blocks - 1) / p.blocks;
    if (n > f.L / 128) n = f.L / 128;
    if (n > 1) {
      p.seglen = int(((f.L + n - 1) / n + 31) / 32 * 32);
      p.nseg = (f.L + p.seglen - 1) / p.seglen;
    }
  }
  p.tiles = (f.L + TB - 1) / TB;
  const int CH = kThreads / p.S, NP = 4 * p.S;
  const size_t seg = p.nseg > 1 ? size_t(p.nseg) * f.Bt * f.D : 0;
  p.oCk = 0;
  p.oCd = round256(p.oCk + size_t(p.tiles) * p.blocks * kThreads * 16);
  p.oHe = round256(p.oCd + (p.nseg > 1 ? size_t(p.tiles) * p.blocks * CH * 4 : 0));
  p.oGs = round256(p.oHe + seg * f.N * 4);
  p.oSd = round256(p.oGs + seg * f.N * 4);
  p.oBc = round256(p.oSd + seg * 4);
  p.oPart = round256(p.oBc + size_t(p.nblk) * f.Bt * f.L * f.G * 2 * NP * 4);
  p.bytes = round256(p.oPart + size_t(p.nseg) * f.Bt * f.D * (f.N + 2) * 4);
  return p;
}

template <typename T, int S, bool VEC>
hipError_t run(const m3_scan_backward_args& a, hipStream_t st) {
  const m3_scan_args& f = a.fwd;
  const Plan pl = plan_of(f);
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  const BwP p{f.x, f.dt, f.z, f.B, f.C, a.dy, f.x_ld, f.dt_ld, f.z_ld, f.B_ld, f.C_ld, f.A, f.D_skip, f.dt_bias, f.h0,
              a.dh_final, f.lengths, a.dx, a.ddt, a.dz, a.dh0, at(pl.oCk), at(pl.oCd), at(pl.oHe), at(pl.oGs), at(pl.oSd),
              at(pl.oBc), at(pl.oPart), f.Bt, f.L, f.D, f.N, f.G, f.D / f.G, pl.nblk, pl.nseg, pl.seglen, f.dt_softplus};
  const uint32_t grid = uint32_t(pl.blocks * pl.nseg);
  if (pl.nseg > 1) states_kernel<T, S, VEC, true><<<grid, kThreads, 0, st>>>(p);
  else states_kernel<T, S, VEC, false><<<grid, kThreads, 0, st>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  reverse_kernel<T, S, VEC><<<grid, kThreads, 0, st>>>(p);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  const int64_t rows = int64_t(f.Bt) * f.L, items = rows * f.G * 2 * 4 * S;
  join_bc_kernel<T, 4 * S><<<uint32_t((items + 255) / 256), 256, 0, st>>>(p.bc, static_cast<T*>(a.dB), static_cast<T*>(a.dC),
                                                                        f.lengths, rows, f.L, f.G, f.N, pl.nblk);
  e = hipGetLastError();
  if (e != hipSuccess) return e;
  ColSum c{};
  c.part = p.part;
  c.P = int64_t(pl.nseg) * f.Bt;
  c.ncols = int64_t(f.D) * (f.N + 2);
  c.dst[0] = a.dA;
  c.n[0] = int64_t(f.D) * f.N;
  c.dst[1] = a.dD;
  c.n[1] = f.D;
  c.dst[2] = a.ddt_bias;
  c.n[2] = f.D;
  return launch_colsum(c, st);
}

template <typename T, bool VEC>
hipError_t by_lanes(const m3_scan_backward_args& a, hipStream_t st) {
  switch (lanes_for(a.fwd.N)) {
    case 2: return run<T, 2, VEC>(a, st);
    case 4: return run<T, 4, VEC>(a, st);
    case 8: return run<T, 8, VEC>(a, st);
    default: return run<T, 16, VEC>(a, st);
  }
}

}  // namespace
}  // namespace scan

size_t scan_backward_workspace(const m3_scan_backward_args& a) { return scan::plan_of(a.fwd).bytes; }
hipError_t launch_scan_backward(const m3_scan_backward_args& a, hipStream_t s) {
  const m3_scan_args& f = a.fwd;
  const bool bf = f.in_dtype == M3_BF16;
  const size_t e = bf ? 2 : 4;
  // the first walk's staging threads take the wider words
  const int S = scan::lanes_for(f.N), ve = (S >= 4 ? 32 : 16) / S;
  const size_t word = e * ve < 16 ? e * ve : 16;
  const bool vec = (f.D / f.G) % ve == 0 && rows_aligned(f.x, f.x_ld, e, word) && rows_aligned(f.dt, f.dt_ld, e, word) &&
                   rows_aligned(f.z, f.z_ld, e, word) && rows_aligned(a.dy, f.D, e, word) && rows_aligned(a.dx, f.D, e, word) &&
                   rows_aligned(a.ddt, f.D, e, word) && rows_aligned(a.dz, f.D, e, word) &&
                   (f.N % 4 != 0 || (rows_aligned(f.B, f.B_ld, e, 4 * e) && rows_aligned(f.C, f.C_ld, e, 4 * e)));
  if (bf) return vec ? scan::by_lanes<bf16_t, true>(a, s) : scan::by_lanes<bf16_t, false>(a, s);
  return vec ? scan::by_lanes<float, true>(a, s) : scan::by_lanes<float, false>(a, s);
}

}  // namespace m3
