// Backward of the selective scan (see scan_common.hpp for the forward).
//
// With do_t = dy_t silu(z_t) and g_t the gradient of the state after token t:
//   g_t = C_t do_t + a_{t+1} g_{t+1},      a_t = exp(delta_t A)
//   dC_t[n] = sum_d do_t h_t = sum_d do_t (a_t h_{t-1}) + B_t[n] sum_d do_t u_t
//   dB_t[n] = sum_d g_t u_t
//   dx_t = D do_t + delta_t sum_n g_t B_t
//   ddelta_t = x_t sum_n g_t B_t + sum_n g_t (a_t h_{t-1}) A
//   dA = sum_t g_t (a_t h_{t-1}) delta_t,   dz_t = dy_t o_t silu'(z_t)
//
// Two walks.  The first runs forward over the tokens and keeps the state in
// front of every 16th one.  The second walks these 16-token tiles from the last
// to the first: it computes a tile's decays and states again, keeps them in
// registers (2 x 16 x S per lane) and runs the reverse recurrence over them, so
// each decay is computed twice in all and no state goes to memory per token.
// dB and dC are summed over a wave's 16 channels in registers, over the block's
// waves in LDS and over the blocks from a workspace, in a fixed order.
// The token axis can be cut into segments walked at once: the first walk then
// starts every segment from zero and also forms, in the same forward pass, what
// the segment contributes to the gradient in front of it,
//   sum_t (prod_{r<=t} a_r) C_t do_t,
// and the second walk joins states from the left and gradients from the right.
//
// A wave holds 16 channels and one block of 4 S states, lane = 16 s + channel
// with the states S s .. S s + S - 1; a block of eight waves (four scan, four stage) is
// 64 / NB channels of NB state blocks, whose sums over the states the staging
// waves join.
#include <type_traits>

#include "scan_common.hpp"

namespace m3 {
namespace scan {
namespace {

constexpr int TB = 16;  // tokens per tile of the reverse walk, and between two kept states

struct BwP {
  Inputs in;
  const float* A;
  const float* h0;
  const float* dhf;
  const int32_t* lengths;
  void* dx;
  void* ddt;
  void* dz;
  float* dh0;
  float* ck;    // [tiles][blocks][256][S] state in front of each tile (of its segment from zero)
  float* cd;    // [tiles][blocks][CHB] sum of delta from the segment's start to the tile
  float* hend;  // [nseg][Bt][D][N] state of a segment from zero (segment 0: from h0)
  float* gsum;  // [nseg][Bt][D][N] a segment's contribution to the gradient in front of it
  float* sdel;  // [nseg][Bt][D] sum of delta
  float* bc;    // [nblk][Bt * L][G][2][NP] sums of dB and dC over a block's channels
  float* part;  // [nseg * Bt][D * N + D + D] sums of dA, dD, ddt_bias
  int Bt, nblk, nseg, seglen, softplus;
};

// Where a block and a scanning lane are.
template <int NB>
struct Where {
  static constexpr int CHB = CH / NB;
  int64_t blocks, unit;
  int seg, cb, g, b, tbeg, tlim, tend;
  __device__ __forceinline__ explicit Where(const BwP& p) {
    int blk = block_on_xcd();
    blocks = int64_t(p.Bt) * p.in.G * p.nblk;
    seg = int(blk / blocks);
    blk = int(blk - seg * blocks);
    unit = blk;
    cb = blk % p.nblk;
    blk /= p.nblk;
    g = blk % p.in.G;
    b = blk / p.in.G;
    const int len = item_length(p.lengths, b, p.in.L);
    tbeg = seg * p.seglen;
    tlim = tbeg + p.seglen < p.in.L ? tbeg + p.seglen : p.in.L;
    tend = tlim < len ? tlim : len;
  }
};
template <int NB, int S>
struct Lane {
  int s, chl, n0, d, nleft;  // state group, channel in the block, first state, channel, states left from n0
  bool live;
  __device__ __forceinline__ Lane(const BwP& p, const Where<NB>& w, int tid) {
    const int wave = tid >> 6;
    s = (tid & 63) >> 4;
    chl = (wave / NB) * 16 + (tid & 15);
    n0 = (wave % NB * 4 + s) * S;
    nleft = p.in.N - n0;
    const int dl = w.cb * Where<NB>::CHB + chl;
    live = dl < p.in.Dg;
    d = w.g * p.in.Dg + (live ? dl : 0);
  }
};

// Four tokens' values of one lane, in registers.
template <int S, bool DO, bool CC>
struct Four {
  float delta[4], u[4], go[4];
  typename States<S>::type B[4], C[4];
  template <int CHB, int NP>
  __device__ __forceinline__ void load(const float* pd, const float* pu, const float* po, const float* pB, const float* pC) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      delta[j] = pd[j * CHB];
      u[j] = pu[j * CHB];
      if (DO) go[j] = po[j * CHB];
      B[j] = load_states<S>(pB + j * NP);
      if (CC) C[j] = load_states<S>(pC + j * NP);
    }
  }
};

// First walk: states in front of the tiles, and with SEG the segments' ends.  Bt 8,
// L 2048, D 2048, N 16 bf16, uncut: 113-121 us, the vector ALUs 70% busy: 256 blocks
// are one per compute unit there, two waves per SIMD.
template <typename T, int NB, int S, Words WD, bool SEG>
__global__ __launch_bounds__(2 * kThreads) void states_kernel(BwP p) {
  constexpr int TT = 32, CHB = CH / NB, VE = TT * CHB / kThreads, NP = 4 * S * NB;
  __shared__ __align__(16) float dl[2][TT][CHB];
  __shared__ __align__(16) float us[2][TT][CHB];
  __shared__ __align__(16) float ds[SEG ? 2 : 1][SEG ? TT : 1][CHB];
  __shared__ __align__(16) float bc[2][SEG ? 2 : 1][TT][NP];
  const int tid = threadIdx.x % kThreads;
  const Where<NB> w(p);
  const int tiles = w.tend > w.tbeg ? (w.tend - w.tbeg + TT - 1) / TT : 0;

  if (threadIdx.x < kThreads) {
    const Lane<NB, S> l(p, w, tid);
    float A2[S], h[S], P[S], gs[S], sum_delta = 0.f;
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const bool on = l.live && k < l.nleft;
      A2[k] = on ? rate(p.A[int64_t(l.d) * p.in.N + l.n0 + k]) : 0.f;
      h[k] = on && p.h0 != nullptr && w.seg == 0 ? p.h0[(int64_t(w.b) * p.in.D + l.d) * p.in.N + l.n0 + k] : 0.f;
      P[k] = 1.f;
      gs[k] = 0.f;
    }
    __syncthreads();
    for (int t = 0; t < tiles; ++t) {
      const int left = w.tend - w.tbeg - t * TT, o = t & 1;
      const float* pd = &dl[o][0][l.chl];
      const float* pu = &us[o][0][l.chl];
      const float* po = &ds[SEG ? o : 0][0][l.chl];
      const float* pB = &bc[o][0][0][l.n0];
      const float* pC = &bc[o][SEG ? 1 : 0][0][l.n0];
      auto keep = [&](int tq) {
        const int64_t at = int64_t((w.tbeg + t * TT + tq) / TB) * w.blocks + w.unit;
        store_pack<float, S>(p.ck + (at * kThreads + tid) * S, h);
        if (SEG && l.s == 0 && l.n0 == 0) p.cd[at * CHB + l.chl] = sum_delta;
      };
      auto four = [&](const Four<S, SEG, SEG>& q) {
        float a[4][S], u[4][S];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < S; ++k) {
            a[j][k] = decay(q.delta[j], A2[k]);
            u[j][k] = q.u[j] * q.B[j][k];
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
#pragma unroll
          for (int k = 0; k < S; ++k) {
            h[k] = fmaf(a[j][k], h[k], u[j][k]);
            if constexpr (SEG) {
              P[k] *= a[j][k];
              gs[k] = fmaf(P[k], q.C[j][k] * q.go[j], gs[k]);
            }
          }
          if (SEG) sum_delta += q.delta[j];
        }
      };
      // the next four tokens on their way from LDS meanwhile
      Four<S, SEG, SEG> q0, q1;
      q0.template load<CHB, NP>(pd, pu, po, pB, pC);
#pragma unroll
      for (int tq = 0; tq < TT; tq += 8) {
        if (tq >= left) break;
        if (tq % TB == 0) keep(tq);
        q1.template load<CHB, NP>(pd + (tq + 4) * CHB, pu + (tq + 4) * CHB, po + (tq + 4) * CHB, pB + (tq + 4) * NP, pC + (tq + 4) * NP);
        four(q0);
        const int tn = tq + 8 < TT ? tq + 8 : tq;
        q0.template load<CHB, NP>(pd + tn * CHB, pu + tn * CHB, po + tn * CHB, pB + tn * NP, pC + tn * NP);
        four(q1);
      }
      __syncthreads();
    }
    if (!SEG || !l.live) return;
    const int64_t at = (int64_t(w.seg) * p.Bt + w.b) * p.in.D + l.d;
#pragma unroll
    for (int k = 0; k < S; ++k)
      if (k < l.nleft) {
        p.hend[at * p.in.N + l.n0 + k] = h[k];
        p.gsum[at * p.in.N + l.n0 + k] = gs[k];
      }
    if (l.s == 0 && l.n0 == 0) p.sdel[at] = sum_delta;
    return;
  }

  Stager<T, TT, CHB, NP, WD, SEG, SEG, SEG> st;
  st.init(p.in, w.b, w.g, w.cb, tid, w.tend);
  float bias[VE];
#pragma unroll
  for (int v = 0; v < VE; ++v) bias[v] = p.in.dtb != nullptr && v < st.ncol ? p.in.dtb[w.g * p.in.Dg + st.cin + v] : 0.f;
  auto stage = [&](int t0, int o) {
    float de[VE], u[VE], go[VE];
    st.values(st.qd, de);
    st.values(st.qx, u);
    if (p.softplus) {
#pragma unroll
      for (int v = 0; v < VE; ++v) de[v] = softplus_fast(de[v] + bias[v]);
    }
#pragma unroll
    for (int v = 0; v < VE; ++v) u[v] *= de[v];
    if constexpr (SEG) {
      float zv[VE];
      st.values(st.qy, go);
      st.values(st.qz, zv);
      if (st.gated) {
#pragma unroll
        for (int v = 0; v < VE; ++v) go[v] *= silu_f(zv[v]);
      }
    }
    if (st.edge(t0)) {
#pragma unroll
      for (int v = 0; v < VE; ++v) {
        const bool on = st.inside(t0, v);
        de[v] = on ? de[v] : 0.f;
        u[v] = on ? u[v] : 0.f;
        if (SEG) go[v] = on ? go[v] : 0.f;
      }
    }
    store_pack<float, VE>(&dl[o][st.r][st.c0], de);
    store_pack<float, VE>(&us[o][st.r][st.c0], u);
    if constexpr (SEG) store_pack<float, VE>(&ds[o][st.r][st.c0], go);
    st.put_bc(t0, &bc[o][0][0][0]);
  };
  if (tiles > 0) {
    st.fetch(w.tbeg);
    stage(w.tbeg, 0);
    st.fetch(w.tbeg + TT);
  }
  __syncthreads();
  for (int i = 0; i < tiles; ++i) {
    if (i + 1 < tiles) {
      stage(w.tbeg + (i + 1) * TT, (i + 1) & 1);
      st.fetch(w.tbeg + (i + 2) * TT);
    }
    __syncthreads();
  }
}

// m ? a : b for an all-ones or all-zeros m, in one instruction: the truth table
// of (m & a) | (~m & b).  (A ternary of sums becomes a branch around them.)
__device__ __forceinline__ float pick(uint32_t m, float a, float b) {
  return __uint_as_float(__builtin_amdgcn_bitop3_b32(m, __float_as_uint(a), __float_as_uint(b), 0xCA));
}
// Sum of v[0..3] over the 16 channels of a row of lanes: lane c of the row ends
// with the sum of v[c & 3].  odd, two: all ones where c & 1, c & 2.
__device__ __forceinline__ float channels_sum(const float* v, uint32_t odd, uint32_t two) {
  const float a = pick(odd, v[1], v[0]) + dpp<0xB1, 0xF, true>(pick(odd, v[0], v[1]));
  const float b = pick(odd, v[3], v[2]) + dpp<0xB1, 0xF, true>(pick(odd, v[2], v[3]));
  float t = pick(two, b, a) + dpp<0x4E, 0xF, true>(pick(two, a, b));
  t += dpp<0x124, 0xF, true>(t);  // rotated by 4 within 16
  t += dpp<0x128, 0xF, true>(t);  // by 8
  return t;
}

// LDS of the reverse walk.  Between two barriers, while the scanning waves walk tile i,
// the staging waves finish tile i - 1 and stage tile i + 1, each at its own pace.  So what
// one of them stages has to lie apart from what another may still read, and with two
// halves, i & 1, nothing of tile i - 1 that was staged may be read any more:
//
//                  tile i - 1         tile i                   tile i + 1
//   dl, us, ds     -                  read by the scan         written
//   bc             -                  read by the scan,        written
//                                     B taken for the finish
//   sdu            -                  taken for the finish     written
//   o, gB, gA, wp  read by the finish written by the scan      -
template <int NB, int S>
struct Shared {
  static constexpr int CHB = CH / NB, NP = 4 * S * NB;
  float dl[2][TB][CHB], us[2][TB][CHB], ds[2][TB][CHB];  // delta, u, do
  float bc[2][2][TB][NP];
  float o[2][NB][TB][CHB], gB[2][NB][TB][CHB], gA[2][NB][TB][CHB];  // sums over a block's states
  float wp[2][4 / NB][TB][2][NP];                                   // dB, and dC without u B^T, of a wave's 16 channels
  float sdu[2][TB];                                                 // sum over the block's channels of do u
};

// Second walk.  Bound by vector issue (86% busy): 82 instructions per token and wave
// for the recurrences and sums, 22 of them the sums of dB and dC over channels, and
// about 16 for staging.  248 registers leave a compute unit one block.  Bt 8, L 2048,
// D 2048, N 16 bf16: 410-450 us.
template <typename T, int NB, int S, Words WD>
__global__ __launch_bounds__(2 * kThreads) void reverse_kernel(BwP p) {
  constexpr int CHB = CH / NB, VE = TB * CHB / kThreads, NP = 4 * S * NB;
  extern __shared__ __align__(16) unsigned char smem[];
  Shared<NB, S>& sh = *reinterpret_cast<Shared<NB, S>*>(smem);
  const int tid = threadIdx.x % kThreads;
  const Where<NB> w(p);
  const int tiles = w.tend > w.tbeg ? (w.tend - w.tbeg + TB - 1) / TB : 0;
  const int64_t ncols = int64_t(p.in.D) * (p.in.N + 2);
  float* part = p.part + (int64_t(w.seg) * p.Bt + w.b) * ncols;

  if (threadIdx.x < kThreads) {
    const Lane<NB, S> l(p, w, tid);
    const int wave = tid >> 6, blk = wave % NB;
    const int64_t at0 = int64_t(w.b) * p.in.D + l.d, per = int64_t(p.Bt) * p.in.D;
    const uint32_t odd = tid & 1 ? ~0u : 0u, two = tid & 2 ? ~0u : 0u, four = tid & 4 ? ~0u : 0u, eight = tid & 8 ? ~0u : 0u;
    const int rv = row_value(l.s);
    float A2[S], gg[S], hin[S], dA[S];
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const bool on = l.live && k < l.nleft;
      A2[k] = on ? rate(p.A[int64_t(l.d) * p.in.N + l.n0 + k]) : 0.f;
      gg[k] = on && p.dhf != nullptr ? p.dhf[at0 * p.in.N + l.n0 + k] : 0.f;
      hin[k] = 0.f;
      dA[k] = 0.f;
    }
    for (int q = 0; q < w.seg; ++q) {  // state in front of the segment
      const float sd = p.sdel[q * per + at0];
#pragma unroll
      for (int k = 0; k < S; ++k)
        hin[k] = fmaf(decay(sd, A2[k]), hin[k], k < l.nleft ? p.hend[(q * per + at0) * p.in.N + l.n0 + k] : 0.f);
    }
    for (int q = p.nseg - 1; q > w.seg; --q) {  // gradient behind it
      const float sd = p.sdel[q * per + at0];
#pragma unroll
      for (int k = 0; k < S; ++k)
        gg[k] = fmaf(decay(sd, A2[k]), gg[k], k < l.nleft ? p.gsum[(q * per + at0) * p.in.N + l.n0 + k] : 0.f);
    }
    Pack<float, S> qh{};
    float qcd = 0.f;
    auto fetch = [&](int tile) {
      const int64_t at = int64_t(w.tbeg / TB + (tile > 0 ? tile : 0)) * w.blocks + w.unit;
      qh = load_pack<float, S>(p.ck + (at * kThreads + tid) * S);
      if (w.seg > 0) qcd = p.cd[at * CHB + l.chl];
    };
    if (tiles > 0) fetch(tiles - 1);
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
      const int o = i & 1;
      float h[S];
#pragma unroll
      for (int k = 0; k < S; ++k) h[k] = w.seg > 0 ? fmaf(decay(qcd, A2[k]), hin[k], qh.e[k]) : qh.e[k];
      fetch(tiles - 2 - i);
      const float* pd = &sh.dl[o][0][l.chl];
      const float* pu = &sh.us[o][0][l.chl];
      const float* po = &sh.ds[o][0][l.chl];
      const float* pB = &sh.bc[o][0][0][l.n0];
      const float* pC = &sh.bc[o][1][0][l.n0];
      // ---- decays and states of the tile, forward
      float a[TB][S], ah[TB][S];
      Four<S, true, true> q[2];
      q[0].template load<CHB, NP>(pd, pu, po, pB, pC);
#pragma unroll
      for (int tq = 0; tq < TB; tq += 4) {
        const Four<S, true, true>& f = q[tq / 4 & 1];
        if (tq + 4 < TB)
          q[tq / 4 + 1 & 1].template load<CHB, NP>(pd + (tq + 4) * CHB, pu + (tq + 4) * CHB, po + (tq + 4) * CHB, pB + (tq + 4) * NP,
                                                   pC + (tq + 4) * NP);
        float y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < S; ++k) a[tq + j][k] = decay(f.delta[j], A2[k]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[j] = 0.f;
#pragma unroll
          for (int k = 0; k < S; ++k) {
            ah[tq + j][k] = a[tq + j][k] * h[k];
            h[k] = fmaf(f.u[j], f.B[j][k], ah[tq + j][k]);
            y[j] = fmaf(f.C[j][k], h[k], y[j]);
          }
        }
        sh.o[o][blk][tq + rv][l.chl] = rows_sum4(y);
      }
      // ---- gradients, backward; the last four tokens' values are at hand
      float dAt[S] = {};
#pragma unroll
      for (int tq = TB - 4; tq >= 0; tq -= 4) {
        const Four<S, true, true>& f = q[tq / 4 & 1];
        if (tq > 0)
          q[tq / 4 + 1 & 1].template load<CHB, NP>(pd + (tq - 4) * CHB, pu + (tq - 4) * CHB, po + (tq - 4) * CHB, pB + (tq - 4) * NP,
                                                   pC + (tq - 4) * NP);
        // the four tokens' S values each, four of them to a sum over the channels
        float sB[4], sA[4], gu[4 * S], dh[4 * S], rB[S], rC[S];
#pragma unroll
        for (int j = 3; j >= 0; --j) {
          sB[j] = sA[j] = 0.f;
#pragma unroll
          for (int k = 0; k < S; ++k) {
            const float gk = fmaf(f.C[j][k], f.go[j], gg[k]);
            dh[j * S + k] = f.go[j] * ah[tq + j][k];
            gu[j * S + k] = gk * f.u[j];
            sB[j] = fmaf(gk, f.B[j][k], sB[j]);
            const float m = gk * ah[tq + j][k];
            sA[j] = fmaf(m, A2[k], sA[j]);
            dAt[k] = fmaf(m, f.delta[j], dAt[k]);
            gg[k] = gk * a[tq + j][k];
          }
#pragma unroll
          for (int q = 0; q < S; ++q) {
            if (4 * q / S != j) continue;  // the four that this token completes
            rB[q] = channels_sum(gu + 4 * q, odd, two);
            rC[q] = channels_sum(dh + 4 * q, odd, two);
          }
        }
        sh.gB[o][blk][tq + rv][l.chl] = rows_sum4(sB);
        sh.gA[o][blk][tq + rv][l.chl] = rows_sum4(sA);
        // lane c of a row writes value c of its 4 S: token c / S, state c % S
        const int c = S == 3 ? ((tid & 15) < 12 ? tid & 15 : (tid & 15) - 4) : tid & (4 * S - 1);
        float* wp = &sh.wp[o][wave / NB][tq + c / S][0][l.n0 + c % S];
        if constexpr (S == 4) {
          wp[0] = pick(eight, pick(four, rB[3], rB[2]), pick(four, rB[1], rB[0]));
          wp[NP] = pick(eight, pick(four, rC[3], rC[2]), pick(four, rC[1], rC[0]));
        } else if constexpr (S == 3) {
          wp[0] = pick(eight, rB[2], pick(four, rB[1], rB[0]));
          wp[NP] = pick(eight, rC[2], pick(four, rC[1], rC[0]));
        } else if constexpr (S == 2) {
          wp[0] = pick(four, rB[1], rB[0]);
          wp[NP] = pick(four, rC[1], rC[0]);
        } else {
          wp[0] = rB[0];
          wp[NP] = rC[0];
        }
      }
#pragma unroll
      for (int k = 0; k < S; ++k) dA[k] += dAt[k];
      __syncthreads();
    }
    if (l.live) {
#pragma unroll
      for (int k = 0; k < S; ++k)
        if (k < l.nleft) {
          part[int64_t(l.d) * p.in.N + l.n0 + k] = dA[k];
          if (w.seg == 0 && p.dh0 != nullptr) p.dh0[at0 * p.in.N + l.n0 + k] = gg[k];
        }
    }
    __syncthreads();
    return;
  }

  // a tile that is partly past the end has its rows at its end: the last state, which may
  // be infinite, then meets the gradients of no row but its tokens'
  Stager<T, TB, CHB, NP, WD, true, true, true, true> st;
  st.init(p.in, w.b, w.g, w.cb, tid, w.tend);
  const int r = st.r, c0 = st.c0;
  const int64_t out0 = int64_t(w.b) * p.in.L * p.in.D + w.g * p.in.Dg;
  const uint32_t oo = uint32_t(r) * uint32_t(p.in.D) + st.cin;
  T* dxp = static_cast<T*>(p.dx) + out0;
  T* ddtp = static_cast<T*>(p.ddt) + out0;
  T* dzp = p.dz == nullptr ? nullptr : static_cast<T*>(p.dz) + out0;
  float bias[VE], dsk[VE], dD[VE], dbias[VE];
#pragma unroll
  for (int v = 0; v < VE; ++v) {
    const int dc = w.g * p.in.Dg + st.cin + v;
    bias[v] = p.in.dtb != nullptr && v < st.ncol ? p.in.dtb[dc] : 0.f;
    dsk[v] = p.in.Dsk != nullptr && v < st.ncol ? p.in.Dsk[dc] : 0.f;
    dD[v] = dbias[v] = 0.f;
  }
  // rows behind the item's length: zero gradients
  for (int t = (w.tend > w.tbeg ? w.tend : w.tbeg) + r; t < w.tlim; t += TB) {
    float zero[VE];
#pragma unroll
    for (int v = 0; v < VE; ++v) zero[v] = 0.f;
    const int64_t at = int64_t(t) * p.in.D + st.cin;
    store_cols<T, VE, WD>(dxp + at, zero, true, st.ncol);
    store_cols<T, VE, WD>(ddtp + at, zero, true, st.ncol);
    if (dzp != nullptr) store_cols<T, VE, WD>(dzp + at, zero, true, st.ncol);
  }
  // this thread's four of the tile's sums of dB and dC, those past the tile repeating it
  constexpr int kSums = TB * 2 * NP, NS = (kSums + 4 * kThreads - 1) / (4 * kThreads);
  float* bcp = p.bc + ((int64_t(w.cb) * p.Bt + w.b) * p.in.L * p.in.G + w.g) * (2 * NP);
  const int64_t bcrow = int64_t(p.in.G) * (2 * NP);
  // of the tile in each half: x, delta, sigmoid(dt), do, dy silu'(z)
  float kx[2][VE], kd[2][VE], ks[2][VE], kg[2][VE], kz[2][VE];
  auto stage = [&](int t0, auto half) {
    constexpr int o = decltype(half)::value;
    float u[VE], zv[VE];
    st.values(st.qx, kx[o]);
    st.values(st.qd, kd[o]);
    st.values(st.qy, kg[o]);
    st.values(st.qz, zv);
    if (p.softplus) {
#pragma unroll
      for (int v = 0; v < VE; ++v) kd[o][v] = softplus_sigmoid(kd[o][v] + bias[v], ks[o][v]);
    } else {
#pragma unroll
      for (int v = 0; v < VE; ++v) ks[o][v] = 1.f;
    }
    if (st.gated) {
#pragma unroll
      for (int v = 0; v < VE; ++v) {
        const float sg = sigmoid_f(zv[v]);
        kz[o][v] = kg[o][v] * dsilu_f(zv[v], sg);
        kg[o][v] *= zv[v] * sg;
      }
    } else {
#pragma unroll
      for (int v = 0; v < VE; ++v) kz[o][v] = 0.f;
    }
#pragma unroll
    for (int v = 0; v < VE; ++v) u[v] = kd[o][v] * kx[o][v];
    if (st.edge(t0)) {
#pragma unroll
      for (int v = 0; v < VE; ++v) {
        const bool on = st.inside(t0, v);
        kx[o][v] = on ? kx[o][v] : 0.f;
        kd[o][v] = on ? kd[o][v] : 0.f;
        ks[o][v] = on ? ks[o][v] : 0.f;
        kg[o][v] = on ? kg[o][v] : 0.f;
        u[v] = on ? u[v] : 0.f;
      }
    }
    store_pack<float, VE>(&sh.dl[o][r][c0], kd[o]);
    store_pack<float, VE>(&sh.us[o][r][c0], u);
    store_pack<float, VE>(&sh.ds[o][r][c0], kg[o]);
    st.put_bc(t0, &sh.bc[o][0][0][0]);
    // the row's sum of do u, over its 16 threads
    float du = 0.f;
#pragma unroll
    for (int v = 0; v < VE; ++v) du = fmaf(kg[o][v], u[v], du);
    du += dpp<0xB1, 0xF, true>(du);
    du += dpp<0x4E, 0xF, true>(du);
    du += dpp<0x141, 0xF, true>(du);
    du += dpp<0x140, 0xF, true>(du);
    if ((tid & 15) == 0) sh.sdu[o][r] = du;
  };
  float ox[VE], od[VE], oz[VE];
  f32x4 obc[NS];
  // of the tile walked, for its finish in the next step: B, and the sums of do u (0 at dB)
  f32x4 wB[NS];
  float wdu[NS];
  auto take = [&](auto half) {
    constexpr int o = decltype(half)::value;
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      const int e = 4 * ((tid + q * kThreads) % (kSums / 4)), t = e / (2 * NP), c = e % (2 * NP);
      wB[q] = *reinterpret_cast<const f32x4*>(&sh.bc[o][0][t][c % NP]);
      wdu[q] = c < NP ? 0.f : sh.sdu[o][t];
    }
  };
  auto finish = [&](auto half) {
    constexpr int o = decltype(half)::value;
    float y[VE], gB[VE], gA[VE];
#pragma unroll
    for (int v = 0; v < VE; ++v) y[v] = gB[v] = gA[v] = 0.f;
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const Pack<float, VE> q0 = load_pack<float, VE>(&sh.o[o][i][r][c0]), q1 = load_pack<float, VE>(&sh.gB[o][i][r][c0]),
                            q2 = load_pack<float, VE>(&sh.gA[o][i][r][c0]);
#pragma unroll
      for (int v = 0; v < VE; ++v) {
        y[v] += q0.e[v];
        gB[v] += q1.e[v];
        gA[v] += q2.e[v];
      }
    }
#pragma unroll
    for (int v = 0; v < VE; ++v) {
      ox[v] = fmaf(dsk[v], kg[o][v], kd[o][v] * gB[v]);
      od[v] = fmaf(kx[o][v], gB[v], gA[v] * kLn2) * ks[o][v];
      oz[v] = kz[o][v] * fmaf(dsk[v], kx[o][v], y[v]);
      dD[v] = fmaf(kg[o][v], kx[o][v], dD[v]);
      dbias[v] += od[v];
    }
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      const int e = 4 * ((tid + q * kThreads) % (kSums / 4)), c = e % (2 * NP);
      f32x4 v = *reinterpret_cast<const f32x4*>(&sh.wp[o][0][0][0][0] + e);
#pragma unroll
      for (int i = 1; i < 4 / NB; ++i) v += *reinterpret_cast<const f32x4*>(&sh.wp[o][i][0][0][0] + e);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = c < NP ? v[k] : fmaf(wdu[q], wB[q][k], v[k]);
      obc[q] = v;
    }
  };
  auto store = [&](int t0) {
    const int64_t first = t0 < w.tend - TB ? t0 : w.tend - TB;  // the token of row 0
    const bool row = st.token(t0, r);
    const int64_t at = first * p.in.D;
    store_cols<T, VE, WD>(dxp + at + oo, ox, row, st.ncol);
    store_cols<T, VE, WD>(ddtp + at + oo, od, row, st.ncol);
    if (dzp != nullptr) store_cols<T, VE, WD>(dzp + at + oo, oz, row, st.ncol);
    float* bt = bcp + first * bcrow;
#pragma unroll
    for (int q = 0; q < NS; ++q) {
      const int i = tid + q * kThreads, e = 4 * i, t = e / (2 * NP), c = e % (2 * NP);
      if (i < kSums / 4 && st.token(t0, t)) *reinterpret_cast<f32x4*>(bt + (t * bcrow + c)) = obc[q];
    }
  };
  const std::integral_constant<int, 0> even;
  const std::integral_constant<int, 1> odd;
  auto start = [&](int i) { return w.tbeg + (tiles - 1 - i) * TB; };  // first token of the tile of step i
  auto step = [&](int i, auto half, auto other) {
    if (i > 0) finish(other);
    take(half);
    if (i + 1 < tiles) {
      stage(start(i + 1), other);
      st.fetch(start(i + 2));
    }
    if (i > 0) store(start(i - 1));
    __syncthreads();
  };
  if (tiles > 0) {
    st.fetch(start(0));
    stage(start(0), even);
    st.fetch(start(1));
  }
  __syncthreads();
  for (int i = 0; i < tiles; i += 2) {
    step(i, even, odd);
    if (i + 1 < tiles) step(i + 1, odd, even);
  }
  if (tiles > 0) {
    if (tiles % 2) finish(even);
    else finish(odd);
    store(start(tiles - 1));
  }
  // ---- sums over the tokens: this thread's rows, then the 16 of each column
#pragma unroll
  for (int v = 0; v < VE; ++v) {
    sh.dl[0][r][c0 + v] = dD[v];
    sh.us[0][r][c0 + v] = dbias[v];
  }
  __syncthreads();
  if (tid < CHB && w.cb * CHB + tid < p.in.Dg) {
    float sd = 0.f, sb = 0.f;
#pragma unroll
    for (int q = 0; q < TB; ++q) {
      sd += sh.dl[0][q][tid];
      sb += sh.us[0][q][tid];
    }
    const int dd = w.g * p.in.Dg + w.cb * CHB + tid;
    part[int64_t(p.in.D) * p.in.N + dd] = sd;
    part[int64_t(p.in.D) * (p.in.N + 1) + dd] = sb;
  }
}

// The call's sums over blocks.  The first `sums` blocks: dA, dD and ddt_bias, over the
// items and segments.  The rest: dB and dC, over the blocks of channels, rounded once;
// zeros behind the lengths.  (In two launches: 2 us more, of 36 for 54 tokens.)
template <typename T, int NP, int COLS>
__global__ __launch_bounds__(1024) void sums_kernel(ColSum c, uint32_t sums, const float* bc, T* dB, T* dC, const int32_t* lengths,
                                                    int64_t rows, int L, int G, int N, int nblk) {
  __shared__ float red[1024];
  if (blockIdx.x < sums) {
    colsum_block<COLS>(c, blockIdx.x, red);
    return;
  }
  const int64_t i = int64_t(blockIdx.x - sums) * 1024 + threadIdx.x;
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
  int NB, nblk, nseg, seglen;
  int64_t tiles, blocks, sums, all;  // the last two: blocks of the joins, of dA, dD and ddt_bias and in all
  size_t oCk, oCd, oHe, oGs, oSd, oBc, oPart, bytes;
};
// Segments of the token axis.  The reverse walk's registers leave a compute unit
// one block, so n segments take ceil(blocks n / 256) / n turns of the uncut time,
// and about 15% more for the segments' ends: the fewest that take least (L 4096,
// D 2048, N 16 bf16 with 384 blocks: 1795 us cut in two, 2026 us not; with 32
// blocks and 16384 tokens 653 us cut in eight, 722 us in 32).  Where the items'
// lengths differ, four blocks per unit (5 items of 0 to 1537 tokens: 280 us, 430
// us with one).  64 tokens to a segment at least.
Plan plan_of(const m3_scan_args& f) {
  Plan p;
  p.NB = state_blocks(f.N);
  const int CHB = CH / p.NB, S = lane_states(f.N), NP = 4 * S * p.NB;
  p.nblk = blocks_per_group(f.D / f.G, p.NB);
  p.blocks = int64_t(f.Bt) * f.G * p.nblk;
  p.nseg = 1;
  p.seglen = (f.L + 31) / 32 * 32;
  const int64_t most = f.L / 64 < 32 ? f.L / 64 : 32;
  int64_t best = 1;
  if (f.lengths != nullptr) {
    best = (1024 + p.blocks - 1) / p.blocks;
    if (best > most) best = most;
  } else {
    double least = double((p.blocks + 255) / 256);
    for (int64_t n = 2; n <= most; ++n) {
      const double turns = 1.15 * double((p.blocks * n + 255) / 256) / double(n);
      if (turns < least - 1e-9) least = turns, best = n;
    }
  }
  if (best > 1) {
    p.seglen = int(((f.L + best - 1) / best + 31) / 32 * 32);
    p.nseg = (f.L + p.seglen - 1) / p.seglen;
  }
  p.tiles = (f.L + TB - 1) / TB;
  p.sums = colsum_blocks(int64_t(p.nseg) * f.Bt, int64_t(f.D) * (f.N + 2));
  p.all = p.sums + (int64_t(f.Bt) * f.L * f.G * 2 * NP + 1023) / 1024;
  const size_t seg = p.nseg > 1 ? size_t(p.nseg) * f.Bt * f.D : 0;
  p.oCk = 0;
  p.oCd = round256(p.oCk + size_t(p.tiles) * p.blocks * kThreads * 4 * S);
  p.oHe = round256(p.oCd + (p.nseg > 1 ? size_t(p.tiles) * p.blocks * CHB * 4 : 0));
  p.oGs = round256(p.oHe + seg * f.N * 4);
  p.oSd = round256(p.oGs + seg * f.N * 4);
  p.oBc = round256(p.oSd + seg * 4);
  p.oPart = round256(p.oBc + size_t(p.nblk) * f.Bt * f.L * f.G * 2 * NP * 4);
  p.bytes = round256(p.oPart + size_t(p.nseg) * f.Bt * f.D * (f.N + 2) * 4);
  return p;
}

template <typename T, int NB, int S, Words WD>
hipError_t run(const m3_scan_backward_args& a, const Plan& pl, hipStream_t st) {
  constexpr int NP = 4 * S * NB;
  static std::atomic<uint64_t> cleared{0};
  const m3_scan_args& f = a.fwd;
  unsigned char* ws = static_cast<unsigned char*>(a.workspace);
  auto at = [&](size_t o) { return reinterpret_cast<float*>(ws + o); };
  const Inputs in{f.x, f.dt, f.z, f.B, f.C, a.dy, f.x_ld, f.dt_ld, f.z_ld, f.B_ld, f.C_ld, f.D_skip, f.dt_bias, f.L, f.D, f.N, f.G,
                  f.D / f.G};
  const BwP p{in, f.A, f.h0, a.dh_final, f.lengths, a.dx, a.ddt, a.dz, a.dh0, at(pl.oCk), at(pl.oCd), at(pl.oHe), at(pl.oGs),
              at(pl.oSd), at(pl.oBc), at(pl.oPart), f.Bt, pl.nblk, pl.nseg, pl.seglen, f.dt_softplus};
  const uint32_t grid = uint32_t(pl.blocks * pl.nseg);
  if (pl.nseg > 1) states_kernel<T, NB, S, WD, true><<<grid, 2 * kThreads, 0, st>>>(p);
  else states_kernel<T, NB, S, WD, false><<<grid, 2 * kThreads, 0, st>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  e = allow_lds(reinterpret_cast<const void*>(&reverse_kernel<T, NB, S, WD>), sizeof(Shared<NB, S>), cleared);
  if (e != hipSuccess) return e;
  reverse_kernel<T, NB, S, WD><<<grid, 2 * kThreads, sizeof(Shared<NB, S>), st>>>(p);
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
  auto* go = colsum_cols(c.P) == 16 ? sums_kernel<T, NP, 16> : sums_kernel<T, NP, 128>;
  go<<<uint32_t(pl.all), 1024, 0, st>>>(c, uint32_t(pl.sums), p.bc, static_cast<T*>(a.dB), static_cast<T*>(a.dC), f.lengths,
                                        int64_t(f.Bt) * f.L, f.L, f.G, f.N, pl.nblk);
  return hipGetLastError();
}

template <typename T, Words WD>
hipError_t by_states(const m3_scan_backward_args& a, const Plan& p, hipStream_t st) {
#define CALL(NB, S) run<T, NB, S, WD>(a, p, st)
  M3_SCAN_STATES(a.fwd.N, CALL)
#undef CALL
}
template <typename T>
hipError_t by_words(const m3_scan_backward_args& a, const Plan& p, Words w, hipStream_t st) {
  if (w == kAligned) return by_states<T, kAligned>(a, p, st);
  return w == kLoose ? by_states<T, kLoose>(a, p, st) : by_states<T, kSingle>(a, p, st);
}

}  // namespace
}  // namespace scan

size_t scan_backward_workspace(const m3_scan_backward_args& a) {
  const scan::Plan p = scan::plan_of(a.fwd);
  return launchable(p.blocks * p.nseg, 2 * scan::kThreads) && launchable(p.all, 1024) ? p.bytes : 0;
}
hipError_t launch_scan_backward(const m3_scan_backward_args& a, hipStream_t s) {
  const m3_scan_args& f = a.fwd;
  const bool bf = f.in_dtype == M3_BF16;
  const size_t e = bf ? 2 : 4;
  const scan::Plan p = scan::plan_of(f);
  // four channels, and four values of B or C, as whole words
  const bool aligned = (f.D / f.G) % 4 == 0 && f.N % 4 == 0 && rows_aligned(f.x, f.x_ld, e, 4 * e) &&
                   rows_aligned(f.dt, f.dt_ld, e, 4 * e) && rows_aligned(f.z, f.z_ld, e, 4 * e) && rows_aligned(a.dy, f.D, e, 4 * e) &&
                   rows_aligned(a.dx, f.D, e, 4 * e) && rows_aligned(a.ddt, f.D, e, 4 * e) && rows_aligned(a.dz, f.D, e, 4 * e) &&
                   rows_aligned(f.B, f.B_ld, e, 4 * e) && rows_aligned(f.C, f.C_ld, e, 4 * e);
  const scan::Words w = scan::words_of(f.D / f.G, f.N, aligned);
  return bf ? scan::by_words<bf16_t>(a, p, w, s) : scan::by_words<float>(a, p, w, s);
}

}  // namespace m3
