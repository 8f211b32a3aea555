// Selective scan over prompts and single tokens (see scan_common.hpp).
#include <type_traits>

#include "scan_common.hpp"

namespace m3 {
namespace scan {
namespace {

struct ScanP {
  Inputs in;
  const float* A;
  const float* h0;
  const int32_t* lengths;
  void* y;
  float* hfin;
  float* hend;  // [nseg - 1][Bt][D][N] states of the segments from zero (segment 0: from h0)
  float* sdel;  // [nseg - 1][Bt][D] sums of delta
  int Bt, nblk, nseg, seglen, softplus;
};

constexpr int TT = 32;  // tokens per tile

// Four tokens' values of one lane, in registers.
template <int S, bool FULL>
struct Four {
  float delta[4], u[4];
  typename States<S>::type B[4], C[4];
  // at this lane's channel of delta and u, and its states of B and C
  template <int CHB, int NP>
  __device__ __forceinline__ void load(const float* pd, const float* pu, const float* pB, const float* pC) {
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      delta[j] = pd[j * CHB];
      u[j] = pu[j * CHB];
      B[j] = load_states<S>(pB + j * NP);
      if (FULL) C[j] = load_states<S>(pC + j * NP);
    }
  }
};

// FULL: y and the last state, segment s starting from the join of the states
// before it.  Otherwise the states and sums of delta of the segments alone.
//
// A block is eight waves of two kinds, one of each per SIMD: four scan, 16
// channels and 4 S states each (64 / NB channels of NB state blocks); four stage,
// that is, they load the next tile, form delta and u and put them into the other
// half of LDS, and join, gate and store the y of the tile before.  So the loads'
// latency and the exponentials of softplus and SiLU lie beside the recurrence and
// not between its tiles, with one barrier per tile.  128 registers, so that a
// compute unit holds two blocks where there are as many.  Bt 8, L 4096, D 2048, N 16
// bf16, gated: 290-320 us with the clock, 29 vector instructions per token and wave
// and the vector ALUs 81-87% busy; the recurrence's own instructions take 164 us.
template <typename T, int NB, int S, Words WD, bool FULL>
__global__ __launch_bounds__(2 * kThreads, 4) void scan_kernel(ScanP p) {
  constexpr int CHB = CH / NB, VE = TT * CHB / kThreads, NP = 4 * S * NB;
  constexpr int YS = CHB == 16 ? 16 : CHB + 16;  // the four tokens' rows written together lie on different banks
  __shared__ __align__(16) float dl[2][TT][CHB];
  __shared__ __align__(16) float us[2][TT][CHB];
  __shared__ __align__(16) float bc[2][FULL ? 2 : 1][TT][NP];
  __shared__ __align__(16) float ys[FULL ? 2 : 1][FULL ? NB : 1][FULL ? TT + 1 : 1][YS];  // row TT takes what is not wanted

  const int tid = threadIdx.x % kThreads;
  const bool scanner = threadIdx.x < kThreads;
  int blk = block_on_xcd();
  const int cb = blk % p.nblk;
  blk /= p.nblk;
  const int g = blk % p.in.G;
  blk /= p.in.G;
  const int b = blk % p.Bt, seg = blk / p.Bt;
  const int len = item_length(p.lengths, b, p.in.L);
  const int tbeg = seg * p.seglen;
  const int tend = tbeg + p.seglen < len ? tbeg + p.seglen : len;
  const int tiles = tend > tbeg ? (tend - tbeg + TT - 1) / TT : 0;

  if (scanner) {
    const int wave = tid >> 6, s = (tid & 63) >> 4, chl = (wave / NB) * 16 + (tid & 15);
    const int sb = wave % NB, n0 = (sb * 4 + s) * S, nleft = p.in.N - n0;
    const int dloc = cb * CHB + chl;
    const bool live = dloc < p.in.Dg;
    const int d = g * p.in.Dg + (live ? dloc : 0);
    float A2[S], h[S], sum_delta = 0.f;
#pragma unroll
    for (int k = 0; k < S; ++k) {
      const bool on = live && k < nleft;
      A2[k] = on ? rate(p.A[int64_t(d) * p.in.N + n0 + k]) : 0.f;
      h[k] = on && p.h0 != nullptr && (FULL || seg == 0) ? p.h0[(int64_t(b) * p.in.D + d) * p.in.N + n0 + k] : 0.f;
    }
    if constexpr (FULL) {
      for (int q = 0; q < seg; ++q) {
        const int64_t at = (int64_t(q) * p.Bt + b) * p.in.D + d;
        const float sd = p.sdel[at];
#pragma unroll
        for (int k = 0; k < S; ++k) {
          const float e = k < nleft ? p.hend[at * p.in.N + n0 + k] : 0.f;
          h[k] = q == 0 ? e : fmaf(decay(sd, A2[k]), h[k], e);
        }
      }
    }
    __syncthreads();
    for (int t = 0; t < tiles; ++t) {
      const int left = tend - tbeg - t * TT, o = t & 1;
      const float* pd = &dl[o][0][chl];
      const float* pu = &us[o][0][chl];
      const float* pB = &bc[o][0][0][n0];
      const float* pC = &bc[o][FULL ? 1 : 0][0][n0];
      float* py = &ys[FULL ? o : 0][FULL ? sb : 0][0][chl];
      // Four tokens at a time, the next four on their way from LDS meanwhile; two
      // register sets in turn.  Tokens past the end have delta = u = B = C = 0 and
      // leave the state alone.  Decays and inputs of the four come ahead of their
      // recurrence: independent work that covers the exponentials' latency and that
      // of the sums over states of the four tokens before.
      float y[4] = {0.f, 0.f, 0.f, 0.f};
      auto four = [&](int to, const Four<S, FULL>& q) {
        float a[4][S], w[4][S];
        if constexpr (FULL) py[to * YS] = rows_sum4(y);
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < S; ++k) {
            a[j][k] = decay(q.delta[j], A2[k]);
            w[j][k] = q.u[j] * q.B[j][k];
          }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[j] = 0.f;
#pragma unroll
          for (int k = 0; k < S; ++k) {
            h[k] = fmaf(a[j][k], h[k], w[j][k]);
            if (FULL) y[j] = fmaf(q.C[j][k], h[k], y[j]);
          }
          if (!FULL) sum_delta += q.delta[j];
        }
        __builtin_amdgcn_sched_barrier(0);
      };
      const int nt = left < TT ? (left + 7) & ~7 : TT;
      const int rv = row_value(s);
      Four<S, FULL> q0, q1;
      q0.template load<CHB, NP>(pd, pu, pB, pC);
#pragma unroll
      for (int tq = 0; tq < TT; tq += 8) {
        if (tq >= nt) break;
        q1.template load<CHB, NP>(pd + (tq + 4) * CHB, pu + (tq + 4) * CHB, pB + (tq + 4) * NP, pC + (tq + 4) * NP);
        four(tq > 0 ? tq - 4 + rv : TT, q0);
        const int tn = tq + 8 < TT ? tq + 8 : tq;
        q0.template load<CHB, NP>(pd + tn * CHB, pu + tn * CHB, pB + tn * NP, pC + tn * NP);
        four(tq + rv, q1);
      }
      if constexpr (FULL) py[(nt - 4 + rv) * YS] = rows_sum4(y);
      __syncthreads();
    }
    if (!live) return;
    if constexpr (FULL) {
      if (p.hfin == nullptr || seg != p.nseg - 1) return;
#pragma unroll
      for (int k = 0; k < S; ++k)
        if (k < nleft) p.hfin[(int64_t(b) * p.in.D + d) * p.in.N + n0 + k] = h[k];
    } else {
      const int64_t at = (int64_t(seg) * p.Bt + b) * p.in.D + d;
#pragma unroll
      for (int k = 0; k < S; ++k)
        if (k < nleft) p.hend[at * p.in.N + n0 + k] = h[k];
      if (s == 0 && sb == 0) p.sdel[at] = sum_delta;
    }
    return;
  }

  Stager<T, TT, CHB, NP, WD, FULL, false, FULL> st;
  st.init(p.in, b, g, cb, tid, tend);
  const int r = st.r, c0 = st.c0;
  T* yp = FULL ? static_cast<T*>(p.y) + int64_t(b) * p.in.L * p.in.D + g * p.in.Dg : nullptr;
  float bias[VE], dsk[VE];
#pragma unroll
  for (int v = 0; v < VE; ++v) {
    const int dc = g * p.in.Dg + st.cin + v;
    bias[v] = p.in.dtb != nullptr && v < st.ncol ? p.in.dtb[dc] : 0.f;
    dsk[v] = FULL && p.in.Dsk != nullptr && v < st.ncol ? p.in.Dsk[dc] : 0.f;
  }
  // skip[o], gate[o]: D x and silu(z) of the tile in half o, for its y
  float skip[2][VE], gate[2][VE];
  auto stage = [&](int t0, auto half) {
    constexpr int o = decltype(half)::value;
    float de[VE], u[VE];
    st.values(st.qd, de);
    st.values(st.qx, u);
    if (p.softplus) {
#pragma unroll
      for (int v = 0; v < VE; ++v) de[v] = softplus_fast(de[v] + bias[v]);
    }
    if constexpr (FULL) {
      st.values(st.qz, gate[o]);
      if (st.gated) {
#pragma unroll
        for (int v = 0; v < VE; ++v) gate[o][v] = silu_f(gate[o][v]);
      } else {
#pragma unroll
        for (int v = 0; v < VE; ++v) gate[o][v] = 1.f;
      }
#pragma unroll
      for (int v = 0; v < VE; ++v) skip[o][v] = dsk[v] * u[v];
    }
#pragma unroll
    for (int v = 0; v < VE; ++v) u[v] *= de[v];
    if (st.edge(t0)) {  // tokens past the end and channels past the group
#pragma unroll
      for (int v = 0; v < VE; ++v) {
        const bool on = st.inside(t0, v);
        de[v] = on ? de[v] : 0.f;
        u[v] = on ? u[v] : 0.f;
      }
    }
    store_pack<float, VE>(&dl[o][r][c0], de);
    store_pack<float, VE>(&us[o][r][c0], u);
    st.put_bc(t0, &bc[o][0][0][0]);
  };
  float out[VE];
  auto finish = [&](auto half) {
    constexpr int o = decltype(half)::value;
    unpack<float, VE>(load_pack<float, VE>(&ys[o][0][r][c0]), out);
#pragma unroll
    for (int i = 1; i < NB; ++i) {
      const Pack<float, VE> q = load_pack<float, VE>(&ys[o][i][r][c0]);
#pragma unroll
      for (int v = 0; v < VE; ++v) out[v] += q.e[v];
    }
#pragma unroll
    for (int v = 0; v < VE; ++v) out[v] = (out[v] + skip[o][v]) * gate[o][v];
  };
  auto store = [&](int t0) { store_cols<T, VE, WD>(yp + int64_t(t0) * p.in.D + (uint32_t(r) * uint32_t(p.in.D) + st.cin), out, t0 + r < tend, st.ncol); };
  auto step = [&](int i, auto half, auto other) {
    const int t0 = tbeg + i * TT;
    if constexpr (FULL)
      if (i > 0) finish(other);
    if (i + 1 < tiles) {
      stage(t0 + TT, other);
      st.fetch(t0 + 2 * TT);
    }
    // last, so that no wait for the loads above waits for it as well
    if (FULL && i > 0) store(t0 - TT);
    __syncthreads();
  };
  const std::integral_constant<int, 0> even;
  const std::integral_constant<int, 1> odd;
  if (tiles > 0) {
    st.fetch(tbeg);
    stage(tbeg, even);
    st.fetch(tbeg + TT);
  }
  __syncthreads();
  for (int i = 0; i < tiles; i += 2) {
    step(i, even, odd);
    if (i + 1 < tiles) step(i + 1, odd, even);
  }
  if constexpr (FULL) {
    if (tiles == 0) return;
    if (tiles % 2) finish(even);
    else finish(odd);
    store(tbeg + (tiles - 1) * TT);
  }
}

struct StepP {
  const void* x;
  const void* dt;
  const void* z;
  const void* B;
  const void* C;
  int64_t xld, dtld, zld, Bld, Cld;
  const float* A;
  const float* Dsk;
  const float* dtb;
  const float* h;
  float* hout;
  void* y;
  int Bt, D, N, Dg, softplus, nblk;
};

// Sum over S neighbouring lanes, in each of them.
template <int S>
__device__ __forceinline__ float lanes_sum(float v) {
  if constexpr (S >= 2) v += dpp<0xB1, 0xF, true>(v);    // lane ^ 1
  if constexpr (S >= 4) v += dpp<0x4E, 0xF, true>(v);    // lane ^ 2
  if constexpr (S >= 8) v += dpp<0x141, 0xF, true>(v);   // mirrored within 8
  if constexpr (S >= 16) v += dpp<0x140, 0xF, true>(v);  // mirrored within 16
  return v;
}

// One token: S lanes per channel, 4 states each in one 16-byte word, for NI items
// whose loads are started together; the state is read and written once,
// everything else is small beside it.  256 items, D 2048, N 16: 13.4 us, 5.3 TB/s
// (16.6 us with one item per lane and 64-bit index arithmetic).
template <typename T, int S, int NI, bool VEC>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(StepP p) {
  const int s = threadIdx.x % S, n0 = 4 * s;
  const int d = (int(blockIdx.x % uint32_t(p.nblk)) * kThreads + int(threadIdx.x)) / S;
  const int b0 = int(blockIdx.x / uint32_t(p.nblk)) * NI;
  if (d >= p.D) return;
  const bool on = n0 < p.N;
  const int g = d / p.Dg, ns = on ? n0 : 0, left = p.N - n0;  // lanes without states read the first ones
  auto quad = [&](auto* q) {
    using E = std::remove_const_t<std::remove_pointer_t<decltype(q)>>;
    if constexpr (VEC) return load_pack<E, 4>(q);
    else return load_some<E, 4>(q, left);
  };
  const Pack<float, 4> A = quad(p.A + int64_t(d) * p.N + ns);
  Pack<float, 4> h[NI];
  Pack<T, 4> B[NI], C[NI];
  T x[NI], dt[NI], z[NI];
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int b = b0 + i < p.Bt ? b0 + i : p.Bt - 1;
    h[i] = quad(p.h + (int64_t(b) * p.D + d) * p.N + ns);
    B[i] = quad(static_cast<const T*>(p.B) + int64_t(b) * p.Bld + int64_t(g) * p.N + ns);
    C[i] = quad(static_cast<const T*>(p.C) + int64_t(b) * p.Cld + int64_t(g) * p.N + ns);
    x[i] = static_cast<const T*>(p.x)[int64_t(b) * p.xld + d];
    dt[i] = static_cast<const T*>(p.dt)[int64_t(b) * p.dtld + d];
    z[i] = p.z != nullptr ? static_cast<const T*>(p.z)[int64_t(b) * p.zld + d] : T{};
  }
  const float bias = p.dtb != nullptr ? p.dtb[d] : 0.f, dsk = p.Dsk != nullptr ? p.Dsk[d] : 0.f;
#pragma unroll
  for (int i = 0; i < NI; ++i) {
    const int b = b0 + i;
    const float xv = to_f32(x[i]);
    const float delta = p.softplus ? softplus_fast(to_f32(dt[i]) + bias) : to_f32(dt[i]);
    float o = 0.f, hn[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      hn[k] = fmaf(decay(delta, rate(A.e[k])), h[i].e[k], delta * xv * to_f32(B[i].e[k]));
      o = fmaf(to_f32(C[i].e[k]), hn[k], o);
    }
    o = lanes_sum<S>(on ? o : 0.f);
    if (b >= p.Bt) break;
    if (on) {
      float* ho = p.hout + (int64_t(b) * p.D + d) * p.N + n0;
      if constexpr (VEC) store_pack<float, 4>(ho, hn);
      else store_some<float, 4>(ho, hn, left);
    }
    if (s == 0) {
      o = fmaf(dsk, xv, o);
      if (p.z != nullptr) o *= silu_f(to_f32(z[i]));
      from_f32(o, static_cast<T*>(p.y)[int64_t(b) * p.D + d]);
    }
  }
}

struct Plan {
  int NB, nblk, nseg, seglen;
};
// Segments of the token axis.  A cut costs a second pass over nearly all tokens
// (states alone, two thirds of the work), so it pays where the blocks leave
// enough of the 256 compute units idle: L 4096, D 2048, N 16 bf16 with 128 blocks
// 230 us cut and 289 us not, with 192 blocks 371 us and 290 us.  Then two blocks
// per unit (1 item of 16384 tokens: 270 us, with four 290 us, with one 282 us),
// but four where the items' lengths differ and blocks behind them have nothing to
// do (5 items of 0 to 1537 tokens, 160 blocks: 85 us, with two 100 us, uncut 114
// us); 64 tokens to a segment
// at least (512 tokens: 24 us, with 128 29 us).  Few channels leave few blocks and many
// segments: one item of 1024 tokens of 64 channels takes 24 us cut and 73 us uncut, of
// 8192 tokens of 64, 128 and 256 channels 73, 74 and 132 us and 546 us, of 65536 tokens
// 471, 283 and 237 us and 4320 us.  The last segments' joins, which read the segments in
// front one after the other, weigh most there.
Plan plan_of(const m3_scan_args& a) {
  Plan p;
  p.NB = state_blocks(a.N);
  p.nblk = blocks_per_group(a.D / a.G, p.NB);
  p.nseg = 1;
  p.seglen = a.L;
  const int64_t blocks = int64_t(a.Bt) * a.G * p.nblk;
  if (blocks >= (a.lengths != nullptr ? 256 : 160)) return p;
  int64_t n = ((a.lengths != nullptr ? 1024 : 512) + blocks - 1) / blocks;
  if (n > a.L / 64) n = a.L / 64;
  if (n < 2) return p;
  p.seglen = int(((a.L + n - 1) / n + 31) / 32 * 32);
  p.nseg = (a.L + p.seglen - 1) / p.seglen;
  return p;
}

template <typename T, int NB, int S, Words WD>
hipError_t run(const m3_scan_args& a, Plan pl, hipStream_t st) {
  if (a.workspace == nullptr) pl.nseg = 1, pl.seglen = a.L;
  const Inputs in{a.x, a.dt, a.z, a.B, a.C, nullptr, a.x_ld, a.dt_ld, a.z_ld, a.B_ld, a.C_ld, a.D_skip, a.dt_bias, a.L, a.D, a.N,
                  a.G, a.D / a.G};
  ScanP p{in, a.A, a.h0, a.lengths, a.y, a.h_final, nullptr, nullptr, a.Bt, pl.nblk, pl.nseg, pl.seglen, a.dt_softplus};
  const int64_t per = int64_t(a.Bt) * a.G * pl.nblk;
  if (pl.nseg > 1) {
    p.hend = static_cast<float*>(a.workspace);
    p.sdel = p.hend + int64_t(pl.nseg - 1) * a.Bt * a.D * a.N;
    scan_kernel<T, NB, S, WD, false><<<uint32_t(per * (pl.nseg - 1)), 2 * kThreads, 0, st>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  scan_kernel<T, NB, S, WD, true><<<uint32_t(per * pl.nseg), 2 * kThreads, 0, st>>>(p);
  return hipGetLastError();
}
template <typename T, int S, int NI, bool VEC>
hipError_t run_step(const m3_scan_step_args& a, hipStream_t st) {
  const int64_t nblk = (int64_t(a.D) * S + kThreads - 1) / kThreads;
  const StepP p{a.x, a.dt, a.z, a.B, a.C, a.x_ld, a.dt_ld, a.z_ld, a.B_ld, a.C_ld, a.A, a.D_skip, a.dt_bias, a.h, a.h_out, a.y,
                a.Bt, a.D, a.N, a.D / a.G, a.dt_softplus, int(nblk)};
  scan_step_kernel<T, S, NI, VEC><<<uint32_t(nblk * ((int64_t(a.Bt) + NI - 1) / NI)), kThreads, 0, st>>>(p);
  return hipGetLastError();
}
// Several items per lane once the lanes would fill the card twice (256 CUs of 2048).
int items_of(const m3_scan_step_args& a, int S) { return int64_t(a.Bt) * a.D * S >= 1 << 20 ? 4 : 1; }
template <typename T, int S, bool VEC>
hipError_t step_items(const m3_scan_step_args& a, hipStream_t st) {
  return items_of(a, S) == 4 ? run_step<T, S, 4, VEC>(a, st) : run_step<T, S, 1, VEC>(a, st);
}

template <typename T, Words WD>
hipError_t by_states(const m3_scan_args& a, const Plan& p, hipStream_t st) {
#define CALL(NB, S) run<T, NB, S, WD>(a, p, st)
  M3_SCAN_STATES(a.N, CALL)
#undef CALL
}
template <typename T>
hipError_t by_words(const m3_scan_args& a, const Plan& p, Words w, hipStream_t st) {
  if (w == kAligned) return by_states<T, kAligned>(a, p, st);
  return w == kLoose ? by_states<T, kLoose>(a, p, st) : by_states<T, kSingle>(a, p, st);
}
int step_lanes(int N) { return N <= 4 ? 1 : N <= 8 ? 2 : N <= 16 ? 4 : N <= 32 ? 8 : 16; }
template <typename T, bool VEC>
hipError_t step_by_lanes(const m3_scan_step_args& a, hipStream_t st) {
  switch (step_lanes(a.N)) {
    case 1: return step_items<T, 1, VEC>(a, st);
    case 2: return step_items<T, 2, VEC>(a, st);
    case 4: return step_items<T, 4, VEC>(a, st);
    case 8: return step_items<T, 8, VEC>(a, st);
    default: return step_items<T, 16, VEC>(a, st);
  }
}

}  // namespace
}  // namespace scan

bool scan_fits(const m3_scan_args& a) {
  const scan::Plan p = scan::plan_of(a);
  return launchable(int64_t(a.Bt) * a.G * p.nblk * p.nseg, 2 * scan::kThreads);
}
size_t scan_workspace(const m3_scan_args& a) {
  const scan::Plan p = scan::plan_of(a);
  return p.nseg < 2 ? 0 : round256(size_t(p.nseg - 1) * a.Bt * a.D * (a.N + 1) * 4);
}
hipError_t launch_scan(const m3_scan_args& a, hipStream_t s) {
  const bool bf = a.in_dtype == M3_BF16;
  const size_t e = bf ? 2 : 4;
  const scan::Plan p = scan::plan_of(a);
  // four channels, and four values of B or C, as whole words
  const bool aligned = (a.D / a.G) % 4 == 0 && a.N % 4 == 0 && rows_aligned(a.x, a.x_ld, e, 4 * e) &&
                   rows_aligned(a.dt, a.dt_ld, e, 4 * e) && rows_aligned(a.z, a.z_ld, e, 4 * e) && rows_aligned(a.y, a.D, e, 4 * e) &&
                   rows_aligned(a.B, a.B_ld, e, 4 * e) && rows_aligned(a.C, a.C_ld, e, 4 * e);
  const scan::Words w = scan::words_of(a.D / a.G, a.N, aligned);
  return bf ? scan::by_words<bf16_t>(a, p, w, s) : scan::by_words<float>(a, p, w, s);
}
bool scan_step_fits(const m3_scan_step_args& a) {
  const int S = scan::step_lanes(a.N), NI = scan::items_of(a, S);
  return launchable((int64_t(a.D) * S + scan::kThreads - 1) / scan::kThreads * ((int64_t(a.Bt) + NI - 1) / NI), scan::kThreads);
}
hipError_t launch_scan_step(const m3_scan_step_args& a, hipStream_t s) {
  const bool bf = a.in_dtype == M3_BF16;
  const size_t e = bf ? 2 : 4;
  const bool vec = a.N % 4 == 0 && rows_aligned(a.h, a.N, 4, 16) && rows_aligned(a.h_out, a.N, 4, 16) &&
                   rows_aligned(a.A, a.N, 4, 16) && rows_aligned(a.B, a.B_ld, e, 4 * e) && rows_aligned(a.C, a.C_ld, e, 4 * e);
  if (bf) return vec ? scan::step_by_lanes<bf16_t, true>(a, s) : scan::step_by_lanes<bf16_t, false>(a, s);
  return vec ? scan::step_by_lanes<float, true>(a, s) : scan::step_by_lanes<float, false>(a, s);
}

}  // namespace m3
