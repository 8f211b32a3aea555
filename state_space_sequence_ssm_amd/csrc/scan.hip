// Selective scan over prompts and single tokens (see scan_common.hpp).
#include "scan_common.hpp"

namespace m3 {
namespace scan {
namespace {

struct ScanP {
  const void* x;
  const void* dt;
  const void* z;
  const void* B;
  const void* C;
  int64_t xld, dtld, zld, Bld, Cld;
  const float* A;
  const float* Dsk;
  const float* dtb;
  const float* h0;
  const int32_t* lengths;
  void* y;
  float* hfin;
  float* hend;  // [nseg - 1][Bt][D][N] states of the segments from zero (segment 0: from h0)
  float* sdel;  // [nseg - 1][Bt][D] sums of delta
  int Bt, L, D, N, G, Dg, nblk, nseg, seglen, softplus;
};

constexpr int tile(int S) { return S >= 4 ? 32 : 16; }  // tokens per tile

// Four tokens' values of one lane, in registers.
template <int K, bool FULL>
struct Four {
  float2 du[4];
  float B[4][K], C[4][K];
  template <int TT, int DS, int NP>
  __device__ __forceinline__ void load(int t, const float2 (&d)[TT][DS], const float (&bc)[2][TT][NP], int dcol, int s) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      du[i] = d[t + i][dcol];
#pragma unroll
      for (int k = 0; k < K; ++k) {
        B[i][k] = bc[0][t + i][s * K + k];
        if (FULL) C[i][k] = bc[1][t + i][s * K + k];
      }
    }
  }
};

// FULL: y and the last state, segment s starting from the join of the states
// before it.  Otherwise the states and sums of delta of the segments alone.
//
// A block is eight waves of two kinds, one of each per SIMD: four scan, 256 / S
// channels of S lanes; four stage, that is, they load the next tile, form delta
// and u and put them into the other half of LDS, and gate and store the tile
// before.  So the loads' latency and the exponentials of softplus and SiLU lie
// beside the recurrence and not between its tiles, with one barrier per tile.
template <typename T, int K, int S, bool VEC, bool FULL>
__global__ __launch_bounds__(2 * kThreads) void scan_kernel(ScanP p) {
  constexpr int CH = kThreads / S, TT = tile(S), VE = TT / S, NP = K * S;
  constexpr int NQ = (TT * NP / 2 + kThreads - 1) / kThreads;  // quads of B and C per thread
  constexpr int YS = CH + 64 / S;                              // the S rows written together lie on different banks
  constexpr int DS = CH + CH / 32 * 2;  // 16 bytes more every 32 channels: staging's words on different banks
  __shared__ __align__(16) float2 du[2][TT][DS];
  __shared__ __align__(16) float bc[2][2][TT][NP];
  __shared__ __align__(16) float ys[FULL ? 2 : 1][FULL ? TT : 1][YS];

  const int tid = threadIdx.x % kThreads;
  const bool scanner = threadIdx.x < kThreads;
  int blk = block_on_xcd();
  const int cb = blk % p.nblk;
  blk /= p.nblk;
  const int g = blk % p.G;
  blk /= p.G;
  const int b = blk % p.Bt, seg = blk / p.Bt;
  const int len = item_length(p.lengths, b, p.L);
  const int tbeg = seg * p.seglen;
  const int tend = tbeg + p.seglen < len ? tbeg + p.seglen : len;
  const int tiles = tend > tbeg ? (tend - tbeg + TT - 1) / TT : 0;

  if (scanner) {
    const int s = tid % S, chl = tid / S;
    const int dl = cb * CH + chl;
    const bool live = dl < p.Dg;
    const int d = g * p.Dg + (live ? dl : 0);
    const int dcol = chl + chl / 32 * 2;
    const uint32_t odd = s & 1 ? ~0u : 0u, two = s & 2 ? ~0u : 0u;
    float A2[K], h[K], sum_delta = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int n = s * K + k;
      const bool on = live && n < p.N;
      A2[k] = on ? p.A[int64_t(d) * p.N + n] * kLog2e : 0.f;
      h[k] = on && p.h0 != nullptr && (FULL || seg == 0) ? p.h0[(int64_t(b) * p.D + d) * p.N + n] : 0.f;
    }
    if constexpr (FULL) {
      for (int q = 0; q < seg; ++q) {
        const int64_t at = (int64_t(q) * p.Bt + b) * p.D + d;
        const float sd = p.sdel[at];
#pragma unroll
        for (int k = 0; k < K; ++k) {
          const int n = s * K + k;
          const float e = n < p.N ? p.hend[at * p.N + n] : 0.f;
          h[k] = q == 0 ? e : fmaf(decay(sd, A2[k]), h[k], e);
        }
      }
    }
    __syncthreads();
    for (int i = 0; i < tiles; ++i) {
      const int left = tend - tbeg - i * TT, o = i & 1;
      // four tokens at a time, the next four on their way from LDS meanwhile; two
      // register sets in turn.  Tokens past the end have delta = u = B = C = 0 and
      // leave the state alone.
      auto four = [&](int tq, const Four<K, FULL>& q) {
        float a[4][K], w[4][K], y[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int k = 0; k < K; ++k) {
            a[j][k] = decay(q.du[j].x, A2[k]);
            w[j][k] = q.du[j].y * q.B[j][k];
          }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          y[j] = 0.f;
#pragma unroll
          for (int k = 0; k < K; ++k) {
            h[k] = fmaf(a[j][k], h[k], w[j][k]);
            if (FULL) y[j] = fmaf(q.C[j][k], h[k], y[j]);
          }
          if (!FULL) sum_delta += q.du[j].x;
        }
        if constexpr (FULL) {
          float r0, r1;
          lanes_sum4<S>(y, odd, two, r0, r1);
          if constexpr (S >= 4) {
            if (s < 4) ys[o][tq + s][chl] = r0;
          } else {
            ys[o][tq + s][chl] = r0;
            ys[o][tq + 2 + s][chl] = r1;
          }
        }
      };
      const int nt = left < TT ? (left + 7) & ~7 : TT;
      Four<K, FULL> q0, q1;
      q0.load(0, du[o], bc[o], dcol, s);
      for (int tq = 0; tq < nt; tq += 8) {
        q1.load(tq + 4, du[o], bc[o], dcol, s);
        four(tq, q0);
        q0.load(tq + 8 < TT ? tq + 8 : 0, du[o], bc[o], dcol, s);
        four(tq + 4, q1);
      }
      __syncthreads();
    }
    if (!live) return;
    if constexpr (FULL) {
      if (p.hfin == nullptr || seg != p.nseg - 1) return;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (s * K + k < p.N) p.hfin[(int64_t(b) * p.D + d) * p.N + s * K + k] = h[k];
    } else {
      const int64_t at = (int64_t(seg) * p.Bt + b) * p.D + d;
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (s * K + k < p.N) p.hend[at * p.N + s * K + k] = h[k];
      if (s == 0) p.sdel[at] = sum_delta;
    }
    return;
  }

  // staging: token r of the tile, channels c0 ..
  const int r = tid / (CH / VE), c0 = (tid % (CH / VE)) * VE;
  const int ncol = p.Dg - (cb * CH + c0) < VE ? p.Dg - (cb * CH + c0) : VE;
  const int dc = g * p.Dg + cb * CH + c0;
  const int64_t row0 = int64_t(b) * p.L;
  const T* xp = static_cast<const T*>(p.x) + row0 * p.xld + dc;
  const T* dtp = static_cast<const T*>(p.dt) + row0 * p.dtld + dc;
  const T* zp = p.z == nullptr ? nullptr : static_cast<const T*>(p.z) + row0 * p.zld + dc;
  T* yp = FULL ? static_cast<T*>(p.y) + row0 * p.D + dc : nullptr;
  float bias[VE], dsk[VE];
#pragma unroll
  for (int v = 0; v < VE; ++v) {
    bias[v] = p.dtb != nullptr && v < ncol ? p.dtb[dc + v] : 0.f;
    dsk[v] = FULL && p.Dsk != nullptr && v < ncol ? p.Dsk[dc + v] : 0.f;
  }
  const bool bcvec = VEC && p.N % 4 == 0;

  Pack<T, VE> qx{}, qd{}, qz{};
  Pack<T, 4> qb[NQ];
  auto fetch = [&](int t0) {
    const int t = t0 + r;
    const bool row = t < tend;
    qx = load_cols<T, VE, VEC>(xp + int64_t(t) * p.xld, row, ncol);
    qd = load_cols<T, VE, VEC>(dtp + int64_t(t) * p.dtld, row, ncol);
    if (FULL && zp != nullptr) qz = load_cols<T, VE, VEC>(zp + int64_t(t) * p.zld, row, ncol);
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int e = tid + i * kThreads, q = e % (NP / 4), tt = (e / (NP / 4)) % TT, which = e / (NP / 4 * TT);
      qb[i] = Pack<T, 4>{};
      if (which < (FULL ? 2 : 1) && t0 + tt < tend && 4 * q < p.N) {
        const int64_t ld = which ? p.Cld : p.Bld;
        const T* src = static_cast<const T*>(which ? p.C : p.B) + (row0 + t0 + tt) * ld + int64_t(g) * p.N + 4 * q;
        qb[i] = bcvec ? load_pack<T, 4>(src) : load_some<T, 4>(src, p.N - 4 * q);
      }
    }
  };
  auto stage = [&](int t0, int o) {
#pragma unroll
    for (int v = 0; v < VE; ++v) {
      const float dl_ = step_of(to_f32(qd.e[v]), p.softplus != 0, bias[v], t0 + r < tend);
      du[o][r][c0 + c0 / 32 * 2 + v] = float2{dl_, dl_ * to_f32(qx.e[v])};
    }
#pragma unroll
    for (int i = 0; i < NQ; ++i) {
      const int e = tid + i * kThreads, q = e % (NP / 4), tt = (e / (NP / 4)) % TT, which = e / (NP / 4 * TT);
      if (which < 2) {
        float f[4];
        unpack<T, 4>(qb[i], f);
        *reinterpret_cast<f32x4*>(&bc[o][which][tt][4 * q]) = f32x4{f[0], f[1], f[2], f[3]};
      }
    }
  };
  auto finish = [&](int t0, int o, const Pack<T, VE>& x, const Pack<T, VE>& z) {
    float out[VE];
#pragma unroll
    for (int v = 0; v < VE; ++v) {
      out[v] = fmaf(dsk[v], to_f32(x.e[v]), ys[o][r][c0 + v]);
      if (zp != nullptr) out[v] *= silu_f(to_f32(z.e[v]));
    }
    store_cols<T, VE, VEC>(yp + int64_t(t0 + r) * p.D, out, t0 + r < tend, ncol);
  };
  // x and z of the tile staged last and of the one before it
  Pack<T, VE> x1{}, z1{}, x2{}, z2{};
  if (tiles > 0) {
    fetch(tbeg);
    stage(tbeg, 0);
    x1 = qx;
    z1 = qz;
    if (tiles > 1) fetch(tbeg + TT);
  }
  __syncthreads();
  for (int i = 0; i < tiles; ++i) {
    const int t0 = tbeg + i * TT;
    const Pack<T, VE> xo = x2, zo = z2;  // tile i - 1
    x2 = x1;
    z2 = z1;
    if (i + 1 < tiles) {
      stage(t0 + TT, (i + 1) & 1);
      x1 = qx;
      z1 = qz;
      if (i + 2 < tiles) fetch(t0 + 2 * TT);
    }
    if constexpr (FULL)
      if (i > 0) finish(t0 - TT, (i - 1) & 1, xo, zo);
    __syncthreads();
  }
  if constexpr (FULL)
    if (tiles > 0) finish(tbeg + (tiles - 1) * TT, (tiles - 1) & 1, x2, z2);
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
  int Bt, D, N, G, Dg, softplus, nb;
};

// One token: S lanes per (item, channel), 4 states each in one 16-byte word;
// the state is read and written once, everything else is small beside it.
template <typename T, int S, bool VEC>
__global__ __launch_bounds__(kThreads) void scan_step_kernel(StepP p) {
  const int s = threadIdx.x % S;
  const int64_t unit = (int64_t(blockIdx.x) * kThreads + threadIdx.x) / S;
  const int b = int(unit / p.D), d = int(unit - int64_t(b) * p.D);
  if (b >= p.Bt) return;
  const int g = d / p.Dg, n0 = 4 * s;
  const int64_t at = unit * p.N + n0;
  Pack<float, 4> h{}, A{};
  Pack<T, 4> B{}, C{};
  const T* Bp = static_cast<const T*>(p.B) + int64_t(b) * p.Bld + int64_t(g) * p.N + n0;
  const T* Cp = static_cast<const T*>(p.C) + int64_t(b) * p.Cld + int64_t(g) * p.N + n0;
  if (n0 < p.N) {
    if constexpr (VEC) {
      h = load_pack<float, 4>(p.h + at);
      A = load_pack<float, 4>(p.A + int64_t(d) * p.N + n0);
      B = load_pack<T, 4>(Bp);
      C = load_pack<T, 4>(Cp);
    } else {
      h = load_some<float, 4>(p.h + at, p.N - n0);
      A = load_some<float, 4>(p.A + int64_t(d) * p.N + n0, p.N - n0);
      B = load_some<T, 4>(Bp, p.N - n0);
      C = load_some<T, 4>(Cp, p.N - n0);
    }
  }
  const float x = to_f32(static_cast<const T*>(p.x)[int64_t(b) * p.xld + d]);
  const float raw = to_f32(static_cast<const T*>(p.dt)[int64_t(b) * p.dtld + d]);
  const float delta = step_of(raw, p.softplus != 0, p.dtb != nullptr ? p.dtb[d] : 0.f, true);
  const float u = delta * x;
  float o = 0.f, hn[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    hn[k] = fmaf(decay(delta, A.e[k] * kLog2e), h.e[k], u * to_f32(B.e[k]));
    o = fmaf(to_f32(C.e[k]), hn[k], o);
  }
  if (n0 < p.N) {
    if constexpr (VEC) store_pack<float, 4>(p.hout + at, hn);
    else store_some<float, 4>(p.hout + at, hn, p.N - n0);
  }
  o = lanes_sum<S>(o);
  if (s != 0) return;
  if (p.Dsk != nullptr) o = fmaf(p.Dsk[d], x, o);
  if (p.z != nullptr) o *= silu_f(to_f32(static_cast<const T*>(p.z)[int64_t(b) * p.zld + d]));
  from_f32(o, static_cast<T*>(p.y)[unit]);
}

struct Plan {
  int K, S, nblk, nseg, seglen;
};
// Segments of the token axis: with fewer blocks than two per compute unit the
// axis is cut, at least 128 tokens to a segment.
Plan plan_of(const m3_scan_args& a) {
  Plan p;
  p.K = 4;
  p.S = lanes_for(a.N);
#ifdef M3_K2
  if (a.N > 8 && a.N <= 16) p.K = 2, p.S = 8;
#endif
  p.nblk = blocks_per_group(a.D / a.G, p.S);
  p.nseg = 1;
  p.seglen = a.L;
  const int64_t blocks = int64_t(a.Bt) * a.G * p.nblk;
  if (blocks >= 256) return p;
  int64_t n = (512 + blocks - 1) / blocks;
  if (n > a.L / 128) n = a.L / 128;
  if (n < 2) return p;
  p.seglen = int(((a.L + n - 1) / n + 31) / 32 * 32);
  p.nseg = (a.L + p.seglen - 1) / p.seglen;
  return p;
}

template <typename T, int K, int S, bool VEC>
hipError_t run(const m3_scan_args& a, Plan pl, hipStream_t st) {
  if (a.workspace == nullptr) pl.nseg = 1, pl.seglen = a.L;
  ScanP p{a.x, a.dt, a.z, a.B, a.C, a.x_ld, a.dt_ld, a.z_ld, a.B_ld, a.C_ld, a.A, a.D_skip, a.dt_bias, a.h0, a.lengths, a.y,
          a.h_final, nullptr, nullptr, a.Bt, a.L, a.D, a.N, a.G, a.D / a.G, pl.nblk, pl.nseg, pl.seglen, a.dt_softplus};
  const int64_t per = int64_t(a.Bt) * a.G * pl.nblk;
  if (pl.nseg > 1) {
    p.hend = static_cast<float*>(a.workspace);
    p.sdel = p.hend + int64_t(pl.nseg - 1) * a.Bt * a.D * a.N;
    scan_kernel<T, K, S, VEC, false><<<uint32_t(per * (pl.nseg - 1)), 2 * kThreads, 0, st>>>(p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  scan_kernel<T, K, S, VEC, true><<<uint32_t(per * pl.nseg), 2 * kThreads, 0, st>>>(p);
  return hipGetLastError();
}
template <typename T, int S, bool VEC>
hipError_t run_step(const m3_scan_step_args& a, hipStream_t st) {
  const StepP p{a.x, a.dt, a.z, a.B, a.C, a.x_ld, a.dt_ld, a.z_ld, a.B_ld, a.C_ld, a.A, a.D_skip, a.dt_bias, a.h, a.h_out, a.y,
                a.Bt, a.D, a.N, a.G, a.D / a.G, a.dt_softplus, 1};
  const int64_t lanes = int64_t(a.Bt) * a.D * S;
  scan_step_kernel<T, S, VEC><<<uint32_t((lanes + kThreads - 1) / kThreads), kThreads, 0, st>>>(p);
  return hipGetLastError();
}

template <typename T, bool VEC>
hipError_t by_lanes(const m3_scan_args& a, const Plan& p, hipStream_t st) {
  switch (p.S) {
    case 2: return run<T, 4, 2, VEC>(a, p, st);
    case 4: return run<T, 4, 4, VEC>(a, p, st);
    case 8: return p.K == 2 ? run<T, 2, 8, VEC>(a, p, st) : run<T, 4, 8, VEC>(a, p, st);
    default: return run<T, 4, 16, VEC>(a, p, st);
  }
}
template <typename T, bool VEC>
hipError_t step_by_lanes(const m3_scan_step_args& a, hipStream_t st) {
  if (a.N <= 4) return run_step<T, 1, VEC>(a, st);
  switch (lanes_for(a.N)) {
    case 2: return run_step<T, 2, VEC>(a, st);
    case 4: return run_step<T, 4, VEC>(a, st);
    case 8: return run_step<T, 8, VEC>(a, st);
    default: return run_step<T, 16, VEC>(a, st);
  }
}

}  // namespace
}  // namespace scan

size_t scan_workspace(const m3_scan_args& a) {
  const scan::Plan p = scan::plan_of(a);
  return p.nseg < 2 ? 0 : round256(size_t(p.nseg - 1) * a.Bt * a.D * (a.N + 1) * 4);
}
hipError_t launch_scan(const m3_scan_args& a, hipStream_t s) {
  const bool bf = a.in_dtype == M3_BF16;
  const size_t e = bf ? 2 : 4;
  // a staging thread's channels, and four values of B or C, as whole words
  const scan::Plan p = scan::plan_of(a);
  const int ve = scan::tile(p.S) / p.S;
  const size_t word = e * ve < 16 ? e * ve : 16;
  const bool vec = (a.D / a.G) % ve == 0 && rows_aligned(a.x, a.x_ld, e, word) && rows_aligned(a.dt, a.dt_ld, e, word) &&
                   rows_aligned(a.z, a.z_ld, e, word) && rows_aligned(a.y, a.D, e, word) &&
                   (a.N % 4 != 0 || (rows_aligned(a.B, a.B_ld, e, 4 * e) && rows_aligned(a.C, a.C_ld, e, 4 * e)));
  if (bf) return vec ? scan::by_lanes<bf16_t, true>(a, p, s) : scan::by_lanes<bf16_t, false>(a, p, s);
  return vec ? scan::by_lanes<float, true>(a, p, s) : scan::by_lanes<float, false>(a, p, s);
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
