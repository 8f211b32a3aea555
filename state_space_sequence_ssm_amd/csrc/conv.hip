// Short causal depthwise convolution: prompts, single tokens and backward.
//
//   y[t,d] = act(bias[d] + sum_k w[d,k] x[t-(W-1)+k, d])
//
// Memory bound: 2 W + 4 operations per element against 2 elements moved.
#include "layer_internal.hpp"

namespace m3 {
namespace {

constexpr int kRows = 4;  // token rows loaded together by one thread

// First of word cv's channels.  Where words have the alignment of their elements only
// (RAG: widths or rows that are no multiple of one) the last is moved back to end with
// the row; the channels it shares with the word before come to the same values in both.
template <int V, bool RAG>
__device__ __forceinline__ int first_channel(uint32_t cv, int D) {
  const int d0 = int(cv) * V;
  return RAG && d0 + V > D ? D - V : d0;
}

struct ConvP {
  const void* x;
  int64_t ld;
  const float* w;
  const float* bias;
  const int32_t* lengths;
  const void* state;
  void* state_out;
  void* y;
  int L, D, tt;
  uint32_t nv, ntiles, total;
  int silu;
};

// One thread: V channels (one 16-byte word per row) down a tile of `tt`
// tokens, the last W - 1 inputs held in registers, so that a row is read once
// per tile and W - 1 rows again at its start.  Bt 8, L 4096, D 2048, W 4 bf16: 58 us,
// 4.6 TB/s where a plain copy reaches 5.15.
template <typename T, int W, int V, bool RAG>
__global__ __launch_bounds__(256) void conv_kernel(ConvP p) {
  const uint32_t idx = blockIdx.x * 256u + threadIdx.x;
  if (idx >= p.total) return;
  const uint32_t cv = idx % p.nv, r = idx / p.nv;
  const int tile = int(r % p.ntiles), b = int(r / p.ntiles);
  const int d0 = first_channel<V, RAG>(cv, p.D);
  const int len = item_length(p.lengths, b, p.L);
  const int t0 = tile * p.tt;
  const int t1 = t0 + p.tt < len ? t0 + p.tt : len;
  const T* x = static_cast<const T*>(p.x) + int64_t(b) * p.L * p.ld + d0;
  const T* state = static_cast<const T*>(p.state);
  if (state != nullptr) state += int64_t(b) * (W - 1) * p.D + d0;

  float xs[W - 1 + kRows][V];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    if (tile > 0 && t0 < len) {
      unpack<T, V>(load_word<T, V, RAG>(x + int64_t(t0 - (W - 1) + j) * p.ld), xs[j]);
    } else if (tile == 0 && state != nullptr) {
      unpack<T, V>(load_word<T, V, RAG>(state + int64_t(j) * p.D), xs[j]);
    } else {
#pragma unroll
      for (int i = 0; i < V; ++i) xs[j][i] = 0.f;
    }
  }
  if (tile == 0 && p.state_out != nullptr) {
    // inputs len - (W-1) .. len - 1; rows of `state` are read in ascending
    // order ahead of the row written, so the carry may be updated in place
    T* so = static_cast<T*>(p.state_out) + int64_t(b) * (W - 1) * p.D + d0;
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int t = len - (W - 1) + j;
      Pack<T, V> q{};
      if (t >= 0) q = load_word<T, V, RAG>(x + int64_t(t) * p.ld);
      else if (state != nullptr) q = load_word<T, V, RAG>(state + int64_t(len + j) * p.D);
      if constexpr (RAG) put_loose<T, V>(so + int64_t(j) * p.D, q);
      else *reinterpret_cast<Pack<T, V>*>(so + int64_t(j) * p.D) = q;
    }
  }
  if (t0 >= t1) return;

  float w[W][V], bias[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    bias[i] = p.bias != nullptr ? p.bias[d0 + i] : 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) w[k][i] = p.w[int64_t(d0 + i) * W + k];
  }
  T* y = static_cast<T*>(p.y) + int64_t(b) * p.L * p.D + d0;
  // kRows rows at a time, the next ones on their way meanwhile; rows past the
  // tile's end re-read its last row.  No branch around loads or stores but in the
  // last group: one would make each wait for a load wait for the stores too.
  Pack<T, V> q[kRows];
  auto fetch = [&](int t) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) q[i] = load_word<T, V, RAG>(x + int64_t(t + i < t1 ? t + i : t1 - 1) * p.ld);
  };
  auto rows = [&](int t, bool all) {
#pragma unroll
    for (int i = 0; i < kRows; ++i) unpack<T, V>(q[i], xs[W - 1 + i]);
    if (all) fetch(t + kRows);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
      float o[V];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float a = bias[v];
#pragma unroll
        for (int k = 0; k < W; ++k) a = fmaf(w[k][v], xs[i + k][v], a);
        o[v] = a;
      }
      if (p.silu) {
#pragma unroll
        for (int v = 0; v < V; ++v) o[v] = silu_f(o[v]);
      }
      if (all || t + i < t1) store_word<T, V, RAG>(y + int64_t(t + i) * p.D, o);
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int v = 0; v < V; ++v) xs[j][v] = xs[j + kRows][v];
  };
  fetch(t0);
  int t = t0;
  for (; t + kRows <= t1; t += kRows) rows(t, true);
  if (t < t1) rows(t, false);
}

struct ConvStepP {
  const void* x;
  int64_t ld;
  const float* w;
  const float* bias;
  const void* state;
  void* state_out;
  void* y;
  int D;
  uint32_t nv, total;
  int silu;
};

// One token: a thread holds V channels of one item, reads their W - 1 carried
// inputs and the new one, writes y and the carry moved up by one row.  Blocks of
// one wave, so that a single sequence spreads over compute units: 2.6 us.
template <typename T, int W, int V>
__global__ __launch_bounds__(64) void conv_step_kernel(ConvStepP p) {
  const uint32_t idx = blockIdx.x * 64u + threadIdx.x;
  if (idx >= p.total) return;
  const uint32_t cv = idx % p.nv, b = idx / p.nv;
  const int d0 = int(cv) * V;
  const T* st = static_cast<const T*>(p.state) + int64_t(b) * (W - 1) * p.D + d0;
  T* so = static_cast<T*>(p.state_out) + int64_t(b) * (W - 1) * p.D + d0;
  Pack<T, V> q[W];
#pragma unroll
  for (int j = 0; j < W - 1; ++j) q[j] = load_pack<T, V>(st + int64_t(j) * p.D);
  q[W - 1] = load_pack<T, V>(static_cast<const T*>(p.x) + int64_t(b) * p.ld + d0);
  float o[V];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    float a = p.bias != nullptr ? p.bias[d0 + v] : 0.f;
#pragma unroll
    for (int k = 0; k < W; ++k) a = fmaf(p.w[int64_t(d0 + v) * W + k], to_f32(q[k].e[v]), a);
    o[v] = p.silu ? silu_f(a) : a;
  }
  store_pack<T, V>(static_cast<T*>(p.y) + int64_t(b) * p.D + d0, o);
#pragma unroll
  for (int j = 0; j < W - 1; ++j) *reinterpret_cast<Pack<T, V>*>(so + int64_t(j) * p.D) = q[j + 1];
}

struct ConvBwP {
  const void* x;
  int64_t ld;
  const float* w;
  const float* bias;
  const int32_t* lengths;
  const void* state;
  const void* dy;
  void* dx;
  void* dstate;
  float* part;  // [Bt * ngroups][W + 1][D]
  int L, D, tt;
  uint32_t nv, ncb, ngroups;
  int lgcx;
  int silu;
};

// dpre[t] = dy[t] act'(pre[t]);  dx[t] = sum_j dpre[t+j] w[W-1-j];
// dw[k] = sum_t dpre[t] x[t-(W-1)+k];  dbias = sum_t dpre[t].
// One thread: V channels down `tt` tokens and the W - 1 after them, whose dpre
// its last dx need, four at a time with the next four on their way; a block is CX
// columns times 256 / CX tiles, whose sums of dw and dbias are joined in LDS
// before they go to the workspace.  Bt 8, L 4096, D 2048, W 4 bf16: 83 us, 4.8 TB/s,
// and 5 us for the join.
template <typename T, int W, int V, bool RAG>
__global__ __launch_bounds__(256) void conv_backward_kernel(ConvBwP p) {
  __shared__ float red[256 * (W + 1) * V];
  const int CX = 1 << p.lgcx, RY = 256 >> p.lgcx;
  const int col = threadIdx.x & (CX - 1), row = threadIdx.x >> p.lgcx;
  const uint32_t bi = blockIdx.x;
  const uint32_t cb = bi % p.ncb, rest = bi / p.ncb;
  const uint32_t grp = rest % p.ngroups, b = rest / p.ngroups;
  const uint32_t cv = (cb << p.lgcx) + col;
  const int t0 = (int(grp) * RY + row) * p.tt;
  const int len = item_length(p.lengths, int(b), p.L);
  const int d0 = first_channel<V, RAG>(cv, p.D);
  float dw[W + 1][V];
#pragma unroll
  for (int k = 0; k <= W; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) dw[k][v] = 0.f;
  const int tend = t0 + p.tt < p.L ? t0 + p.tt : p.L;  // dx rows [t0, tend)
  T* dx = static_cast<T*>(p.dx) + int64_t(b) * p.L * p.D + d0;
  T* dst = static_cast<T*>(p.dstate);
  if (dst != nullptr) dst += int64_t(b) * (W - 1) * p.D + d0;
  if (cv < p.nv && t0 < p.L && t0 >= len) {  // behind the item's tokens
    float zero[V];
#pragma unroll
    for (int v = 0; v < V; ++v) zero[v] = 0.f;
    for (int t = t0; t < tend; ++t) store_word<T, V, RAG>(dx + int64_t(t) * p.D, zero);
    for (int j = 0; j < W - 1; ++j)
      if (t0 == 0 && dst != nullptr) store_word<T, V, RAG>(dst + int64_t(j) * p.D, zero);
  } else if (cv < p.nv && t0 < p.L) {
    const T* x = static_cast<const T*>(p.x) + int64_t(b) * p.L * p.ld + d0;
    const T* dy = static_cast<const T*>(p.dy) + int64_t(b) * p.L * p.D + d0;
    const T* state = static_cast<const T*>(p.state);
    if (state != nullptr) state += int64_t(b) * (W - 1) * p.D + d0;
    float w[W][V], bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      bias[i] = p.bias != nullptr ? p.bias[d0 + i] : 0.f;
#pragma unroll
      for (int k = 0; k < W; ++k) w[k][i] = p.w[int64_t(d0 + i) * W + k];
    }
    const int tsum = tend < len ? tend : len;  // rows [t0, tsum) have a part in dw and dbias
    const int have = len - 1;                  // the last row with values
    // xs[j] = x[t - (W-1) + j], dp[j] = dpre[t - (W-1) + j]
    float xs[W - 1 + kRows][V], dp[W - 1 + kRows][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int t = t0 - (W - 1) + j;
#pragma unroll
      for (int v = 0; v < V; ++v) xs[j][v] = dp[j][v] = 0.f;
      if (t >= 0) {
        if (t < len) unpack<T, V>(load_word<T, V, RAG>(x + int64_t(t) * p.ld), xs[j]);
      } else if (state != nullptr) {
        unpack<T, V>(load_word<T, V, RAG>(state + int64_t(t + W - 1) * p.D), xs[j]);
      }
    }
    Pack<T, V> qx[kRows], qd[kRows];
    auto fetch = [&](int t) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int64_t at = t + i < have ? t + i : have;
        qx[i] = load_word<T, V, RAG>(x + at * p.ld);
        qd[i] = load_word<T, V, RAG>(dy + at * p.D);
      }
    };
    // rows t .. t + 3; inner: all of them hold values, and they and the dx they complete
    // lie in the tile.  A row behind the length has no part in anything: its zeros are put
    // in place after the activation, whose argument may hold inputs that are not finite.
    auto rows = [&](int t, bool inner) {
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        unpack<T, V>(qx[i], xs[W - 1 + i]);
        unpack<T, V>(qd[i], dp[W - 1 + i]);
      }
      fetch(t + kRows);
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        if (p.silu) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
            float a = bias[v];
#pragma unroll
            for (int k = 0; k < W; ++k) a = fmaf(w[k][v], xs[i + k][v], a);
            dp[W - 1 + i][v] *= dsilu_f(a, sigmoid_f(a));
          }
        }
        if (!inner) {
#pragma unroll
          for (int v = 0; v < V; ++v) dp[W - 1 + i][v] = t + i < len ? dp[W - 1 + i][v] : 0.f;
        }
        if (inner || t + i < tsum) {
#pragma unroll
          for (int v = 0; v < V; ++v) {
#pragma unroll
            for (int k = 0; k < W; ++k) dw[k][v] = fmaf(dp[W - 1 + i][v], xs[i + k][v], dw[k][v]);
            dw[W][v] += dp[W - 1 + i][v];
          }
        }
        float o[V];
#pragma unroll
        for (int v = 0; v < V; ++v) {
          o[v] = 0.f;
#pragma unroll
          for (int j = 0; j < W; ++j) o[v] = fmaf(dp[i + j][v], w[W - 1 - j][v], o[v]);
        }
        const int q = t + i - (W - 1);  // the dx row that is complete now
        if (inner) {
          store_word<T, V, RAG>(dx + int64_t(q) * p.D, o);
        } else if (q >= t0) {
          if (q < tend) store_word<T, V, RAG>(dx + int64_t(q) * p.D, o);
        } else if (q < 0 && dst != nullptr) {
          store_word<T, V, RAG>(dst + int64_t(q + W - 1) * p.D, o);
        }
      }
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int v = 0; v < V; ++v) {
          xs[j][v] = xs[j + kRows][v];
          dp[j][v] = dp[j + kRows][v];
        }
    };
    fetch(t0);
    rows(t0, false);
    int t = t0 + kRows;
    for (; t + kRows <= tsum; t += kRows) rows(t, true);
    for (; t < tend + W - 1; t += kRows) rows(t, false);
  }
#pragma unroll
  for (int k = 0; k <= W; ++k)
#pragma unroll
    for (int v = 0; v < V; ++v) red[((row * (W + 1) + k) * V + v) * CX + col] = dw[k][v];
  __syncthreads();
  float* part = p.part + (int64_t(b) * p.ngroups + grp) * (W + 1) * p.D;
  for (int i = threadIdx.x; i < (W + 1) * V * CX; i += 256) {
    const int c = i & (CX - 1), kv = i >> p.lgcx, k = kv / V, v = kv % V;
    const uint32_t cc = (cb << p.lgcx) + c;
    float s = 0.f;
    for (int r = 0; r < RY; ++r) s += red[((r * (W + 1) + k) * V + v) * CX + c];
    if (cc < p.nv) part[int64_t(k) * p.D + first_channel<V, RAG>(cc, p.D) + v] = s;
  }
}

template <int COLS>
__global__ __launch_bounds__(1024) void colsum_kernel(ColSum c) {
  __shared__ float red[1024];
  colsum_block<COLS>(c, blockIdx.x, red);
}

// Tokens per tile.  Long tiles read fewer rows twice (W - 1 of tt + W - 1) and
// write fewer partial sums, short ones give more threads: halved while the threads
// are fewer than a quarter of the card's lanes (256 CUs of 2048).  Bt 8, L 4096, D
// 2048 bf16: 58 us with 64 tokens, 64 us with 32; backward 89 us with 128, 103 us
// with 64 (measured with selections for padding in every row; 83 us without them).
int conv_tile(int64_t Bt, int L, int64_t nv, int most) {
  int tt = most;
  while (tt > 8 && Bt * ((L + tt - 1) / tt) * nv < 131072) tt /= 2;
  return tt;
}

template <typename T, int W, int V, bool RAG>
hipError_t run_conv(const m3_conv_args& a, hipStream_t s) {
  const int64_t nv = (a.D + V - 1) / V;
  ConvP p{a.x, a.x_ld, a.w, a.bias, a.lengths, a.state, a.state_out, a.y, a.L, a.D, 0, 0, 0, 0, a.silu};
  p.tt = conv_tile(a.Bt, a.L, nv, 64);
  p.nv = uint32_t(nv);
  p.ntiles = uint32_t((a.L + p.tt - 1) / p.tt);
  p.total = uint32_t(nv * p.ntiles * a.Bt);
  conv_kernel<T, W, V, RAG><<<(p.total + 255) / 256, 256, 0, s>>>(p);
  return hipGetLastError();
}
template <typename T, int W, int V>
hipError_t run_step(const m3_conv_step_args& a, hipStream_t s) {
  const int64_t nv = a.D / V;
  ConvStepP p{a.x, a.x_ld, a.w, a.bias, a.state, a.state_out, a.y, a.D, uint32_t(nv), uint32_t(nv * a.Bt), a.silu};
  conv_step_kernel<T, W, V><<<(p.total + 63) / 64, 64, 0, s>>>(p);
  return hipGetLastError();
}

struct BwGeom {
  int lgcx, tt;
  int64_t nv, ncb, ngroups;
};
BwGeom bw_geom(const m3_conv_backward_args& a, int V) {
  BwGeom g;
  g.nv = (a.D + V - 1) / V;
  g.lgcx = 3;
  while (g.lgcx < 6 && (int64_t(1) << g.lgcx) < g.nv) ++g.lgcx;
  g.ncb = (g.nv + (int64_t(1) << g.lgcx) - 1) >> g.lgcx;
  g.tt = conv_tile(a.Bt, a.L, g.nv, 128);
  const int64_t per = int64_t(g.tt) * (256 >> g.lgcx);
  g.ngroups = (a.L + per - 1) / per;
  return g;
}
template <typename T, int W, int V, bool RAG>
hipError_t run_bw(const m3_conv_backward_args& a, hipStream_t s) {
  const BwGeom g = bw_geom(a, V);
  ConvBwP p{a.x, a.x_ld, a.w, a.bias, a.lengths, a.state, a.dy, a.dx, a.dstate, static_cast<float*>(a.workspace),
            a.L, a.D, g.tt, uint32_t(g.nv), uint32_t(g.ncb), uint32_t(g.ngroups), g.lgcx, a.silu};
  conv_backward_kernel<T, W, V, RAG><<<uint32_t(g.ncb * g.ngroups * a.Bt), 256, 0, s>>>(p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  ColSum c{};
  c.part = p.part;
  c.P = g.ngroups * a.Bt;
  c.ncols = int64_t(W + 1) * a.D;
  c.dst[0] = a.dw;
  c.n[0] = int64_t(W) * a.D;
  c.dst[1] = a.dbias;
  c.n[1] = a.D;
  c.taps = W;
  c.D = a.D;
  return launch_colsum(c, s);
}

template <typename T, int V, bool RAG>
hipError_t by_taps(const m3_conv_args& a, hipStream_t s) {
  if (a.W == 2) return run_conv<T, 2, V, RAG>(a, s);
  return a.W == 3 ? run_conv<T, 3, V, RAG>(a, s) : run_conv<T, 4, V, RAG>(a, s);
}
template <typename T, int V>
hipError_t step_by_taps(const m3_conv_step_args& a, hipStream_t s) {
  if (a.W == 2) return run_step<T, 2, V>(a, s);
  return a.W == 3 ? run_step<T, 3, V>(a, s) : run_step<T, 4, V>(a, s);
}
template <typename T, int V, bool RAG>
hipError_t bw_by_taps(const m3_conv_backward_args& a, hipStream_t s) {
  if (a.W == 2) return run_bw<T, 2, V, RAG>(a, s);
  return a.W == 3 ? run_bw<T, 3, V, RAG>(a, s) : run_bw<T, 4, V, RAG>(a, s);
}

}  // namespace

hipError_t launch_colsum(const ColSum& c, hipStream_t s) {
  const uint32_t blocks = uint32_t(colsum_blocks(c.P, c.ncols));
  if (colsum_cols(c.P) == 16) colsum_kernel<16><<<blocks, 1024, 0, s>>>(c);
  else colsum_kernel<128><<<blocks, 1024, 0, s>>>(c);
  return hipGetLastError();
}

hipError_t launch_conv(const m3_conv_args& a, hipStream_t s) {
  const bool bf = a.in_dtype == M3_BF16;
  const size_t e = bf ? 2 : 4;
  if (rows_aligned(a.x, a.x_ld, e, 16) && rows_aligned(a.y, a.D, e, 16) && rows_aligned(a.state, a.D, e, 16) &&
      rows_aligned(a.state_out, a.D, e, 16))
    return bf ? by_taps<bf16_t, 8, false>(a, s) : by_taps<float, 4, false>(a, s);
  // a carry updated in place has room for one writer per channel; 16384 tokens of 2047
  // channels bf16 take 37 us in words, 47 us one at a time
  if (a.D >= (bf ? 8 : 4) && (a.state_out == nullptr || a.state_out != a.state))
    return bf ? by_taps<bf16_t, 8, true>(a, s) : by_taps<float, 4, true>(a, s);
  return bf ? by_taps<bf16_t, 1, false>(a, s) : by_taps<float, 1, false>(a, s);
}
hipError_t launch_conv_step(const m3_conv_step_args& a, hipStream_t s) {
  const bool bf = a.in_dtype == M3_BF16;
  const size_t e = bf ? 2 : 4;
  if (rows_aligned(a.x, a.x_ld, e, 16) && rows_aligned(a.y, a.D, e, 16) && rows_aligned(a.state, a.D, e, 16) &&
      rows_aligned(a.state_out, a.D, e, 16))
    return bf ? step_by_taps<bf16_t, 8>(a, s) : step_by_taps<float, 4>(a, s);
  return bf ? step_by_taps<bf16_t, 1>(a, s) : step_by_taps<float, 1>(a, s);
}
// Four channels per thread in the backward, whose windows of x and dpre are twice
// the forward's registers; 16384 tokens of 2047 channels bf16 take 53 us in words
// and 73 us one at a time.
size_t conv_backward_workspace(const m3_conv_backward_args& a) {
  const BwGeom g = bw_geom(a, a.D >= 4 ? 4 : 1);
  const int64_t P = g.ngroups * a.Bt, ncols = int64_t(a.W + 1) * a.D;
  return launchable(g.ncb * P, 256) && launchable(colsum_blocks(P, ncols), 1024) ? round256(size_t(P) * ncols * 4) : 0;
}
hipError_t launch_conv_backward(const m3_conv_backward_args& a, hipStream_t s) {
  const bool bf = a.in_dtype == M3_BF16;
  const size_t e = bf ? 2 : 4;
  if (rows_aligned(a.x, a.x_ld, e, 4 * e) && rows_aligned(a.dy, a.D, e, 4 * e) && rows_aligned(a.dx, a.D, e, 4 * e) &&
      rows_aligned(a.state, a.D, e, 4 * e) && rows_aligned(a.dstate, a.D, e, 4 * e))
    return bf ? bw_by_taps<bf16_t, 4, false>(a, s) : bw_by_taps<float, 4, false>(a, s);
  if (a.D >= 4) return bf ? bw_by_taps<bf16_t, 4, true>(a, s) : bw_by_taps<float, 4, true>(a, s);
  return bf ? bw_by_taps<bf16_t, 1, false>(a, s) : bw_by_taps<float, 1, false>(a, s);
}

}  // namespace m3
