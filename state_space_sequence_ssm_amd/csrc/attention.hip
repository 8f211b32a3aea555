// Linear attention with a decay per head: plans of its walks, the joins of segments and of
// shared heads, and the step of single tokens.
#include "mixer_internal.hpp"

namespace m3 {
namespace {

// ---------------------------------------------------------------- plans
int blocks32(int k) { return k <= 32 ? 1 : k <= 64 ? 2 : k <= 128 ? 4 : 8; }
struct Shape {
  int kb, nct;
};
int64_t units(const m3_linear_attention_args& a) { return int64_t(a.Bt) * a.H; }
// Columns of c per block: 64 where eight waves share a block (bf16, a and b of up to 128), and
// otherwise 128 where such a state fits the registers and blocks of them fill the card (fp32,
// Bt 16, L 1024, 32 heads of 128 x 128: 503 us, by 64 columns 650; of 64 x 128: 310 and 296).
bool two_roles(const m3_linear_attention_args& a, int b_cols) { return a.in_dtype == M3_BF16 && b_cols <= 128; }
Shape walk_shape(const m3_linear_attention_args& a, int b_cols, int c_cols) {
  const bool wide = c_cols > 64 && b_cols <= 128 && units(a) >= 256 && !two_roles(a, b_cols);
  return {blocks32(b_cols), wide ? 2 : 1};
}
// Of segments' own states: there are never 256 items' heads to cut.
Shape states_shape(int b_cols) { return {blocks32(b_cols), 1}; }
int tiles(int c_cols, Shape s) { return (c_cols + 64 * s.nct - 1) / (64 * s.nct); }
// blocks per segment of the forward, and of the backward's three walks
int64_t forward_blocks(const m3_linear_attention_args& a) { return units(a) * tiles(a.V, walk_shape(a, a.K, a.V)); }
int64_t backward_blocks(const m3_linear_attention_args& a) {
  return units(a) * (2 * tiles(a.K, walk_shape(a, a.V, a.K)) + tiles(a.V, walk_shape(a, a.K, a.V)));
}

// Segments of the token axis, at most one for each 256 tokens or part of them, in whole chunks
// (192 tokens at least, but for the last one): `want` blocks where there are fewer than 256.  One
// a compute unit of the forward's blocks of eight waves (16 heads of 128 x 128, bf16, one item of
// 4096 tokens: 58 us, with two 67, uncut 131; of 16384: 138, 143, 488), two of four waves (fp32,
// 4 x 4096 tokens of 16 heads of 64 x 64: 120 us, with one 137, uncut 342), and two for the
// backward's three walks (16384 tokens as above: 412 us, with one 489).
void segments(int64_t blocks, int most_blocks, int L, int& len, int& segs) {
  int64_t want = blocks >= 256 ? 1 : (most_blocks + blocks - 1) / blocks;
  const int64_t most = (L + 255) / 256;
  if (want > most) want = most;
  len = int(((L + want - 1) / want + 63) / 64 * 64);
  segs = (L + len - 1) / len;
}
struct Cut {
  int len, segs;
};
Cut uncut(int L) { return {(L + 63) / 64 * 64, 1}; }

size_t states_bytes(const m3_linear_attention_args& a, int segs) {
  return segs > 1 ? round256(size_t(a.Bt) * a.H * segs * a.K * a.V * 4) : 0;
}
Cut forward_cut(const m3_linear_attention_args& a) {
  Cut c;
  segments(forward_blocks(a), two_roles(a, a.K) ? 256 : 512, a.L, c.len, c.segs);
  return c;
}
Cut backward_cut(const m3_linear_attention_args& a) {
  Cut c;
  segments(backward_blocks(a), 512, a.L, c.len, c.segs);
  return c;
}

WalkSide side(const m3_linear_attention_args& a, const void* p, int64_t ld, int heads, int cols) {
  const size_t e = a.in_dtype == M3_BF16 ? 2 : 4;
  return {p, ld, heads, cols, rows_aligned(p, ld, e, 16) && (size_t(cols) * e) % 16 == 0};
}
WalkPlan plan_of(const m3_linear_attention_args& a, Cut c) {
  WalkPlan p{};
  p.Bt = a.Bt;
  p.L = a.L;
  p.H = a.H;
  p.seg_len = c.len;
  p.segs = c.segs;
  p.log_decay = a.log_decay;
  p.lengths = a.lengths;
  return p;
}
WalkJob job_of(const WalkSide& x, const WalkSide& b, const WalkSide& c, bool rev, int64_t sn, int64_t sv) {
  WalkJob j{};
  j.a = x;
  j.b = b;
  j.c = c;
  j.rev = rev;
  j.e = rev ? 0 : 1;
  j.s = j.u = j.w = 1.f;
  j.sn = sn;
  j.sv = sv;
  return j;
}
void to(WalkJob& j, void* out, bool f32, size_t elem) {
  j.out = out;
  j.out_f32 = f32;
  const uintptr_t at = reinterpret_cast<uintptr_t>(out);
  const int cols = j.c.cols, four = cols % 4 == 0 && at % (4 * (f32 ? 4 : elem)) == 0;
  j.out_words = four && (f32 || elem == 4 || (cols % 8 == 0 && at % 16 == 0)) ? 2 : four;
}
hipError_t run(const m3_linear_attention_args& a, WalkPlan& p, bool states, hipStream_t s) {
  const WalkJob& f = p.job[0];  // the others' states have its shape
  const Shape h = states ? states_shape(f.b.cols) : walk_shape(a, f.b.cols, f.c.cols);
  for (int i = 0; i < p.jobs; ++i) p.job[i].blocks = tiles(p.job[i].c.cols, h);
  return a.in_dtype == M3_BF16 ? launch_walk_bf16(p, h.kb, h.nct, states, s) : launch_walk_f32(p, h.kb, h.nct, states, s);
}

// ---------------------------------------------------------------- joins
// The states in front of every segment from the segments' own: E_0 = init,
// E_(s+1) = l^len E_s + own_s.
struct JoinSet {
  float* states;
  const float* init;
};
struct JoinP {
  JoinSet set[2];
  int sets, segs, len, L, H;
  int64_t per, units;
  const float* log_decay;
  const int32_t* lengths;
};
__global__ __launch_bounds__(256) void join_kernel(JoinP p, int blocks) {
  const int part = blockIdx.x % blocks;
  const int64_t id = blockIdx.x / blocks, unit = id % p.units;
  const JoinSet set = id / p.units ? p.set[1] : p.set[0];
  const int64_t i = int64_t(part) * 256 + threadIdx.x;
  if (i >= p.per) return;
  const int n = item_length(p.lengths, int(unit / p.H), p.L);
  const float g2 = p.log_decay[unit % p.H] * 1.4426950408889634f, whole = exp2f(g2 * float(p.len));
  float* at = set.states + unit * p.segs * p.per + i;
  float E = set.init == nullptr ? 0.f : set.init[unit * p.per + i];
  at[0] = E;
  const int held = n == 0 ? 1 : (n + p.len - 1) / p.len;
#pragma unroll 4
  for (int s = 1; s < held; ++s) {
    E = fmaf(whole, E, at[s * p.per]);
    at[s * p.per] = E;
  }
}
hipError_t join(const JoinP& p, hipStream_t s) {
  const int blocks = int((p.per + 255) / 256);
  join_kernel<<<dim3(uint32_t(blocks * p.units * p.sets)), dim3(256), 0, s>>>(p, blocks);
  return hipGetLastError();
}

// Gradients of shared heads: the sum over the heads of the walk that share one, in order.
struct ShareP {
  const float* part;  // [Bt, L, H, cols]
  void* out;          // [Bt, L, Hk, cols]
  const int32_t* lengths;
  int64_t total;  // Bt L Hk cols
  int L, Hk, per, cols;
};
template <typename T>
__global__ __launch_bounds__(256) void share_kernel(ShareP p) {
  for (int64_t i = int64_t(blockIdx.x) * 256 + threadIdx.x; i < p.total; i += int64_t(gridDim.x) * 256) {
    const int64_t row = i / p.cols, token = row / p.Hk;
    float s = 0.f;
    if (int(token % p.L) < item_length(p.lengths, int(token / p.L), p.L)) {
      const float* at = p.part + row * p.per * p.cols + i % p.cols;
      for (int k = 0; k < p.per; ++k) s += at[int64_t(k) * p.cols];
    }
    store_scalar<T>(static_cast<T*>(p.out) + i, s);
  }
}
hipError_t share(const m3_linear_attention_args& a, const float* part, void* out, int cols, hipStream_t s) {
  const int64_t total = int64_t(a.Bt) * a.L * a.Hk * cols;
  const ShareP p{part, out, a.lengths, total, a.L, a.Hk, a.H / a.Hk, cols};
  const dim3 grid(uint32_t(total < (1 << 24) ? (total + 255) / 256 : 1 << 16));
  if (a.in_dtype == M3_BF16) share_kernel<bf16_t><<<grid, dim3(256), 0, s>>>(p);
  else share_kernel<float><<<grid, dim3(256), 0, s>>>(p);
  return hipGetLastError();
}

// ---------------------------------------------------------------- single tokens
struct StepP {
  const void* q;
  const void* k;
  const void* v;
  int64_t q_ld, k_ld, v_ld;
  const float* log_decay;
  const float* h;
  float* h_out;
  void* y;
  int H, Hk, K, V, lgvl, tiles;
  float scale;
};
// l = exp(g) as a sum of two parts of its own sign.  Of slow decays (1 - l = 2^-12 for a memory
// of 4096 tokens) one float of l would hold 1 - l to 2^-13 of it only, the same way in every
// step; here hi + lo is off by a few 2^-24 of 1 - l.  A lo that is above 0 keeps l times infinity.
struct Decay {
  float hi, lo;
  __device__ __forceinline__ explicit Decay(float g) {
    if (fabsf(g) < 0.5f) {
      const float d = expm1f(g), one = 1.f + d;
      hi = one - 0x1p-23f;  // exact
      lo = (d - (one - 1.f)) + 0x1p-23f;
    } else {
      hi = lo = 0.5f * expf(g);
    }
  }
};
// S = l S + k v^T, y = scale q^T S.  One block per (sequence, head, tile of columns): 2^lgvl
// lanes along a row of the state, W columns each, the other groups of lanes on other rows.
// Bound by the state's way in and out: 256 sequences of 16 heads of 128 x 128, 107 us, 5.0 TB/s.
template <typename T, int W>
__global__ __launch_bounds__(256) void attention_step_kernel(StepP p) {
  __shared__ float sq[256], sk[256], red[256 * W];
  const int tile = blockIdx.x % p.tiles;
  const int64_t unit = blockIdx.x / p.tiles;
  const int h = int(unit % p.H), hk = h / (p.H / p.Hk);
  const int64_t item = unit / p.H;
  const T* q = static_cast<const T*>(p.q) + item * p.q_ld + int64_t(h) * p.K;
  const T* k = static_cast<const T*>(p.k) + item * p.k_ld + int64_t(hk) * p.K;
  const T* v = static_cast<const T*>(p.v) + item * p.v_ld + int64_t(hk) * p.V;
  if (int(threadIdx.x) < p.K) {
    sq[threadIdx.x] = load_scalar<T>(q + threadIdx.x) * p.scale;
    sk[threadIdx.x] = load_scalar<T>(k + threadIdx.x);
  }
  const int lanes = 1 << p.lgvl, groups = 256 >> p.lgvl;
  const int lane = threadIdx.x & (lanes - 1), group = threadIdx.x >> p.lgvl;
  const int c = (tile * lanes + lane) * W;
  const bool in = c < p.V;
  const Decay l(p.log_decay[h]);
  float vv[W], y[W];
#pragma unroll
  for (int i = 0; i < W; ++i) {
    vv[i] = in ? load_scalar<T>(v + c + i) : 0.f;
    y[i] = 0.f;
  }
  __syncthreads();
  if (in) {
    const float* from = p.h + unit * p.K * p.V + c;
    float* to = p.h_out + unit * p.K * p.V + c;
#pragma unroll 8
    for (int r = group; r < p.K; r += groups) {
      Pack<float, W> s = load_pack<float, W>(from + r * p.V);
      const float kr = sk[r], qr = sq[r];
#pragma unroll
      for (int i = 0; i < W; ++i) {
        s.e[i] = fmaf(l.hi, s.e[i], fmaf(kr, vv[i], l.lo * s.e[i]));
        y[i] = fmaf(qr, s.e[i], y[i]);
      }
      *reinterpret_cast<Pack<float, W>*>(to + r * p.V) = s;
    }
  }
#pragma unroll
  for (int i = 0; i < W; ++i) red[group * lanes * W + lane * W + i] = y[i];
  for (int n = groups / 2; n > 0; n /= 2) {
    __syncthreads();
    if (group < n)
#pragma unroll
      for (int i = 0; i < W; ++i) red[(group * lanes + lane) * W + i] += red[((group + n) * lanes + lane) * W + i];
  }
  if (group == 0 && in) {
    T* o = static_cast<T*>(p.y) + unit * p.V + c;
#pragma unroll
    for (int i = 0; i < W; ++i) store_scalar<T>(o + i, red[lane * W + i]);
  }
}
struct StepShape {
  int w, lgvl, tiles;
};
StepShape step_shape(const m3_linear_attention_step_args& a) {
  const uintptr_t at = reinterpret_cast<uintptr_t>(a.h) | reinterpret_cast<uintptr_t>(a.h_out);
  StepShape s{a.V % 4 == 0 && at % 16 == 0 ? 4 : 1, 0, 1};
  while (s.lgvl < 6 && (s.w << s.lgvl) < a.V) ++s.lgvl;
  s.tiles = (a.V + (s.w << s.lgvl) - 1) / (s.w << s.lgvl);
  return s;
}

}  // namespace

// ---------------------------------------------------------------- entry points
// The walks' launches; joins are of less than 256 items' heads, as only such are cut.
bool attention_fits(const m3_linear_attention_args& a) { return launchable(forward_blocks(a) * forward_cut(a).segs, 512); }
size_t attention_workspace(const m3_linear_attention_args& a) { return states_bytes(a, forward_cut(a).segs); }

hipError_t launch_attention(const m3_linear_attention_args& a, hipStream_t s) {
  const Cut c = a.workspace == nullptr ? uncut(a.L) : forward_cut(a);
  WalkPlan p = plan_of(a, c);
  WalkJob j = job_of(side(a, a.q, a.q_ld, a.H, a.K), side(a, a.k, a.k_ld, a.Hk, a.K), side(a, a.v, a.v_ld, a.Hk, a.V), false, a.V, 1);
  j.s = j.w = a.scale;
  j.init = a.h0;
  j.fin = a.h_final;
  j.states = static_cast<float*>(a.workspace);
  to(j, a.y, a.in_dtype == M3_F32, 2);
  p.job[0] = j;
  p.jobs = 1;
  if (c.segs > 1) {
    hipError_t e = run(a, p, true, s);
    if (e != hipSuccess) return e;
    e = join({{{j.states, a.h0}, {}}, 1, c.segs, c.len, a.L, a.H, int64_t(a.K) * a.V, int64_t(a.Bt) * a.H, a.log_decay, a.lengths}, s);
    if (e != hipSuccess) return e;
  }
  return run(a, p, false, s);
}

bool attention_step_fits(const m3_linear_attention_step_args& a) {
  return launchable(int64_t(a.Bt) * a.H * step_shape(a).tiles, 256);
}
hipError_t launch_attention_step(const m3_linear_attention_step_args& a, hipStream_t s) {
  const StepShape h = step_shape(a);
  const StepP p{a.q, a.k, a.v, a.q_ld, a.k_ld, a.v_ld, a.log_decay, a.h, a.h_out, a.y, a.H, a.Hk, a.K, a.V, h.lgvl, h.tiles, a.scale};
  const dim3 grid(uint32_t(int64_t(a.Bt) * a.H * h.tiles)), block(256);
  if (a.in_dtype == M3_BF16) {
    if (h.w == 4) attention_step_kernel<bf16_t, 4><<<grid, block, 0, s>>>(p);
    else attention_step_kernel<bf16_t, 1><<<grid, block, 0, s>>>(p);
  } else {
    if (h.w == 4) attention_step_kernel<float, 4><<<grid, block, 0, s>>>(p);
    else attention_step_kernel<float, 1><<<grid, block, 0, s>>>(p);
  }
  return hipGetLastError();
}

bool attention_backward_fits(const m3_linear_attention_backward_args& b) {
  return launchable(backward_blocks(b.fwd) * backward_cut(b.fwd).segs, 512);
}
// Workspace: the states in front of every segment, of the forward and of the reverse walk, and
// with shared heads every head's own dk and dv in fp32.
size_t attention_backward_workspace(const m3_linear_attention_backward_args& b) {
  const m3_linear_attention_args& a = b.fwd;
  const size_t rows = size_t(a.Bt) * a.L * a.H;
  return 2 * states_bytes(a, backward_cut(a).segs) + (a.Hk == a.H ? 0 : round256(rows * a.K * 4) + round256(rows * a.V * 4));
}

hipError_t launch_attention_backward(const m3_linear_attention_backward_args& b, hipStream_t s) {
  const m3_linear_attention_args& a = b.fwd;
  const Cut c = backward_cut(a);
  const size_t held = states_bytes(a, c.segs), rows = size_t(a.Bt) * a.L * a.H;
  char* ws = static_cast<char*>(b.workspace);
  float* fs = reinterpret_cast<float*>(ws);
  float* rs = reinterpret_cast<float*>(ws + held);
  const bool shared = a.Hk != a.H;
  void* dk = shared ? ws + 2 * held : b.dk;
  void* dv = shared ? ws + 2 * held + round256(rows * a.K * 4) : b.dv;
  const WalkSide q = side(a, a.q, a.q_ld, a.H, a.K), k = side(a, a.k, a.k_ld, a.Hk, a.K), v = side(a, a.v, a.v_ld, a.Hk, a.V),
                 dy = side(a, b.dy, int64_t(a.H) * a.V, a.H, a.V);
  const bool f32 = a.in_dtype == M3_F32;
  // dq = walk of (dy, v, k) over S^T; dk = reverse walk of (v, dy, q) over R^T; dv = of (k, q, dy) over R
  WalkJob jq = job_of(dy, v, k, false, 1, a.V), jk = job_of(v, dy, q, true, 1, a.V), jv = job_of(k, q, dy, true, a.V, 1);
  jq.s = jq.w = a.scale;
  jq.init = a.h0;
  jq.states = fs;
  to(jq, b.dq, f32, 2);
  jk.s = jk.u = jv.s = jv.u = a.scale;
  jk.init = jv.init = b.dh_final;
  jk.states = jv.states = rs;
  jv.fin = b.dh0;
  to(jk, dk, f32 || shared, 2);
  to(jv, dv, f32 || shared, 2);
  jq.zero_tail = a.lengths != nullptr;
  jk.zero_tail = jv.zero_tail = a.lengths != nullptr && !shared;
  hipError_t e;
  if (c.segs > 1) {
    WalkPlan p = plan_of(a, c);
    p.job[0] = job_of(q, k, v, false, a.V, 1);
    p.job[0].states = fs;
    p.job[1] = jv;
    p.jobs = 2;
    e = run(a, p, true, s);
    if (e != hipSuccess) return e;
    e = join({{{fs, a.h0}, {rs, b.dh_final}}, 2, c.segs, c.len, a.L, a.H, int64_t(a.K) * a.V, int64_t(a.Bt) * a.H, a.log_decay, a.lengths}, s);
    if (e != hipSuccess) return e;
  }
  WalkPlan p = plan_of(a, c);
  const Shape sk = walk_shape(a, a.V, a.K), sv = walk_shape(a, a.K, a.V);
  p.job[0] = jk;
  p.job[1] = jq;
  p.job[2] = jv;
  p.jobs = sk.kb == sv.kb && sk.nct == sv.nct ? 3 : 2;
  e = run(a, p, false, s);
  if (e != hipSuccess) return e;
  if (p.jobs == 2) {
    p.job[0] = jv;
    p.jobs = 1;
    e = run(a, p, false, s);
    if (e != hipSuccess) return e;
  }
  if (!shared) return hipSuccess;
  e = share(a, static_cast<const float*>(dk), b.dk, a.K, s);
  return e != hipSuccess ? e : share(a, static_cast<const float*>(dv), b.dv, a.V, s);
}

}  // namespace m3
