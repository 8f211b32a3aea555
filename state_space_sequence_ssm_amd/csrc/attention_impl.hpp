// The chunked walk of linear attention (see mixer_internal.hpp for its formula) on the
// matrix cores: y, dq, dk and dv, and the states of segments.
#pragma once
#include <atomic>

#include "m3ssm_internal.hpp"
#include "mixer_internal.hpp"

namespace m3 {
namespace walk {

constexpr int kChunk = 64;

// ---------------------------------------------------------------- operands
// Both matrix products take their operands from registers: lane (g = lane / 16, l16)
// supplies row (column) l16 at 8 positions of the contracted axis, 4 g + 0..3 of one block
// of 16 and of the next.  That is also how a 16 x 16 accumulator lies (row 4 g + i, column
// l16), so that scores and states go from one product to the next without a detour.
template <typename T>
struct Op;
template <>
struct Op<bf16_t> {
  typedef uint16_t elem;
  typedef bf16x8 frag;
  typedef u32x2 half;  // 4 positions
  static constexpr int kWord = 8;
  // scores in 2, states read in 2 and their updates' weights in 3 bf16 parts: 16 and 24
  // bits, so that what a product adds to the outputs' own rounding (2^-9) and to the fp32
  // state is below either
  static constexpr int kScore = 2, kState = 2, kWeight = 3;
  template <int D>
  static __device__ __forceinline__ int at(int r, int c) {  // 8-byte units swizzled by row, as the core's prefill
    const int r0 = r & 1, r1 = (r >> 1) & 1, r2 = (r >> 2) & 1, r3 = (r >> 3) & 1;
    int x;
    if constexpr (D >= 128) x = ((r0 ^ r3) << 1) | (r1 << 2) | (r2 << 3) | (r0 << 4);
    else if constexpr (D == 64) x = ((r0 ^ r3) << 1) | (r1 << 2) | (r2 << 3);
    else x = ((r1 ^ r3) << 1) | (r2 << 2);
    return r * D + (((c >> 2) ^ x) << 2);
  }
  template <int D>
  static constexpr int size() { return kChunk * D * 2; }
  // row r, contracted positions of the block pair at column c
  template <int D>
  static __device__ __forceinline__ frag row(const elem* t, int r, int c, int g) {
    return cat8(*reinterpret_cast<const u32x2*>(t + at<D>(r, c + 4 * g)),
                *reinterpret_cast<const u32x2*>(t + at<D>(r, c + 16 + 4 * g)));
  }
  // column c + l16, contracted positions: rows of the block pair at row r
  template <int D>
  static __device__ __forceinline__ frag col(const elem* t, int r, int c, int lane) {
    const int rr = r + (lane >> 4) * 4 + ((lane & 15) >> 2), cc = c + (lane & 3) * 4;
    return cat8(lds_read_tr(t + at<D>(rr, cc)), lds_read_tr(t + at<D>(rr + 16, cc)));
  }
  static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c) { return m3::mma(a, b, c); }
  static __device__ __forceinline__ frag join(half lo, half hi) { return cat8(lo, hi); }
  static __device__ __forceinline__ void values(frag f, float (&v)[8]) {
    const u32x4 w = __builtin_bit_cast(u32x4, f);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  // v in N bf16 parts, each the rounding of what is left (not a number where v is not finite)
  template <int N>
  static __device__ __forceinline__ void split(f32x4 v, half (&o)[N]) {
#pragma unroll
    for (int k = 0; k < N; ++k) {
      o[k] = pack4(v);
      if (k + 1 < N) v -= unpack4(o[k]);
    }
  }
};
template <>
struct Op<float> {
  typedef float elem;
  struct frag {
    f32x4 lo, hi;
  };
  typedef f32x4 half;
  static constexpr int kWord = 4;
  static constexpr int kScore = 1, kState = 1, kWeight = 1;
  // rows 4 words apart from a multiple of 64 banks' worth: whole rows, columns and words
  // are read and written without conflicts
  template <int D>
  static __device__ __forceinline__ int at(int r, int c) { return r * (D + 4) + c; }
  template <int D>
  static constexpr int size() { return kChunk * (D + 4) * 4; }
  template <int D>
  static __device__ __forceinline__ frag row(const elem* t, int r, int c, int g) {
    return {*reinterpret_cast<const f32x4*>(t + at<D>(r, c + 4 * g)), *reinterpret_cast<const f32x4*>(t + at<D>(r, c + 16 + 4 * g))};
  }
  template <int D>
  static __device__ __forceinline__ frag col(const elem* t, int r, int c, int lane) {
    const elem* q = t + at<D>(r + (lane >> 4) * 4, c + (lane & 15));
    frag f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.lo[i] = q[at<D>(i, 0)];
      f.hi[i] = q[at<D>(16 + i, 0)];
    }
    return f;
  }
  static __device__ __forceinline__ f32x4 mma(frag a, frag b, f32x4 c) {
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.lo[i], b.lo[i], c, 0, 0, 0);
#pragma unroll
    for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a.hi[i], b.hi[i], c, 0, 0, 0);
    return c;
  }
  static __device__ __forceinline__ frag join(half lo, half hi) { return {lo, hi}; }
  static __device__ __forceinline__ void values(frag f, float (&v)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] = f.lo[i];
      v[4 + i] = f.hi[i];
    }
  }
  template <int N>
  static __device__ __forceinline__ void split(f32x4 v, half (&o)[N]) {
    static_assert(N == 1, "exact");
    o[0] = v;
  }
};

// l^d for whole d >= 0: 1 at 0 also where l = 0
__device__ __forceinline__ float power(float g2, int d) { return d == 0 ? 1.f : __builtin_amdgcn_exp2f(g2 * float(d)); }

// ---------------------------------------------------------------- one tile on its way
// 64 rows of D elements (columns past `cols` and rows past n zero) from the tokens of a
// chunk into LDS, 16-byte words over 256 threads.
template <typename T, int D>
struct Tile {
  static constexpr int W = Op<T>::kWord, kRow = D / W, N = kChunk * kRow / 256;
  static_assert(N >= 1, "a word per thread at least");
  u32x4 w[N];
  // base: head's elements of position 0 of the chunk; step: elements to the next position
  __device__ __forceinline__ void load(const T* base, int64_t step, int n, int cols, bool words) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * 256 + int(threadIdx.x), r = at / kRow, c = at % kRow * W;
      const bool in = r < n && c < cols;
      const T* p = base + (in ? r : 0) * step + (in ? c : 0);
      if (words) {
        w[i] = *reinterpret_cast<const u32x4*>(p);
      } else {
        const int left = in ? cols - c : 0;
        Pack<T, W> q;
        if (left >= W) q = load_loose<T, W>(p);
        else q = load_some<T, W>(p, left);
        __builtin_memcpy(&w[i], &q, 16);
      }
      if (!in) w[i] = u32x4{0, 0, 0, 0};
    }
  }
  __device__ __forceinline__ void store(typename Op<T>::elem* t) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int at = i * 256 + int(threadIdx.x), r = at / kRow, c = at % kRow * W;
      *reinterpret_cast<u32x4*>(t + Op<T>::template at<D>(r, c)) = w[i];
    }
  }
};

template <typename T>
__device__ __forceinline__ void put4(const WalkJob& j, T* out, int64_t at, f32x4 v, int n) {
  if (j.out_f32 || sizeof(T) == 4) {
    float* o = reinterpret_cast<float*>(out) + at;
    if (j.out_words && n >= 4) {
      *reinterpret_cast<f32x4*>(o) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) o[i] = v[i];
    }
  } else {
    T* o = out + at;
    if (j.out_words && n >= 4) {
      store4<T>(o, v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) store_scalar<T>(o + i, v[i]);
    }
  }
}

// One block of 4 waves walks one segment of one (item, head) for 64 NCT columns of c: wave w
// holds columns 16 NCT w.. of the state, all 32 KB rows of it, in accumulators.
//   A: tiles of a, b, c into LDS.  B: the triangle's 10 score tiles, dealt over the waves, weighted by
//   l^(p-j) and handed round through LDS; a E from the state.  C: scores times c, out, the state.
template <typename T, int KB, int NCT, bool STATES>
struct Lds {
  static constexpr int D = 32 * KB, V = 64 * NCT;
  static constexpr int a = 0, b = STATES ? 0 : Op<T>::template size<D>(), c = b + Op<T>::template size<D>(),
                       p = c + Op<T>::template size<V>(), end = p + (STATES ? 0 : 10 * Op<T>::kScore * 64 * int(sizeof(typename Op<T>::half)));
};

template <typename T, int KB, int NCT, bool STATES>
__global__ __launch_bounds__(256) void walk_kernel(WalkPlan plan) {
  typedef Op<T> O;
  typedef Lds<T, KB, NCT, STATES> M;
  typedef typename O::elem elem;
  constexpr int D = M::D, V = M::V, NS = O::kScore, NE = O::kState, NW = O::kWeight;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  elem* sa = reinterpret_cast<elem*>(lds + M::a);
  elem* sb = reinterpret_cast<elem*>(lds + M::b);
  elem* sc = reinterpret_cast<elem*>(lds + M::c);
  typename O::half* sp = reinterpret_cast<typename O::half*>(lds + M::p);

  // which job, item, head, segment and columns
  int64_t id = blockIdx.x;
  const int units = plan.Bt * plan.H, segs = STATES ? plan.segs - 1 : plan.segs;
  int ji = 0;
  while (ji + 1 < plan.jobs && id >= int64_t(plan.job[ji].blocks) * units * segs) {
    id -= int64_t(plan.job[ji].blocks) * units * segs;
    ++ji;
  }
  const WalkJob& j = plan.job[ji];
  const int vt = int(id % j.blocks), unit = int(id / j.blocks % units), seg = int(id / j.blocks / units);
  const int item = unit / plan.H, h = unit % plan.H;
  const int n = item_length(plan.lengths, item, plan.L);
  const int from = seg * plan.seg_len, to = min(n, from + plan.seg_len);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, g = lane >> 4, l16 = lane & 15;
  const int v0 = vt * V, vc = min(j.c.cols - v0, V);
  const float g2 = plan.log_decay[h] * 1.4426950408889634f;

  if constexpr (!STATES) {
    if (j.zero_tail) {  // rows behind the item's tokens
      const int first = max(n, from), last = min(plan.L, from + plan.seg_len);
      T* o = static_cast<T*>(j.out);
      for (int64_t i = threadIdx.x; i < int64_t(last - first) * vc; i += 256)
        o[((int64_t(item) * plan.L + first + i / vc) * plan.H + h) * j.c.cols + v0 + i % vc] = T{};
    }
  }
  const bool last_seg = from + plan.seg_len >= n;  // of this item
  if (STATES ? last_seg : (from >= n && seg > 0)) return;

  // the state: rows 16 r + 4 g + i, columns 16 (wave NCT + ct) + l16
  f32x4 E[2 * KB][NCT];
  const int64_t per = int64_t(j.b.cols) * j.c.cols;
  const float* init = nullptr;
  if constexpr (!STATES) init = plan.segs > 1 ? j.states + (int64_t(unit) * plan.segs + seg) * per : j.init == nullptr ? nullptr : j.init + unit * per;
#pragma unroll
  for (int r = 0; r < 2 * KB; ++r)
#pragma unroll
    for (int ct = 0; ct < NCT; ++ct) {
      const int v = 16 * (wave * NCT + ct) + l16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 16 * r + 4 * g + i;
        E[r][ct][i] = init != nullptr && row < j.b.cols && v < vc ? init[row * j.sn + (v0 + v) * j.sv] : 0.f;
      }
    }

  const int64_t first = j.rev ? int64_t(item) * plan.L + n - 1 : int64_t(item) * plan.L;
  const int dir = j.rev ? -1 : 1;
  auto rows = [&](const WalkSide& s, int p) {
    return static_cast<const T*>(s.p) + (first + int64_t(dir) * p) * s.ld + int64_t(h / (plan.H / s.heads)) * s.cols;
  };
  for (int p0 = from; p0 < to; p0 += kChunk) {
    const int nc = min(kChunk, to - p0);
    {
      Tile<T, D> t;
      if constexpr (!STATES) {
        t.load(rows(j.a, p0), dir * j.a.ld, nc, j.a.cols, j.a.words);
        t.store(sa);
      }
      t.load(rows(j.b, p0), dir * j.b.ld, nc, j.b.cols, j.b.words);
      t.store(sb);
      Tile<T, V> tc;
      tc.load(rows(j.c, p0) + v0, dir * j.c.ld, nc, vc, j.c.words);
      tc.store(sc);
    }
    __syncthreads();
    f32x4 acc[4][NCT];
    if constexpr (!STATES) {
      // scores transposed: rows j, columns p
#pragma unroll
      for (int k = 0; k < 3; ++k) {
        const int idx = wave + 4 * k;
        if (idx < 10) {
          const int tt = idx < 1 ? 0 : idx < 3 ? 1 : idx < 6 ? 2 : 3, jt = idx - tt * (tt + 1) / 2;
          f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int R = 0; R < KB; ++R)
            s = O::mma(O::template row<D>(sb, 16 * jt + l16, 32 * R, g), O::template row<D>(sa, 16 * tt + l16, 32 * R, g), s);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int d = 16 * (tt - jt) + l16 - 4 * g - i;
            s[i] = d < 0 ? 0.f : s[i] * (j.s * power(g2, d));
          }
          typename O::half o[NS];
          O::template split<NS>(s, o);
#pragma unroll
          for (int q = 0; q < NS; ++q) sp[(idx * NS + q) * 64 + lane] = o[q];
        }
      }
      // a E, transposed: rows v, columns p
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) acc[tt][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int R = 0; R < KB; ++R) {
        typename O::frag e[NCT][NE];
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) {
          typename O::half lo[NE], hi[NE];
          O::template split<NE>(E[2 * R][ct], lo);
          O::template split<NE>(E[2 * R + 1][ct], hi);
#pragma unroll
          for (int q = 0; q < NE; ++q) e[ct][q] = O::join(lo[q], hi[q]);
        }
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          const typename O::frag fa = O::template row<D>(sa, 16 * tt + l16, 32 * R, g);
#pragma unroll
          for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
            for (int q = 0; q < NE; ++q) acc[tt][ct] = O::mma(e[ct][q], fa, acc[tt][ct]);
        }
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const float f = j.w * power(g2, 16 * tt + l16 + j.e);
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) acc[tt][ct] *= f;
      }
      __syncthreads();
    }
    // the chunk's part of c, as the products take it
    typename O::frag fc[2][NCT];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int ct = 0; ct < NCT; ++ct) fc[m][ct] = O::template col<V>(sc, 32 * m, 16 * (wave * NCT + ct), lane);
    if constexpr (!STATES) {
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int m = 0; m <= tt / 2; ++m)
#pragma unroll
          for (int q = 0; q < NS; ++q) {
            const int i0 = tt * (tt + 1) / 2 + 2 * m;
            const typename O::half lo = sp[(i0 * NS + q) * 64 + lane];
            typename O::half hi{};
            if (2 * m + 1 <= tt) hi = sp[((i0 + 1) * NS + q) * 64 + lane];
            const typename O::frag fp = O::join(lo, hi);
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) acc[tt][ct] = O::mma(fc[m][ct], fp, acc[tt][ct]);
          }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const int p = 16 * tt + l16;
        if (p < nc) {
          const int64_t token = first + int64_t(dir) * (p0 + p);
#pragma unroll
          for (int ct = 0; ct < NCT; ++ct) {
            const int v = 16 * (wave * NCT + ct) + 4 * g;
            if (v < vc) put4<T>(j, static_cast<T*>(j.out), (token * plan.H + h) * j.c.cols + v0 + v, acc[tt][ct], vc - v);
          }
        }
      }
    }
    // the state behind the chunk
    typename O::frag wc[2][NCT][NW];
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      f32x4 wl, wh;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        wl[i] = j.u * power(g2, max(0, nc - j.e - (32 * m + 4 * g + i)));
        wh[i] = j.u * power(g2, max(0, nc - j.e - (32 * m + 16 + 4 * g + i)));
      }
#pragma unroll
      for (int ct = 0; ct < NCT; ++ct) {
        float v[8];
        O::values(fc[m][ct], v);
        typename O::half lo[NW], hi[NW];
        O::template split<NW>(wl * f32x4{v[0], v[1], v[2], v[3]}, lo);
        O::template split<NW>(wh * f32x4{v[4], v[5], v[6], v[7]}, hi);
#pragma unroll
        for (int q = 0; q < NW; ++q) wc[m][ct][q] = O::join(lo[q], hi[q]);
      }
    }
    const float whole = power(g2, nc);
#pragma unroll
    for (int r = 0; r < 2 * KB; ++r) {
#pragma unroll
      for (int ct = 0; ct < NCT; ++ct) E[r][ct] *= whole;
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        const typename O::frag fb = O::template col<D>(sb, 32 * m, 16 * r, lane);
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
          for (int q = 0; q < NW; ++q) E[r][ct] = O::mma(fb, wc[m][ct][q], E[r][ct]);
      }
    }
    __syncthreads();
  }

  float* fin = STATES ? j.states + (int64_t(unit) * plan.segs + seg + 1) * per : last_seg && j.fin != nullptr ? j.fin + unit * per : nullptr;
  if (fin == nullptr) return;
#pragma unroll
  for (int r = 0; r < 2 * KB; ++r)
#pragma unroll
    for (int ct = 0; ct < NCT; ++ct) {
      const int v = 16 * (wave * NCT + ct) + l16;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = 16 * r + 4 * g + i;
        if (row < j.b.cols && v < vc) fin[row * j.sn + (v0 + v) * j.sv] = E[r][ct][i];
      }
    }
}

template <typename T, int KB, int NCT, bool STATES>
hipError_t launch(const WalkPlan& p, hipStream_t s) {
  int64_t blocks = 0;
  for (int i = 0; i < p.jobs; ++i) blocks += int64_t(p.job[i].blocks) * p.Bt * p.H * (STATES ? p.segs - 1 : p.segs);
  constexpr int bytes = Lds<T, KB, NCT, STATES>::end;
  static std::atomic<uint64_t> cleared{0};
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(&walk_kernel<T, KB, NCT, STATES>), bytes, cleared);
  if (e != hipSuccess) return e;
  walk_kernel<T, KB, NCT, STATES><<<dim3(uint32_t(blocks)), dim3(256), bytes, s>>>(p);
  return hipGetLastError();
}

template <typename T>
hipError_t dispatch(const WalkPlan& p, int kb, int nct, bool states_only, hipStream_t s) {
  const int key = kb * 10 + nct;
  if (states_only) {
    switch (key) {
      case 11: return launch<T, 1, 1, true>(p, s);
      case 12: return launch<T, 1, 2, true>(p, s);
      case 21: return launch<T, 2, 1, true>(p, s);
      case 22: return launch<T, 2, 2, true>(p, s);
      case 41: return launch<T, 4, 1, true>(p, s);
      case 42: return launch<T, 4, 2, true>(p, s);
      case 81: return launch<T, 8, 1, true>(p, s);
    }
  } else {
    switch (key) {
      case 11: return launch<T, 1, 1, false>(p, s);
      case 12: return launch<T, 1, 2, false>(p, s);
      case 21: return launch<T, 2, 1, false>(p, s);
      case 22: return launch<T, 2, 2, false>(p, s);
      case 41: return launch<T, 4, 1, false>(p, s);
      case 42: return launch<T, 4, 2, false>(p, s);
      case 81: return launch<T, 8, 1, false>(p, s);
    }
  }
  return hipErrorInvalidValue;
}

}  // namespace walk
}  // namespace m3
