// The chunked walk of linear attention (see mixer_internal.hpp for its formula) on the
// matrix cores: y, dq, dk and dv, and the states of segments.
#pragma once
#include <atomic>
#include <type_traits>

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
  // bits, so that what a product adds to the outputs' own rounding (2^-8) and to the fp32
  // state is below either
  static constexpr int kScore = 2, kState = 2, kWeight = 3;
  // Rows of D elements, padded by 32 bytes, so that 8 bytes of 4 columns of each of 8 rows (a
  // transposing read) meet every bank once; and every address is a lane's own plus a constant.
  template <int D>
  static constexpr int stride() { return D + 16; }
  // row r, contracted positions of the block pair at column c
  template <int S>
  static __device__ __forceinline__ frag row(const elem* t, int r, int c, int lane) {
    const elem* p = t + ((lane & 15) * S + (lane >> 4) * 4) + (r * S + c);
    return cat8(*reinterpret_cast<const u32x2*>(p), *reinterpret_cast<const u32x2*>(p + 16));
  }
  // column c + l16, contracted positions: rows of the block pair at row r
  template <int S>
  static __device__ __forceinline__ frag col(const elem* t, int r, int c, int lane) {
    const elem* p = t + (((lane >> 4) * 4 + ((lane & 15) >> 2)) * S + (lane & 3) * 4) + (r * S + c);
    return cat8(lds_read_tr(p), lds_read_tr(p + 16 * S));
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
  static constexpr int stride() { return D + 4; }
  template <int S>
  static __device__ __forceinline__ frag row(const elem* t, int r, int c, int lane) {
    const elem* p = t + ((lane & 15) * S + (lane >> 4) * 4) + (r * S + c);
    return {*reinterpret_cast<const f32x4*>(p), *reinterpret_cast<const f32x4*>(p + 16)};
  }
  template <int S>
  static __device__ __forceinline__ frag col(const elem* t, int r, int c, int lane) {
    const elem* p = t + ((lane >> 4) * 4 * S + (lane & 15)) + (r * S + c);
    frag f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f.lo[i] = p[i * S];
      f.hi[i] = p[(16 + i) * S];
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

// Tiles in LDS: where the words of 16 bytes of row r from column c on go.  Padded rows, for
// the one-phase walk; rows swizzled by XOR as its a and as its b and c, for the two-role walk.
template <typename T, int D>
struct Padded {
  typedef typename Op<T>::elem elem;
  static constexpr int S = Op<T>::template stride<D>(), kBytes = kChunk * S * int(sizeof(elem));
  static __device__ __forceinline__ void put(elem* t, int r, int c, u32x4 w) { *reinterpret_cast<u32x4*>(t + r * S + c) = w; }
};
constexpr int shift_of(int D) { return D >= 128 ? 0 : D == 64 ? 1 : 2; }
// a: operands of 8 positions lie together, 16 bytes; 16 rows of one meet every bank once
template <int D>
struct SwizzledA {
  static constexpr int S = D, kBytes = kChunk * D * 2;
  static __device__ __forceinline__ int mix(int r) { return (r & 15) >> shift_of(D); }
  static __device__ __forceinline__ void put(uint16_t* t, int r, int c, u32x4 w) {
    const int u = c / 32 * 4 + (c & 8) / 4, h = (c & 16) / 4;  // units of columns c.. and c + 4..
    *reinterpret_cast<u32x2*>(t + r * D + (u ^ mix(r)) * 8 + h) = u32x2{w[0], w[1]};
    *reinterpret_cast<u32x2*>(t + r * D + ((u + 1) ^ mix(r)) * 8 + h) = u32x2{w[2], w[3]};
  }
  // a lane's element offset of the operand of row l16 at block pair R
  static __device__ __forceinline__ int row(int R, int lane) { return (lane & 15) * D + ((4 * R + (lane >> 4)) ^ mix(lane & 15)) * 8; }
};
// b and c: units of 8 bytes; 16 rows of two of them, and 8 rows of four, meet every bank once
template <int D>
struct SwizzledB {
  static constexpr int S = D, kBytes = kChunk * D * 2;
  static __device__ __forceinline__ int mix(int r) { return (((r & 7) >> shift_of(D)) << 2) | ((r >> 3 & 1) << 1); }
  static __device__ __forceinline__ void put(uint16_t* t, int r, int c, u32x4 w) {
    *reinterpret_cast<u32x4*>(t + r * D + ((c / 4) ^ mix(r)) * 4) = w;
  }
  static __device__ __forceinline__ int row(int c, int lane) { return (lane & 15) * D + ((c / 4 + (lane >> 4)) ^ mix(lane & 15)) * 4; }
  // where the lane points for a transposing read of columns c..c + 15, rows 4 g + 0..3 of 16
  static __device__ __forceinline__ int col(int c, int lane) {
    const int r = (lane >> 4) * 4 + ((lane & 15) >> 2);
    return r * D + ((c / 4 + (lane & 3)) ^ mix(r)) * 4;
  }
};

// c of the two-role walk, 64 columns.  An operand's 16 columns are 4 of each of four words of 8 of
// one half, so that two operands of a token are 16 bytes of each of its output's four lanes:
// tile w's column m is 32 (w / 2) + 8 (m / 4) + 4 (w % 2) + m % 4.  Units of 8 bytes; 8 rows of
// the four of a tile meet every bank once.
struct SwizzledC {
  static constexpr int S = 64, kBytes = kChunk * 64 * 2;
  static __device__ __forceinline__ int column(int tile, int m) { return 32 * (tile >> 1) + 8 * (m >> 2) + 4 * (tile & 1) + (m & 3); }
  static __device__ __forceinline__ int mix(int r) { return ((r >> 2 & 1) << 3) | (r >> 1 & 1); }
  static __device__ __forceinline__ void put(uint16_t* t, int r, int c, u32x4 w) {
    *reinterpret_cast<u32x2*>(t + r * S + ((c / 4) ^ mix(r)) * 4) = u32x2{w[0], w[1]};
    *reinterpret_cast<u32x2*>(t + r * S + ((c / 4 + 1) ^ mix(r)) * 4) = u32x2{w[2], w[3]};
  }
  // where the lane points for a transposing read of a tile's columns, rows 4 g + 0..3 of 16
  static __device__ __forceinline__ int col(int tile, int lane) {
    const int r = (lane >> 4) * 4 + ((lane & 15) >> 2);
    return r * S + ((column(tile, 4 * (lane & 3)) / 4) ^ mix(r)) * 4;
  }
};

// 64 tokens' rows of D elements (columns past the head's and rows past the chunk's zero) on
// their way through registers into LDS, 16-byte words over 256 threads.  Rows are loaded in
// the tokens' order and stored in the walk's.
template <typename T, int D, typename To>
struct Tile {
  typedef typename Op<T>::elem elem;
  static constexpr int W = Op<T>::kWord, kRow = D / W, kRows = 256 / kRow, N = kChunk / kRows;
  static_assert(N >= 1 && 256 % kRow == 0, "whole rows over the block");
  typedef u32x4 words[N];
  uint32_t at;  // this thread's bytes from a chunk's first element
  int r0, c0;   // its first row and its column
  __device__ __forceinline__ Tile(int64_t ld, int cols, int thread) {
    r0 = thread / kRow;
    c0 = thread % kRow * W;
    at = (uint32_t(r0) * uint32_t(ld) + uint32_t(c0 < cols ? c0 : 0)) * uint32_t(sizeof(T));
  }
  // a whole chunk of whole words; columns past the head's are others' here, and zeroed when stored
  __device__ __forceinline__ void load(words& w, const T* base, int64_t ld) const {
#pragma unroll
    for (int i = 0; i < N; ++i)
      w[i] = *reinterpret_cast<const u32x4*>(reinterpret_cast<const char*>(base + int64_t(i * kRows) * ld) + at);
  }
  // whole chunks: a place per thread and constant steps (rows of one are 16 apart, which the
  // swizzles do not see)
  __device__ __forceinline__ void store_whole(words& w, elem* t, int cols, bool rev) const {
    if (cols < D) {
#pragma unroll
      for (int i = 0; i < N; ++i) w[i] = c0 < cols ? w[i] : u32x4{0, 0, 0, 0};
    }
    if constexpr (kRows % 16 == 0) {
      if (rev) {
#pragma unroll
        for (int i = 0; i < N; ++i) To::put(t + (N - 1 - i) * kRows * To::S, kRows - 1 - r0, c0, w[i]);
      } else {
#pragma unroll
        for (int i = 0; i < N; ++i) To::put(t + i * kRows * To::S, r0, c0, w[i]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) To::put(t, rev ? kChunk - 1 - i * kRows - r0 : i * kRows + r0, c0, w[i]);
    }
  }
  // n tokens, any words
  __device__ __forceinline__ void load_any(words& w, const T* base, int64_t ld, int n, int cols) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = i * kRows + r0, left = r < n ? cols - c0 : 0;
      const T* p = base + int64_t(r < n ? r : 0) * ld + (left > 0 ? c0 : 0);
      Pack<T, W> q;
      if (left >= W) q = load_loose<T, W>(p);
      else q = load_some<T, W>(p, left);
      __builtin_memcpy(&w[i], &q, 16);
    }
  }
  __device__ __forceinline__ void store(words& w, elem* t, int n, int cols, bool rev) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int r = i * kRows + r0;
      if (cols < D) w[i] = c0 < cols ? w[i] : u32x4{0, 0, 0, 0};
      To::put(t, rev && r < n ? n - 1 - r : r, c0, w[i]);
    }
  }
};

// Four consecutive columns of the output, n of them within the head.
template <typename T, bool FAST>
__device__ __forceinline__ void put4(bool f32, bool words, char* out, uint32_t at, f32x4 v, int n) {
  if (sizeof(T) == 4 || f32) {
    float* o = reinterpret_cast<float*>(out + at * 4u);
    if (FAST || (words && n >= 4)) {
      *reinterpret_cast<f32x4*>(o) = v;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) o[i] = v[i];
    }
  } else {
    T* o = reinterpret_cast<T*>(out + at * uint32_t(sizeof(T)));
    if (FAST || (words && n >= 4)) {
      store4<T>(o, v[0], v[1], v[2], v[3]);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (i < n) store_scalar<T>(o + i, v[i]);
    }
  }
}

// ---------------------------------------------------------------- what a block walks
// One segment of one (item, head) for V columns of c: 4 waves hold V / 4 columns of the state
// each, all its rows, in accumulators.
template <typename T, int V, bool STATES, bool MIXED = false>
struct Place {
  const WalkPlan& plan;
  const WalkJob& j;
  int vt, unit, seg, item, h, n, from, to, v0, vc, chunks, rest;
  bool rev, last_seg, idle;
  float g2;
  int64_t per;
  static __device__ __forceinline__ int job_of(const WalkPlan& plan, int64_t& id) {
    const int units = plan.Bt * plan.H, segs = STATES ? plan.segs - 1 : plan.segs;
    int ji = 0;
    while (ji + 1 < plan.jobs && id >= int64_t(plan.job[ji].blocks) * units * segs) {
      id -= int64_t(plan.job[ji].blocks) * units * segs;
      ++ji;
    }
    return ji;
  }
  __device__ __forceinline__ Place(const WalkPlan& p, int64_t id) : plan(p), j(p.job[job_of(p, id)]) {
    const int units = plan.Bt * plan.H;
    vt = int(id % j.blocks);
    unit = int(id / j.blocks % units);
    seg = int(id / j.blocks / units);
    item = unit / plan.H;
    h = unit % plan.H;
    n = __builtin_amdgcn_readfirstlane(item_length(plan.lengths, item, plan.L));  // the same for the block
    from = seg * plan.seg_len;
    to = min(n, from + plan.seg_len);
    v0 = vt * V;
    vc = min(j.c.cols - v0, V);
    rev = j.rev != 0;
    g2 = __builtin_bit_cast(float, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, plan.log_decay[h] * 1.4426950408889634f)));
    per = int64_t(j.b.cols) * j.c.cols;
    last_seg = from + plan.seg_len >= n;  // of this item
    idle = STATES ? last_seg : (from >= n && seg > 0);
    chunks = to > from ? (to - from + kChunk - 1) / kChunk : 0;
    rest = to - from - (chunks - 1) * kChunk;
  }
  __device__ __forceinline__ int held(int k) const { return k + 1 < chunks ? kChunk : rest; }
  // the first token in memory of chunk k
  __device__ __forceinline__ int64_t token(int k) const {
    return int64_t(item) * plan.L + (rev ? n - from - k * kChunk - held(k) : from + k * kChunk);
  }
  __device__ __forceinline__ const T* head(const WalkSide& s) const {
    return static_cast<const T*>(s.p) + int64_t(h / (plan.H / s.heads)) * s.cols;
  }
  // zeros into the output's rows behind the item's tokens
  __device__ __forceinline__ void zero_tail(int threads) const {
    const int first = max(n, from), last = min(plan.L, from + plan.seg_len);
    T* o = static_cast<T*>(j.out);
    for (int64_t i = threadIdx.x; i < int64_t(last - first) * vc; i += threads)
      o[((int64_t(item) * plan.L + first + i / vc) * plan.H + h) * j.c.cols + v0 + i % vc] = T{};
  }
  // the state's rows 16 r + 4 g + i, columns:
  static __device__ __forceinline__ int column(int tile, int lane) {
    return MIXED ? SwizzledC::column(tile, lane & 15) : 16 * tile + (lane & 15);
  }
  template <int NR, int NCT>
  __device__ __forceinline__ void start(f32x4 (&E)[NR][NCT], int wave, int lane) const {
    const float* init = nullptr;
    if constexpr (!STATES) init = plan.segs > 1 ? j.states + (int64_t(unit) * plan.segs + seg) * per : j.init == nullptr ? nullptr : j.init + unit * per;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int ct = 0; ct < NCT; ++ct) {
        const int v = column(wave * NCT + ct, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * r + 4 * (lane >> 4) + i;
          E[r][ct][i] = init != nullptr && row < j.b.cols && v < vc ? init[row * j.sn + (v0 + v) * j.sv] : 0.f;
        }
      }
  }
  template <int NR, int NCT>
  __device__ __forceinline__ void finish(const f32x4 (&E)[NR][NCT], int wave, int lane) const {
    float* fin = STATES ? j.states + (int64_t(unit) * plan.segs + seg + 1) * per : last_seg && j.fin != nullptr ? j.fin + unit * per : nullptr;
    if (fin == nullptr) return;
#pragma unroll
    for (int r = 0; r < NR; ++r)
#pragma unroll
      for (int ct = 0; ct < NCT; ++ct) {
        const int v = column(wave * NCT + ct, lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int row = 16 * r + 4 * (lane >> 4) + i;
          if (row < j.b.cols && v < vc) fin[row * j.sn + (v0 + v) * j.sv] = E[r][ct][i];
        }
      }
  }
  // chunks in front of this one are whole ones of whole words
  __device__ __forceinline__ int quick() const {
    const bool words = (STATES || (j.a.words && j.out_words == 2 && vc == V)) && j.b.words && j.c.words;
    return words ? (rest == kChunk ? chunks : chunks - 1) : 0;
  }
};

// Weights l^(p - j) s of a triangle's tiles (rows j = 4 g + i, columns p = l16), and l^(p + e) w.
struct Powers {
  float near[4], far[4], out[4], far2, far3;
  __device__ __forceinline__ Powers(float g2, const WalkJob& j, int lane) {
    const int g = lane >> 4, l16 = lane & 15;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = l16 - 4 * g - i;
      near[i] = d < 0 ? 0.f : j.s * power(g2, d);
      far[i] = j.s * power(g2, 16 + d);
      out[i] = j.w * power(g2, 16 * i + l16 + j.e);
    }
    far2 = power(g2, 16);
    far3 = power(g2, 32);
  }
  // scores of tiles `apart` apart
  __device__ __forceinline__ f32x4 weigh(f32x4 s, int apart, int lane) const {
    const float f = apart == 3 ? far3 : apart == 2 ? far2 : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float v = s[i] * (apart == 0 ? near[i] : far[i] * f);
      s[i] = apart == 0 && (lane & 15) < 4 * (lane >> 4) + i ? 0.f : v;
    }
    return s;
  }
};
// The triangle's 10 tiles (tt, jt <= tt) in order, and the 6 operands of 32 positions they
// make: pair_of(tt, jt / 2); the second halves of (0, 0) and (2, 1) are empty.
__device__ __forceinline__ int column_of(int tile) { return tile < 1 ? 0 : tile < 3 ? 1 : tile < 6 ? 2 : 3; }
constexpr __host__ __device__ int pair_of(int tt, int m) { return (tt * (tt + 2) + 1) / 4 + m; }

// u l^(n - e - i) for the tokens of a whole chunk and of the last one
__device__ __forceinline__ void put_weights(float* sw, float g2, const WalkJob& j, int rest) {
  if (threadIdx.x < 2 * kChunk) {
    const int i = threadIdx.x % kChunk, nc = threadIdx.x < kChunk ? kChunk : rest;
    sw[threadIdx.x] = j.u * power(g2, max(0, nc - j.e - i));
  }
}
// c's operands of 32 tokens times their weights, in parts
template <typename O, int NW>
__device__ __forceinline__ void weigh_column(typename O::frag f, f32x4 wl, f32x4 wh, typename O::frag (&o)[NW]) {
  float v[8];
  O::values(f, v);
  typename O::half lo[NW], hi[NW];
  O::template split<NW>(wl * f32x4{v[0], v[1], v[2], v[3]}, lo);
  O::template split<NW>(wh * f32x4{v[4], v[5], v[6], v[7]}, hi);
#pragma unroll
  for (int q = 0; q < NW; ++q) o[q] = O::join(lo[q], hi[q]);
}
// e(R): the state's rows of block pair R as an operand, in parts
template <typename O, int NE>
__device__ __forceinline__ void state_operand(f32x4 a, f32x4 b, typename O::frag (&o)[NE]) {
  typename O::half lo[NE], hi[NE];
  O::template split<NE>(a, lo);
  O::template split<NE>(b, hi);
#pragma unroll
  for (int q = 0; q < NE; ++q) o[q] = O::join(lo[q], hi[q]);
}

// ---------------------------------------------------------------- one-phase walk
// 4 waves, 64 NCT columns: tiles into LDS; scores, dealt over the waves, and the state's part;
// scores times c, out, and the state behind the chunk.  For segments' states, for fp32, and for
// a and b of more than 128 elements, whose tiles leave LDS no room for two chunks.  fp32, Bt 16,
// L 1024, 32 heads of 128 x 128: 503 us, bound by the fp32 matrix instructions, which take 290 of
// them at their peak rate, between waits for LDS; two blocks share a compute unit where they fit.
template <typename T, int KB, int NCT, bool STATES>
struct Lds {
  static constexpr int D = 32 * KB, V = 64 * NCT;
  static constexpr int tD = Padded<T, D>::kBytes, tV = Padded<T, V>::kBytes;
  static constexpr int a = 0, b = STATES ? 0 : tD, c = b + tD, p = c + tV,
                       w = p + (STATES ? 0 : 6 * Op<T>::kScore * 64 * int(sizeof(typename Op<T>::frag))), end = w + 2 * kChunk * 4;
  static_assert(end <= 160 * 1024, "a compute unit's LDS");
};

template <typename T, int KB, int NCT, bool STATES>
__global__ __launch_bounds__(256, (KB * NCT <= 4 ? 2 : 1)) void walk_kernel(WalkPlan plan) {
  typedef Op<T> O;
  typedef Lds<T, KB, NCT, STATES> M;
  typedef typename O::elem elem;
  typedef typename O::frag frag;
  typedef typename O::half half;
  constexpr int D = M::D, V = M::V, SD = Padded<T, D>::S, SV = Padded<T, V>::S, NS = O::kScore, NE = O::kState, NW = O::kWeight;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  elem* sa = reinterpret_cast<elem*>(lds + M::a);
  elem* sb = reinterpret_cast<elem*>(lds + M::b);
  elem* sc = reinterpret_cast<elem*>(lds + M::c);
  half* sp = reinterpret_cast<half*>(lds + M::p);
  float* sw = reinterpret_cast<float*>(lds + M::w);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), g = lane >> 4, l16 = lane & 15;
  const Place<T, V, STATES> at(plan, block_on_xcd());
  const WalkJob& j = at.j;
  if constexpr (!STATES) {
    if (j.zero_tail) at.zero_tail(256);
  }
  if (at.idle) return;
  f32x4 E[2 * KB][NCT];
  at.start(E, wave, lane);
  put_weights(sw, at.g2, j, at.rest);
  const float whole = power(at.g2, kChunk), whole_rest = power(at.g2, max(0, at.rest));
  const Powers pw(at.g2, j, lane);
  const int chunks = at.chunks;
  const bool rev = at.rev, out_f32 = j.out_f32 != 0, out_words = j.out_words != 0;
  const int a_cols = j.a.cols, b_cols = j.b.cols, vc = at.vc;
  const int64_t a_ld = j.a.ld, b_ld = j.b.ld, c_ld = j.c.ld, way = rev ? -kChunk : kChunk;
  const T *pa = STATES ? nullptr : at.head(j.a), *pb = at.head(j.b), *pc = at.head(j.c) + at.v0;
  typedef Tile<T, D, Padded<T, D>> TD;
  typedef Tile<T, V, Padded<T, V>> TV;
  const TD ta(a_ld, a_cols, threadIdx.x), tb(b_ld, b_cols, threadIdx.x);
  const TV tc(c_ld, vc, threadIdx.x);
  typename TD::words wa, wb;
  typename TV::words wc;
  auto load_any = [&](int k) {
    const int64_t t = at.token(k);
    if constexpr (!STATES) ta.load_any(wa, pa + t * a_ld, a_ld, at.held(k), a_cols);
    tb.load_any(wb, pb + t * b_ld, b_ld, at.held(k), b_cols);
    tc.load_any(wc, pc + t * c_ld, c_ld, at.held(k), vc);
  };
  auto store = [&](int n) {
    if constexpr (!STATES) ta.store(wa, sa, n, a_cols, rev);
    tb.store(wb, sb, n, b_cols, rev);
    tc.store(wc, sc, n, vc, rev);
  };
  if constexpr (!STATES) {
    for (int i = wave; i < 2 * NS; i += 4) sp[(pair_of(i & 1 ? 2 : 0, i & 1) * NS + i / 2) * 128 + lane * 2 + 1] = half{};
  }
  const uint32_t out_row = uint32_t(plan.H) * uint32_t(j.c.cols);
  auto middle = [&](int k, auto fast) {
    constexpr bool FAST = decltype(fast)::value;
    const int nc = FAST ? kChunk : at.held(k);
    const bool full = nc == kChunk;
    __syncthreads();
    f32x4 acc[4][NCT];
    if constexpr (!STATES) {
      // scores transposed: rows j, columns p
#pragma unroll
      for (int x = 0; x < 3; ++x) {
        const int tile = wave + 4 * x;
        if (tile < 10) {
          const int tt = column_of(tile), jt = tile - tt * (tt + 1) / 2;
          f32x4 s = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int R = 0; R < KB; ++R)
            s = O::mma(O::template row<SD>(sb + 16 * jt * SD, 0, 32 * R, lane), O::template row<SD>(sa + 16 * tt * SD, 0, 32 * R, lane), s);
          half o[NS];
          O::template split<NS>(pw.weigh(s, tt - jt, lane), o);
#pragma unroll
          for (int q = 0; q < NS; ++q) sp[((pair_of(tt, jt / 2) * NS + q) * 64 + lane) * 2 + (jt & 1)] = o[q];
        }
      }
      // a E, transposed: rows v, columns p
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) acc[tt][ct] = f32x4{0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int R = 0; R < KB; ++R) {
        frag e[NCT][NE];
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) state_operand<O, NE>(E[2 * R][ct], E[2 * R + 1][ct], e[ct]);
#pragma unroll
        for (int tt = 0; tt < 4; ++tt) {
          const frag fa = O::template row<SD>(sa, 16 * tt, 32 * R, lane);
#pragma unroll
          for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
            for (int q = 0; q < NE; ++q) acc[tt][ct] = O::mma(e[ct][q], fa, acc[tt][ct]);
        }
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt)
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct) acc[tt][ct] *= pw.out[tt];
      __syncthreads();
    }
    frag fc[2][NCT];
#pragma unroll
    for (int m = 0; m < 2; ++m)
#pragma unroll
      for (int ct = 0; ct < NCT; ++ct) fc[m][ct] = O::template col<SV>(sc + 16 * NCT * wave, 32 * m, 16 * ct, lane);
    if constexpr (!STATES) {
#pragma unroll
      for (int m = 0; m < 2; ++m)
#pragma unroll
        for (int q = 0; q < NS; ++q)
#pragma unroll
          for (int tt = 2 * m; tt < 4; ++tt) {
            const frag fp = *reinterpret_cast<const frag*>(sp + ((pair_of(tt, m) * NS + q) * 64 + lane) * 2);
#pragma unroll
            for (int ct = 0; ct < NCT; ++ct) acc[tt][ct] = O::mma(fc[m][ct], fp, acc[tt][ct]);
          }
      char* out = static_cast<char*>(j.out) + (at.token(k) * plan.H * j.c.cols + int64_t(at.h) * j.c.cols + at.v0) * (sizeof(T) == 4 || out_f32 ? 4 : int(sizeof(T)));
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) {
        const int p = 16 * tt + l16;
        if (FAST || p < nc) {
          const uint32_t row = uint32_t(rev ? nc - 1 - p : p) * out_row;
#pragma unroll
          for (int ct = 0; ct < NCT; ++ct) {
            const int v = 16 * (wave * NCT + ct) + 4 * g;
            if (FAST || v < vc) put4<T, FAST>(out_f32, out_words, out, row + v, acc[tt][ct], vc - v);
          }
        }
      }
    }
    // the state behind the chunk
    const float f = full ? whole : whole_rest;
    const float* W = sw + (full ? 0 : kChunk);
#pragma unroll
    for (int r = 0; r < 2 * KB; ++r)
#pragma unroll
      for (int ct = 0; ct < NCT; ++ct) E[r][ct] *= f;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      const f32x4 wl = *reinterpret_cast<const f32x4*>(W + 32 * m + 4 * g), wh = *reinterpret_cast<const f32x4*>(W + 32 * m + 16 + 4 * g);
      frag fw[NCT][NW];
#pragma unroll
      for (int ct = 0; ct < NCT; ++ct) weigh_column<O, NW>(fc[m][ct], wl, wh, fw[ct]);
#pragma unroll
      for (int r = 0; r < 2 * KB; ++r) {
        const frag fb = O::template col<SD>(sb, 32 * m, 16 * r, lane);
#pragma unroll
        for (int ct = 0; ct < NCT; ++ct)
#pragma unroll
          for (int q = 0; q < NW; ++q) E[r][ct] = O::mma(fb, fw[ct][q], E[r][ct]);
      }
    }
    __syncthreads();
  };
  if (chunks > 0) load_any(0);
  const int quick = at.quick();
  int k = 0;
  for (; k + 1 < quick; ++k) {
    const int64_t t = at.token(k) + way;
    if constexpr (!STATES) ta.store_whole(wa, sa, a_cols, rev);
    tb.store_whole(wb, sb, b_cols, rev);
    tc.store_whole(wc, sc, vc, rev);
    if constexpr (!STATES) ta.load(wa, pa + t * a_ld, a_ld);
    tb.load(wb, pb + t * b_ld, b_ld);
    tc.load(wc, pc + t * c_ld, c_ld);
    __builtin_amdgcn_sched_barrier(0);  // asked for now, not where the scheduler finds a register for them
    middle(k, std::true_type{});
  }
  for (; k < chunks; ++k) {
    store(at.held(k));
    if (k + 1 < chunks) load_any(k + 1);
    middle(k, std::false_type{});
  }
  at.finish(E, wave, lane);
}

// ---------------------------------------------------------------- two-role walk
// bf16, a and b of up to 128 elements, 64 columns: 8 waves, two on each SIMD.  The first four
// hold the state: its part of the next chunk's outputs, handed over through LDS, and its
// update.  The other four form the scores and the outputs.  So matrix instructions of the one
// run beside loads, conversions and waits of the other, and a chunk takes one barrier: between
// two of them, for chunk k,
//   state waves: b of k + 2 and c of k + 1 into LDS and those two further on asked for, update
//   with k, then a E for k + 1;
//   others: a of k + 2 into LDS and k + 4's asked for, scores of k + 1 (two waves 2 x 2 tiles
//   of the triangle's lower half each, two 1 x 2 of its upper), scores times c and out for k
//   (the upper half's waves have the half with more of it).
// Bt 8, L 4096, 16 heads of 128 x 128: 165 us, 3.3 TB/s.  A chunk takes 5,700 cycles: the vector
// units issue 2,500 of them, the matrix units are busy 1,650; leaving out any one part (scores
// 35 us, loads, stores or outputs 15 each) saves its own time, so that it is the sum of
// instructions and of LDS's latency under 8 waves, and not memory, that bounds it.  Four waves
// doing all of it took 280 us, one at a time waiting for LDS 212.
template <int KB>
struct PairLds {
  static constexpr int D = 32 * KB;
  static constexpr int tA = SwizzledA<D>::kBytes, tB = SwizzledB<D>::kBytes, tC = SwizzledC::kBytes, tP = 6 * 2 * 64 * 16, tX = 16 * 64 * 16;
  static constexpr int a = 0, b = a + 2 * tA, c = b + 3 * tB, p = c + 2 * tC, x = p + 2 * tP, w = x + 2 * tX, end = w + 2 * kChunk * 4;
  static_assert(end <= 160 * 1024, "a compute unit's LDS");
};

template <int KB>
__global__ __launch_bounds__(512, 1) __attribute__((amdgpu_waves_per_eu(2, 2))) void pair_kernel(WalkPlan plan) {
  typedef Op<bf16_t> O;
  typedef PairLds<KB> M;
  typedef O::frag frag;
  typedef O::half half;
  constexpr int D = M::D, V = 64, NS = O::kScore, NE = O::kState, NW = O::kWeight;
  static_assert(NS == 2, "room for the scores");
  typedef SwizzledA<D> A;
  typedef SwizzledB<D> B;
  typedef SwizzledC C;
  extern __shared__ __attribute__((aligned(16))) char lds[];
  auto sa = [&](int i) { return reinterpret_cast<uint16_t*>(lds + M::a + i * M::tA); };
  auto sb = [&](int i) { return reinterpret_cast<uint16_t*>(lds + M::b + i * M::tB); };
  auto sc = [&](int i) { return reinterpret_cast<uint16_t*>(lds + M::c + i * M::tC); };
  auto sp = [&](int i) { return reinterpret_cast<half*>(lds + M::p + i * M::tP); };
  auto sx = [&](int i) { return reinterpret_cast<f32x4*>(lds + M::x + i * M::tX); };
  float* sw = reinterpret_cast<float*>(lds + M::w);
  const int lane = threadIdx.x & 63, role = __builtin_amdgcn_readfirstlane(threadIdx.x >> 8), wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6) & 3,
            g = lane >> 4, l16 = lane & 15;
  const Place<bf16_t, V, false, true> at(plan, block_on_xcd());
  const WalkJob& j = at.j;
  if (j.zero_tail) at.zero_tail(512);
  if (at.idle) return;
  put_weights(sw, at.g2, j, at.rest);
  const Powers pw(at.g2, j, lane);
  const int chunks = at.chunks;
  // c's operand of tokens 32 m.. and a tile's columns, from where the lane points
  auto column = [&](const uint16_t* t, int m) { return cat8(lds_read_tr(t + 32 * m * V), lds_read_tr(t + (32 * m + 16) * V)); };

  const bool rev = at.rev;
  const int thread = threadIdx.x & 255, vc = at.vc, quick = at.quick();
  const int64_t way = rev ? -kChunk : kChunk;
  std::integral_constant<int, 0> even;
  std::integral_constant<int, 1> odd;
  if (role == 0) {
    f32x4 E[2 * KB][1];
    at.start(E, wave, lane);
    typedef Tile<bf16_t, V, C> TC;
    typedef Tile<bf16_t, D, B> TB;
    const int b_cols = j.b.cols;
    const int64_t b_ld = j.b.ld, c_ld = j.c.ld;
    const TB tb(b_ld, b_cols, thread);
    const TC tc(c_ld, vc, thread);
    typename TB::words wb[2];
    TC::words wc[2];  // of chunk k in set k & 1
    const bf16_t *pb = at.head(j.b), *nb = pb, *pc = at.head(j.c) + at.v0, *nc = pc;  // n: the next whole chunk's first token
    auto any_b = [&](int k, auto set) { tb.load_any(wb[decltype(set)::value], pb + at.token(k) * b_ld, b_ld, at.held(k), b_cols); };
    auto any_c = [&](int k, auto set) { tc.load_any(wc[decltype(set)::value], pc + at.token(k) * c_ld, c_ld, at.held(k), vc); };
    if (quick > 4) {
      nb += at.token(4) * b_ld;
      nc += at.token(3) * c_ld;
    }
    const float whole = power(at.g2, kChunk), whole_rest = power(at.g2, max(0, at.rest));
    const int at_c = C::col(wave, lane);
    int at_a[KB], at_b[2 * KB];
#pragma unroll
    for (int R = 0; R < KB; ++R) at_a[R] = A::row(R, lane);
#pragma unroll
    for (int r = 0; r < 2 * KB; ++r) at_b[r] = B::col(16 * r, lane);
    // Reads of LDS are asked for ahead of the products in front of those that need them:
    // left to itself the scheduler waits for each (12 waits of 230 cycles made 60% of a chunk).
    auto ahead = [] { __builtin_amdgcn_sched_barrier(0); };
    auto rows_of_a = [&](const uint16_t* t, int R, frag (&f)[4]) {
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) f[tt] = as_bf16x8(*reinterpret_cast<const u32x4*>(t + at_a[R] + 16 * tt * D));
    };
    // acc = a E: e, the state in parts
    auto inter = [&](const uint16_t* t, f32x4* x, const frag (&e)[KB][NE], frag (&first)[4]) {
      f32x4 acc[4] = {};
      frag fa[2][4];
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) fa[0][tt] = first[tt];
#pragma unroll
      for (int R = 0; R < KB; ++R) {
        if (R + 1 < KB) rows_of_a(t, R + 1, fa[(R + 1) & 1]);
        ahead();
#pragma unroll
        for (int q = 0; q < NE; ++q)
#pragma unroll
          for (int tt = 0; tt < 4; ++tt) acc[tt] = O::mma(e[R][q], fa[R & 1][tt], acc[tt]);
      }
#pragma unroll
      for (int tt = 0; tt < 4; ++tt) x[(tt * 4 + wave) * 64 + lane] = acc[tt] * pw.out[tt];
    };
    frag e[KB][NE], first[4];
    if (chunks > 0) {
      any_b(0, even);
      tb.store(wb[0], sb(0), at.held(0), b_cols, rev);
      any_c(0, even);
      tc.store(wc[0], sc(0), at.held(0), vc, rev);
      if (chunks > 1) {
        any_b(1, odd);
        tb.store(wb[1], sb(1), at.held(1), b_cols, rev);
        any_c(1, odd);
      }
      if (chunks > 2) {
        any_b(2, even);
        any_c(2, even);
      }
      if (chunks > 3) any_b(3, odd);
      __syncthreads();
      rows_of_a(sa(0), 0, first);
#pragma unroll
      for (int R = 0; R < KB; ++R) state_operand<O, NE>(E[2 * R][0], E[2 * R + 1][0], e[R]);
      inter(sa(0), sx(0), e, first);
    }
    int b0 = 0, b2 = 2;  // b's tiles of chunks k and k + 2
    auto turn = [&](int k, auto set, auto whole_chunks) {  // k & 1 = set
      constexpr int S = decltype(set)::value;
      constexpr bool FAST = decltype(whole_chunks)::value;
      const bool full = FAST || at.held(k) == kChunk, more = FAST || k + 1 < chunks;
      const float f = full ? whole : whole_rest;
      const float* W = sw + (full ? 0 : kChunk);
      __syncthreads();
      const uint16_t *bt = sb(b0), *ct = sc(S);
      auto columns_of_b = [&](int R, frag (&o)[2][2]) {
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int x = 0; x < 2; ++x)
            o[m][x] = cat8(lds_read_tr(bt + at_b[2 * R + x] + 32 * m * D), lds_read_tr(bt + at_b[2 * R + x] + (32 * m + 16) * D));
      };
      frag fc[2], fw[2][NW], fb[2][2][2];
      f32x4 wt[2][2];
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        fc[m] = column(ct + at_c, m);
        wt[m][0] = *reinterpret_cast<const f32x4*>(W + 32 * m + 4 * g);
        wt[m][1] = *reinterpret_cast<const f32x4*>(W + 32 * m + 16 + 4 * g);
      }
      columns_of_b(0, fb[0]);
      if constexpr (FAST) {
        tb.store_whole(wb[S], sb(b2), b_cols, rev);
        tc.store_whole(wc[1 - S], sc(1 - S), vc, rev);
        tb.load(wb[S], nb, b_ld);
        tc.load(wc[1 - S], nc, c_ld);
        nb += way * b_ld;
        nc += way * c_ld;
      } else {
        if (k + 2 < chunks) tb.store(wb[S], sb(b2), at.held(k + 2), b_cols, rev);
        if (k + 4 < chunks) any_b(k + 4, set);
        if (more) tc.store(wc[1 - S], sc(1 - S), at.held(k + 1), vc, rev);
        if (k + 3 < chunks) any_c(k + 3, std::integral_constant<int, 1 - S>());
      }
      ahead();
#pragma unroll
      for (int m = 0; m < 2; ++m) weigh_column<O, NW>(fc[m], wt[m][0], wt[m][1], fw[m]);
#pragma unroll
      for (int R = 0; R < KB; ++R) {
        if (R + 1 < KB) columns_of_b(R + 1, fb[(R + 1) & 1]);
        else if (more) rows_of_a(sa(1 - S), 0, first);
        ahead();
        if (R > 0) state_operand<O, NE>(E[2 * R - 2][0], E[2 * R - 1][0], e[R - 1]);
#pragma unroll
        for (int x = 0; x < 2; ++x) E[2 * R + x][0] *= f;
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int q = 0; q < NW; ++q)
#pragma unroll
            for (int x = 0; x < 2; ++x) E[2 * R + x][0] = O::mma(fb[R & 1][m][x], fw[m][q], E[2 * R + x][0]);
      }
      state_operand<O, NE>(E[2 * KB - 2][0], E[2 * KB - 1][0], e[KB - 1]);
      if (more) inter(sa(1 - S), sx(1 - S), e, first);
      b0 = b0 == 2 ? 0 : b0 + 1;
      b2 = b2 == 2 ? 0 : b2 + 1;
    };
    int k = 0;
    for (; k + 5 < quick; k += 2) {
      turn(k, even, std::true_type{});
      turn(k + 1, odd, std::true_type{});
    }
    for (; k < chunks; k += 2) {
      turn(k, even, std::false_type{});
      if (k + 1 < chunks) turn(k + 1, odd, std::false_type{});
    }
    at.finish(E, wave, lane);
    return;
  }

  const bool out_f32 = j.out_f32 != 0, out_words = j.out_words != 0;
  const int a_cols = j.a.cols;
  const int64_t a_ld = j.a.ld;
  const bf16_t *pa = at.head(j.a), *na = pa;  // n: the next whole chunk's first token
  typedef Tile<bf16_t, D, A> TA;
  const TA ta(a_ld, a_cols, thread);
  typename TA::words wa[2];  // of chunk k in set k & 1
  auto any_a = [&](int k, auto set) {
    constexpr int S = decltype(set)::value;
    ta.load_any(wa[S], pa + at.token(k) * a_ld, a_ld, at.held(k), a_cols);
  };
  int at_a[KB], at_b[2 * KB];
#pragma unroll
  for (int R = 0; R < KB; ++R) {
    at_a[R] = A::row(R, lane);
    at_b[2 * R] = B::row(32 * R, lane);
    at_b[2 * R + 1] = B::row(32 * R + 16, lane);
  }
  // Scores transposed: rows j, columns p.  A wave's tiles share their operands: tokens' tiles t0
  // (and t0 + 1) by tiles j0 and j0 + 1; those above the diagonal are zeros.
  const int t0 = wave < 2 ? 2 : 3 - wave, j0 = wave == 1 ? 2 : 0;
  float weight[4][4];
  int keep = 0;  // a bit for each: on or below the diagonal
#pragma unroll
  for (int x = 0; x < 4; ++x)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int d = 16 * (t0 - j0 + x / 2 - x % 2) + l16 - 4 * g - i;
      keep |= (d >= 0 ? 1 : 0) << (4 * x + i);
      weight[x][i] = j.s * power(at.g2, max(d, 0));
    }
  auto scores_of = [&](const uint16_t* A_, const uint16_t* B_, half* P, auto tiles) {
    constexpr int NT = decltype(tiles)::value;
    A_ += 16 * t0 * D;
    B_ += 16 * j0 * D;
    f32x4 s[2 * NT] = {};
    frag fa[2][NT], fb[2][2];
    auto operands = [&](int R) {
#pragma unroll
      for (int x = 0; x < 2; ++x)
        fb[R & 1][x] = cat8(*reinterpret_cast<const u32x2*>(B_ + 16 * x * D + at_b[2 * R]), *reinterpret_cast<const u32x2*>(B_ + 16 * x * D + at_b[2 * R + 1]));
#pragma unroll
      for (int x = 0; x < NT; ++x) fa[R & 1][x] = as_bf16x8(*reinterpret_cast<const u32x4*>(A_ + 16 * x * D + at_a[R]));
    };
    operands(0);
#pragma unroll
    for (int R = 0; R < KB; ++R) {
      if (R + 1 < KB) operands(R + 1);
      __builtin_amdgcn_sched_barrier(0);  // ahead of these products
#pragma unroll
      for (int x = 0; x < 2 * NT; ++x) s[x] = O::mma(fb[R & 1][x % 2], fa[R & 1][x / 2], s[x]);
    }
#pragma unroll
    for (int x = 0; x < 2 * NT; ++x) {
      f32x4 v;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        v[i] = __builtin_bit_cast(float, __builtin_bit_cast(int, s[x][i] * weight[x][i]) & __builtin_amdgcn_sbfe(keep, 4 * x + i, 1));
      half o[NS];
      O::split<NS>(v, o);
#pragma unroll
      for (int q = 0; q < NS; ++q) P[((pair_of(t0 + x / 2, j0 / 2) * NS + q) * 64 + lane) * 2 + x % 2] = o[q];
    }
  };
  auto scores = [&](const uint16_t* A_, const uint16_t* B_, half* P) {
    if (wave < 2) scores_of(A_, B_, P, std::integral_constant<int, 2>());
    else scores_of(A_, B_, P, std::integral_constant<int, 1>());
  };
  // Outputs: a wave takes 16 tokens, 16 wave + l16, and all 64 columns of them: a lane's are 8 g..
  // and 32 + 8 g.., whole words of 16 bytes.
  const uint32_t out_row = uint32_t(plan.H) * uint32_t(j.c.cols);
  const int64_t out_head = int64_t(at.h) * j.c.cols + at.v0, out_token = int64_t(plan.H) * j.c.cols;
  const int out_size = out_f32 ? 4 : 2;
  int at_c[4];
#pragma unroll
  for (int ct = 0; ct < 4; ++ct) at_c[ct] = C::col(ct, lane);
  auto outputs = [&](int k, int nc, auto fast) {
    constexpr bool FAST = decltype(fast)::value;
    const half* P = sp(k & 1) + (pair_of(wave, 0) * NS * 64 + lane) * 2;
    const uint16_t* t = sc(k & 1);
    f32x4 acc[4];
    auto part = [&](int m) {
      frag fc[4], fp[NS];
#pragma unroll
      for (int ct = 0; ct < 4; ++ct) fc[ct] = column(t + at_c[ct], m);
#pragma unroll
      for (int q = 0; q < NS; ++q) fp[q] = *reinterpret_cast<const frag*>(P + (m * NS + q) * 128);
      if (m == 0) {
#pragma unroll
        for (int ct = 0; ct < 4; ++ct) acc[ct] = sx(k & 1)[(wave * 4 + ct) * 64 + lane];
      }
      __builtin_amdgcn_sched_barrier(0);  // all asked for ahead of the products
#pragma unroll
      for (int q = 0; q < NS; ++q)
#pragma unroll
        for (int ct = 0; ct < 4; ++ct) acc[ct] = O::mma(fc[ct], fp[q], acc[ct]);
    };
    part(0);
    if (wave >= 2) part(1);
    char* out = static_cast<char*>(j.out) + (at.token(k) * out_token + out_head) * out_size;
    const int p = 16 * wave + l16;
    const uint32_t first = uint32_t(rev ? nc - 1 - p : p) * out_row + 8 * g;
    if constexpr (FAST) {
      if (out_f32) {
#pragma unroll
        for (int ct = 0; ct < 4; ++ct) *reinterpret_cast<f32x4*>(out + (first + 32 * (ct >> 1) + 4 * (ct & 1)) * 4u) = acc[ct];
      } else {
#pragma unroll
        for (int x = 0; x < 2; ++x) {
          const u32x2 lo = pack4(acc[2 * x]), hi = pack4(acc[2 * x + 1]);
          *reinterpret_cast<u32x4*>(out + (first + 32 * x) * 2u) = u32x4{lo[0], lo[1], hi[0], hi[1]};
        }
      }
    } else if (p < nc) {
#pragma unroll
      for (int ct = 0; ct < 4; ++ct) {
        const int v = 32 * (ct >> 1) + 4 * (ct & 1), n = vc - 8 * g - v;
        if (n > 0) put4<bf16_t, false>(out_f32, out_words, out, first + v, acc[ct], n);
      }
    }
  };
  if (chunks > 0) {
    any_a(0, even);
    ta.store(wa[0], sa(0), at.held(0), a_cols, rev);
    if (chunks > 1) {
      any_a(1, odd);
      ta.store(wa[1], sa(1), at.held(1), a_cols, rev);
    }
    if (chunks > 2) any_a(2, even);
    if (chunks > 3) any_a(3, odd);
    __syncthreads();
    scores(sa(0), sb(0), sp(0));
  }
  int b1 = 1;  // b's tile of chunk k + 1
  if (quick > 4) na += at.token(4) * a_ld;
  auto turn = [&](int k, auto set, auto whole_chunks) {  // k & 1 = set
    constexpr int S = decltype(set)::value;
    constexpr bool FAST = decltype(whole_chunks)::value;
    __syncthreads();
    if constexpr (FAST) {
      ta.store_whole(wa[S], sa(S), a_cols, rev);
      ta.load(wa[S], na, a_ld);
      na += way * a_ld;
    } else {
      if (k + 2 < chunks) ta.store(wa[S], sa(S), at.held(k + 2), a_cols, rev);
      if (k + 4 < chunks) any_a(k + 4, set);
    }
    __builtin_amdgcn_sched_barrier(0);  // asked for now, not where the scheduler finds a register for them
    if (FAST || k + 1 < chunks) scores(sa(1 - S), sb(b1), sp(1 - S));
    outputs(k, at.held(k), whole_chunks);
    b1 = b1 == 2 ? 0 : b1 + 1;
  };
  int k = 0;
  for (; k + 5 < quick; k += 2) {
    turn(k, even, std::true_type{});
    turn(k + 1, odd, std::true_type{});
  }
  for (; k < chunks; k += 2) {
    turn(k, even, std::false_type{});
    if (k + 1 < chunks) turn(k + 1, odd, std::false_type{});
  }
}

template <int KB>
hipError_t launch_pair(const WalkPlan& p, hipStream_t s) {
  int64_t blocks = 0;
  for (int i = 0; i < p.jobs; ++i) blocks += int64_t(p.job[i].blocks) * p.Bt * p.H * p.segs;
  constexpr int bytes = PairLds<KB>::end;
  static std::atomic<uint64_t> cleared{0};
  const hipError_t e = allow_lds(reinterpret_cast<const void*>(&pair_kernel<KB>), bytes, cleared);
  if (e != hipSuccess) return e;
  pair_kernel<KB><<<dim3(uint32_t(blocks)), dim3(512), bytes, s>>>(p);
  return hipGetLastError();
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
      case 21: return launch<T, 2, 1, true>(p, s);
      case 41: return launch<T, 4, 1, true>(p, s);
      case 81: return launch<T, 8, 1, true>(p, s);
    }
  } else {
    if constexpr (sizeof(T) == 2) {
      switch (key) {
        case 11: return launch_pair<1>(p, s);
        case 21: return launch_pair<2>(p, s);
        case 41: return launch_pair<4>(p, s);
        case 81: return launch<T, 8, 1, false>(p, s);
      }
      return hipErrorInvalidValue;
    }
    if constexpr (sizeof(T) == 4) switch (key) {
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
