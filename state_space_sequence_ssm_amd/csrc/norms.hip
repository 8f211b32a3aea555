// Norms around a block: the gated group RMS norm behind the core and the
// residual RMS norm in front of the next block, forward and backward.
//
// Memory bound: every tensor is read and written once, the row (or group)
// staying in registers between its sums and its outputs.
#include "layer_internal.hpp"

namespace m3 {
namespace {

// How one unit (a row's group) is dealt to lanes: `team` lanes, each with NV
// words of V elements.  BLK = 0: teams of 2^lgteam <= 64 lanes inside waves,
// 256-thread blocks; BLK > 0: one block of BLK lanes per unit.  NV = 0: any
// width, columns walked in a loop and read twice.
//
// A team keeps its group and walks rows `walkers` apart: gains, and in the
// backward the sums of their gradients, stay in registers, and the next row is
// on its way while one is computed.  In all but the last turn every team has a
// row, so loads and stores have no branch around them (a branch would make each
// wait for a load wait for the stores as well).  Lanes past the width repeat the
// team's first word and leave the sums alone.
//
// Words are 16 bytes of T wherever a unit holds one, also where rows are not aligned
// to them or the width is no multiple (RAG): accesses then have the alignment of T, and
// the last word is moved back to end with the unit, its elements in the word before it
// left out of the sums and stored twice with the same value.  16384 rows of 2047 bf16,
// residual backward: 109 us, with one element per word 309 us.  Units of less than a word
// take one element per lane.
struct Geom {
  int V, nv, blk, lgteam;
};

// Sum over the unit's team, in every lane.
template <int BLK>
__device__ __forceinline__ float team_sum(float v, int lgteam, float* red) {
  if constexpr (BLK == 0) {
    if (lgteam >= 1) v += dpp<0xB1, 0xF, true>(v);   // lane ^ 1
    if (lgteam >= 2) v += dpp<0x4E, 0xF, true>(v);   // lane ^ 2
    if (lgteam >= 3) v += dpp<0x141, 0xF, true>(v);  // mirrored within 8
    if (lgteam >= 4) v += dpp<0x140, 0xF, true>(v);  // mirrored within 16
    if (lgteam >= 5) v = add_x16(v);
    if (lgteam >= 6) v = add_x32(v);
    return v;
  } else {
    v = wave_sum(v);
    if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
    __syncthreads();
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < BLK / 64; ++i) s += red[i];
    return s;
  }
}

// Two at once, with one barrier.
template <int BLK>
__device__ __forceinline__ void team_sum2(float& a, float& b, int lgteam, float (&red)[2][16]) {
  if constexpr (BLK == 0) {
    a = team_sum<0>(a, lgteam, nullptr);
    b = team_sum<0>(b, lgteam, nullptr);
  } else {
    a = wave_sum(a);
    b = wave_sum(b);
    if ((threadIdx.x & 63) == 0) {
      red[0][threadIdx.x >> 6] = a;
      red[1][threadIdx.x >> 6] = b;
    }
    __syncthreads();
    a = b = 0.f;
#pragma unroll
    for (int i = 0; i < BLK / 64; ++i) {
      a += red[0][i];
      b += red[1][i];
    }
  }
}

template <int BLK>
constexpr int threads() {
  return BLK == 0 ? 256 : BLK;
}

// Where a lane is: its team's first row and group, and its words' columns.
template <int V, int NV, int BLK, bool RAG>
struct Place {
  static constexpr int NR = NV > 0 ? NV : 1;
  int lane, team, g0, skip[NR];
  uint32_t c[NR];
  int64_t walker;
  bool in[NR];
  __device__ __forceinline__ Place(int lgteam, int G, int Dg) {
    team = BLK ? BLK : 1 << lgteam;
    const uint32_t slot = BLK ? blockIdx.x : (blockIdx.x * 256u + threadIdx.x) >> lgteam;
    lane = BLK ? int(threadIdx.x) : int(threadIdx.x) & (team - 1);
    walker = slot / uint32_t(G);
    g0 = int(slot % uint32_t(G)) * Dg;
#pragma unroll
    for (int i = 0; i < NR; ++i) {
      const int at = (i * team + lane) * V;
      in[i] = at < Dg;
      skip[i] = RAG && in[i] ? max(at + V - Dg, 0) : 0;
      c[i] = in[i] ? at - skip[i] : 0;
    }
  }
  // whether word i's element j is the sums' to take (a lane past the width drops its
  // sums as a whole)
  __device__ __forceinline__ bool counts(int i, int j) const { return !RAG || j >= skip[i]; }
};
// Element c of a row: a 32-bit offset, beside the row's address where the whole block
// shares it.
template <typename T>
__device__ __forceinline__ T* col(T* row, uint32_t c) {
  return reinterpret_cast<T*>(reinterpret_cast<uintptr_t>(row) + c * uint32_t(sizeof(T)));
}
// A gain's values at a word (1 without one), and at all of a lane's words.
template <int V, bool RAG>
__device__ __forceinline__ void gain_word(const float* w, uint32_t c, float (&o)[V]) {
  if (w != nullptr) {
    unpack<float, V>(load_word<float, V, RAG>(col(w, c)), o);
  } else {
#pragma unroll
    for (int j = 0; j < V; ++j) o[j] = 1.f;
  }
}
template <int V, int NR, bool RAG>
__device__ __forceinline__ void gain(const float* w, const uint32_t (&c)[NR], float (&o)[NR][V]) {
#pragma unroll
  for (int i = 0; i < NR; ++i) gain_word<V, RAG>(w, c[i], o[i]);
}

// Gated norm.  32768 rows of 2048 bf16 in 8 groups: 79 us, 5.1 TB/s.
struct GatedP {
  const void* x;
  const void* z;
  const float* w;
  void* y;
  int64_t xld, zld, M, walkers;
  int D, G, Dg, lgteam, gate_first;
  float eps, inv;
};

template <typename T, int V, int NV, int BLK, bool RAG>
__global__ __launch_bounds__(threads<BLK>()) void gated_kernel(GatedP p) {
  __shared__ float red[2][16];
  const Place<V, NV, BLK, RAG> at(p.lgteam, p.G, p.Dg);
  const T* x = static_cast<const T*>(p.x) + at.g0;
  const bool gated = p.z != nullptr, first = p.gate_first != 0;
  const T* z = gated ? static_cast<const T*>(p.z) + at.g0 : nullptr;
  T* y = static_cast<T*>(p.y) + at.g0;
  const float* w = p.w == nullptr ? nullptr : p.w + at.g0;
  const int64_t whole = p.M / p.walkers;
  if constexpr (NV > 0) {
    float wr[NV][V];
    gain<V, NV, RAG>(w, at.c, wr);
    Pack<T, V> qx[NV], qz[NV];
    auto fetch = [&](int64_t k) {
      int64_t row = at.walker + k * p.walkers;
      row = row < p.M ? row : p.M - 1;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        qx[i] = load_word<T, V, RAG>(col(x + row * p.xld, at.c[i]));
        if (gated) qz[i] = load_word<T, V, RAG>(col(z + row * p.zld, at.c[i]));
      }
    };
    auto turn = [&](int64_t k, bool last) {
      float v[NV][V], gate[NV][V];
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        unpack<T, V>(qx[i], v[i]);
        if (gated) {
          unpack<T, V>(qz[i], gate[i]);
#pragma unroll
          for (int j = 0; j < V; ++j) gate[i][j] = silu_f(gate[i][j]);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) gate[i][j] = 1.f;
        }
        if (first) {
#pragma unroll
          for (int j = 0; j < V; ++j) v[i][j] *= gate[i][j];
        }
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float u = at.counts(i, j) ? v[i][j] : 0.f;
          t = fmaf(u, u, t);
        }
        s += at.in[i] ? t : 0.f;
      }
      if (!last) fetch(k + 1);
      const float r = rsqrtf(team_sum<BLK>(s, p.lgteam, red[k & 1]) * p.inv + p.eps);
      const int64_t row = at.walker + k * p.walkers;
      if (last && row >= p.M) return;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float o[V];
        if (first) {
#pragma unroll
          for (int j = 0; j < V; ++j) o[j] = v[i][j] * r * wr[i][j];
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) o[j] = v[i][j] * r * wr[i][j] * gate[i][j];
        }
        store_word<T, V, RAG>(col(y + row * p.D, at.c[i]), o);
      }
    };
    fetch(0);
    for (int64_t k = 0; k < whole; ++k) turn(k, false);
    if (whole * p.walkers < p.M) turn(whole, true);
  } else {
    for (int64_t row = at.walker, k = 0; row < p.M; row += p.walkers, ++k) {
      const T* xr = x + row * p.xld;
      const T* zr = gated ? z + row * p.zld : nullptr;
      float s = 0.f;
      for (int c = at.lane; c < p.Dg; c += at.team) {
        float v = to_f32(xr[c]);
        if (first && gated) v *= silu_f(to_f32(zr[c]));
        s = fmaf(v, v, s);
      }
      const float r = rsqrtf(team_sum<BLK>(s, p.lgteam, red[k & 1]) * p.inv + p.eps);
      for (int c = at.lane; c < p.Dg; c += at.team) {
        const float gate = gated ? silu_f(to_f32(zr[c])) : 1.f;
        from_f32(to_f32(xr[c]) * gate * r * (w != nullptr ? w[c] : 1.f), y[row * p.D + c]);
      }
    }
  }
}

// The widest units of the backward, blocks of 1024 lanes with 128 registers each, read
// gains from the cache in every row and the row when its turn comes.
template <int BLK>
constexpr bool lean() {
  return BLK == 1024;
}

// Makes the compiler take a word's values from the word again, instead of keeping them
// as floats (twice the registers, for bf16) from one pass over a row to the next.
template <typename T, int V>
__device__ __forceinline__ void afresh(Pack<T, V>& q) {
  static_assert(sizeof(q) % 4 == 0, "whole dwords");
#pragma unroll
  for (int i = 0; i < int(sizeof(q) / 4); ++i) {
    uint32_t w;
    __builtin_memcpy(&w, reinterpret_cast<char*>(&q) + 4 * i, 4);
    asm volatile("" : "+v"(w));
    __builtin_memcpy(reinterpret_cast<char*>(&q) + 4 * i, &w, 4);
  }
}

struct GatedBwP {
  const void* x;
  const void* z;
  const float* w;
  const void* dy;
  void* dx;
  void* dz;
  float* part;  // [walkers][D] sums of dw, or null
  int64_t xld, zld, M, walkers;
  int D, G, Dg, lgteam, gate_first;
  float eps, inv;
};

// With v = x silu(z) (or x), n = v r, r = rsqrt(mean(v^2) + eps), u = dy (or dy
// silu(z)) and e = u w:  dv = r (e - n mean(e n)), dw = sum u n.  Both sums of
// a row, v^2 and e v, are known before its outputs are formed.  32768 rows of 2048
// bf16 in 8 groups: 130 us, 5.2 TB/s, and 5 us for the join of dw.
template <typename T, int V, int NV, int BLK, bool RAG>
__global__ __launch_bounds__(threads<BLK>()) void gated_backward_kernel(GatedBwP p) {
  __shared__ float red[2][2][16];
  const Place<V, NV, BLK, RAG> at(p.lgteam, p.G, p.Dg);
  const bool first = p.gate_first != 0, gated = p.z != nullptr;
  const T* x = static_cast<const T*>(p.x) + at.g0;
  const T* z = gated ? static_cast<const T*>(p.z) + at.g0 : nullptr;
  const T* dy = static_cast<const T*>(p.dy) + at.g0;
  T* dx = static_cast<T*>(p.dx) + at.g0;
  T* dz = gated ? static_cast<T*>(p.dz) + at.g0 : nullptr;
  const float* w = p.w == nullptr ? nullptr : p.w + at.g0;
  float* part = p.part == nullptr ? nullptr : p.part + at.walker * p.D + at.g0;
  const int64_t whole = p.M / p.walkers;
  if constexpr (NV > 0) {
    float dw[NV][V], wr[NV][V];
    if constexpr (!lean<BLK>()) gain<V, NV, RAG>(w, at.c, wr);
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) dw[i][j] = 0.f;
    Pack<T, V> qx[NV], qz[NV], qd[NV];
    auto fetch = [&](int64_t k) {
      int64_t row = at.walker + k * p.walkers;
      row = row < p.M ? row : p.M - 1;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        qx[i] = load_word<T, V, RAG>(col(x + row * p.xld, at.c[i]));
        qd[i] = load_word<T, V, RAG>(col(dy + row * p.D, at.c[i]));
        if (gated) qz[i] = load_word<T, V, RAG>(col(z + row * p.zld, at.c[i]));
      }
    };
    auto turn = [&](int64_t k, bool last) {
      if constexpr (lean<BLK>()) fetch(k);
      float xv[NV][V], zv[NV][V], d[NV][V], sg[NV][V];
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        unpack<T, V>(qx[i], xv[i]);
        unpack<T, V>(qd[i], d[i]);
        if (gated) {
          unpack<T, V>(qz[i], zv[i]);
#pragma unroll
          for (int j = 0; j < V; ++j) sg[i][j] = sigmoid_f(zv[i][j]);
        } else {
#pragma unroll
          for (int j = 0; j < V; ++j) zv[i][j] = sg[i][j] = 1.f;
        }
        float t1 = 0.f, t2 = 0.f;
        if constexpr (lean<BLK>()) gain_word<V, RAG>(w, at.c[i], wr[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float gate = zv[i][j] * sg[i][j];
          const float e = d[i][j] * wr[i][j];
          const float v = at.counts(i, j) ? (first ? xv[i][j] * gate : xv[i][j]) : 0.f;
          const float ev = at.counts(i, j) ? (first ? e : e * gate) : 0.f;
          t1 = fmaf(v, v, t1);
          t2 = fmaf(ev, v, t2);
        }
        s1 += at.in[i] ? t1 : 0.f;
        s2 += at.in[i] ? t2 : 0.f;
      }
      if (!lean<BLK>() && !last) fetch(k + 1);
      team_sum2<BLK>(s1, s2, p.lgteam, red[k & 1]);
      const float r = rsqrtf(s1 * p.inv + p.eps), m = s2 * r * p.inv;
      const int64_t row = at.walker + k * p.walkers;
      if (last && row >= p.M) return;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float ox[V], oz[V];
        if constexpr (lean<BLK>()) {
          gain_word<V, RAG>(w, at.c[i], wr[i]);
          afresh(qx[i]);
          afresh(qd[i]);
          unpack<T, V>(qx[i], xv[i]);
          unpack<T, V>(qd[i], d[i]);
          if (gated) {
            afresh(qz[i]);
            unpack<T, V>(qz[i], zv[i]);
#pragma unroll
            for (int j = 0; j < V; ++j) sg[i][j] = sigmoid_f(zv[i][j]);
          }
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float gate = zv[i][j] * sg[i][j];
          const float n = (first ? xv[i][j] * gate : xv[i][j]) * r;
          const float u = first ? d[i][j] : d[i][j] * gate;
          const float dv = r * (u * wr[i][j] - n * m);
          ox[j] = first ? dv * gate : dv;
          oz[j] = (first ? dv * xv[i][j] : d[i][j] * n * wr[i][j]) * dsilu_f(zv[i][j], sg[i][j]);
          dw[i][j] = fmaf(u, n, dw[i][j]);
        }
        store_word<T, V, RAG>(col(dx + row * p.D, at.c[i]), ox);
        if (gated) store_word<T, V, RAG>(col(dz + row * p.D, at.c[i]), oz);
      }
    };
    if constexpr (!lean<BLK>()) fetch(0);
    for (int64_t k = 0; k < whole; ++k) turn(k, false);
    if (whole * p.walkers < p.M) turn(whole, true);
    if (part == nullptr) return;
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (at.in[i]) store_word<float, V, RAG>(col(part, at.c[i]), dw[i]);
  } else {
    if (part != nullptr)
      for (int c = at.lane; c < p.Dg; c += at.team) part[c] = 0.f;
    for (int64_t row = at.walker, k = 0; row < p.M; row += p.walkers, ++k) {
      const T* xr = x + row * p.xld;
      const T* zr = gated ? z + row * p.zld : nullptr;
      const T* dr = dy + row * p.D;
      float s1 = 0.f, s2 = 0.f;
      for (int c = at.lane; c < p.Dg; c += at.team) {
        const float gate = gated ? silu_f(to_f32(zr[c])) : 1.f;
        const float xv = to_f32(xr[c]), e = to_f32(dr[c]) * (w != nullptr ? w[c] : 1.f);
        const float v = first ? xv * gate : xv;
        s1 = fmaf(v, v, s1);
        s2 = fmaf(first ? e : e * gate, v, s2);
      }
      team_sum2<BLK>(s1, s2, p.lgteam, red[k & 1]);
      const float r = rsqrtf(s1 * p.inv + p.eps), m = s2 * r * p.inv;
      for (int c = at.lane; c < p.Dg; c += at.team) {
        const float zv = gated ? to_f32(zr[c]) : 1.f, xv = to_f32(xr[c]), d = to_f32(dr[c]);
        const float sg = gated ? sigmoid_f(zv) : 1.f, gate = zv * sg, wc = w != nullptr ? w[c] : 1.f;
        const float n = (first ? xv * gate : xv) * r;
        const float u = first ? d : d * gate;
        const float dv = r * (u * wc - n * m);
        from_f32(first ? dv * gate : dv, dx[row * p.D + c]);
        if (gated) from_f32((first ? dv * xv : d * n * wc) * dsilu_f(zv, sg), dz[row * p.D + c]);
        if (part != nullptr) part[c] = fmaf(u, n, part[c]);
      }
    }
  }
}

// Residual norm.  256 rows of 2048, fp32 stream: 3.6 us.
struct ResP {
  const void* x;
  const void* res;
  const float* scale;
  const float* w;
  void* y;
  void* res_out;
  int64_t xld, M, walkers;
  int D, lgteam;
  float eps, inv;
};

template <typename T, typename R, int V, int NV, int BLK, bool RAG>
__global__ __launch_bounds__(threads<BLK>()) void residual_kernel(ResP p) {
  __shared__ float red[2][16];
  const Place<V, NV, BLK, RAG> at(p.lgteam, 1, p.D);
  const T* x = static_cast<const T*>(p.x);
  const R* res = static_cast<const R*>(p.res);
  R* out = static_cast<R*>(p.res_out);
  T* y = static_cast<T*>(p.y);
  const int64_t whole = p.M / p.walkers;
  if constexpr (NV > 0) {
    Pack<T, V> qx[NV];
    Pack<R, V> qr[NV];
    auto fetch = [&](int64_t k) {
      int64_t row = at.walker + k * p.walkers;
      row = row < p.M ? row : p.M - 1;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        qx[i] = load_word<T, V, RAG>(col(x + row * p.xld, at.c[i]));
        if (res != nullptr) qr[i] = load_word<R, V, RAG>(col(res + row * p.D, at.c[i]));
        else qr[i] = Pack<R, V>{};
      }
    };
    fetch(0);
    float wr[NV][V], sr[NV][V];
    gain<V, NV, RAG>(p.w, at.c, wr);
    gain<V, NV, RAG>(p.scale, at.c, sr);
    auto turn = [&](int64_t k, bool last) {
      float h[NV][V];
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float t = 0.f;
#pragma unroll
        for (int j = 0; j < V; ++j) {
          h[i][j] = fmaf(sr[i][j], to_f32(qx[i].e[j]), to_f32(qr[i].e[j]));
          const float u = at.counts(i, j) ? h[i][j] : 0.f;
          t = fmaf(u, u, t);
        }
        s += at.in[i] ? t : 0.f;
      }
      if (!last) fetch(k + 1);
      const float r = rsqrtf(team_sum<BLK>(s, p.lgteam, red[k & 1]) * p.inv + p.eps);
      const int64_t row = at.walker + k * p.walkers;
      if (last && row >= p.M) return;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float o[V];
        if (out != nullptr) store_word<R, V, RAG>(col(out + row * p.D, at.c[i]), h[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) o[j] = h[i][j] * r * wr[i][j];
        store_word<T, V, RAG>(col(y + row * p.D, at.c[i]), o);
      }
    };
    for (int64_t k = 0; k < whole; ++k) turn(k, false);
    if (whole * p.walkers < p.M) turn(whole, true);
  } else {
    for (int64_t row = at.walker, k = 0; row < p.M; row += p.walkers, ++k) {
      auto sum = [&](int c) {
        return fmaf(p.scale != nullptr ? p.scale[c] : 1.f, to_f32(x[row * p.xld + c]),
                    res != nullptr ? to_f32(res[row * p.D + c]) : 0.f);
      };
      float s = 0.f;
      for (int c = at.lane; c < p.D; c += at.team) {
        const float h = sum(c);
        s = fmaf(h, h, s);
      }
      const float r = rsqrtf(team_sum<BLK>(s, p.lgteam, red[k & 1]) * p.inv + p.eps);
      for (int c = at.lane; c < p.D; c += at.team) {
        const float h = sum(c);
        if (out != nullptr) from_f32(h, out[row * p.D + c]);
        from_f32(h * r * (p.w != nullptr ? p.w[c] : 1.f), y[row * p.D + c]);
      }
    }
  }
}

struct ResBwP {
  const void* h;
  const void* x;
  const float* scale;
  const float* w;
  const void* dy;
  const void* dro;
  void* dx;
  void* dres;
  float* part;  // [walkers][2][D]: sums of dw and dscale (or [walkers][D] with one of them), or null
  int64_t xld, M, walkers;
  int D, lgteam, has_dw, has_ds;
  float eps, inv;
};

// n = h r, e = dy w:  dh = dro + r (e - n mean(e n)), dw = sum dy n, dscale =
// sum dh x; rows walked as in the gated norm's backward.  32768 rows of 2048 bf16:
// 157 us, 5.1 TB/s, and 7 us for the joins.
template <typename T, typename R, int V, int NV, int BLK, bool RAG>
__global__ __launch_bounds__(threads<BLK>()) void residual_backward_kernel(ResBwP p) {
  __shared__ float red[2][2][16];
  const Place<V, NV, BLK, RAG> at(p.lgteam, 1, p.D);
  float* prow = p.part + at.walker * (p.has_dw + p.has_ds) * p.D;
  float* pw = p.has_dw ? prow : nullptr;
  float* ps = p.has_ds ? prow + (p.has_dw ? p.D : 0) : nullptr;
  const R* h = static_cast<const R*>(p.h);
  const T* x = static_cast<const T*>(p.x);
  const T* dy = static_cast<const T*>(p.dy);
  const R* dro = static_cast<const R*>(p.dro);
  T* dx = static_cast<T*>(p.dx);
  R* dres = static_cast<R*>(p.dres);
  const int64_t whole = p.M / p.walkers;
  if constexpr (NV > 0) {
    Pack<R, V> qh[NV], qr[NV];
    Pack<T, V> qd[NV], qx[NV];
    auto fetch = [&](int64_t k) {
      int64_t row = at.walker + k * p.walkers;
      row = row < p.M ? row : p.M - 1;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        qh[i] = load_word<R, V, RAG>(col(h + row * p.D, at.c[i]));
        qd[i] = load_word<T, V, RAG>(col(dy + row * p.D, at.c[i]));
        if (dro != nullptr) qr[i] = load_word<R, V, RAG>(col(dro + row * p.D, at.c[i]));
        else qr[i] = Pack<R, V>{};
        if (p.has_ds) qx[i] = load_word<T, V, RAG>(col(x + row * p.xld, at.c[i]));
        else qx[i] = Pack<T, V>{};
      }
    };
    if constexpr (!lean<BLK>()) fetch(0);
    float dw[NV][V], ds[NV][V], wr[NV][V], sr[NV][V];
    if constexpr (!lean<BLK>()) {
      gain<V, NV, RAG>(p.w, at.c, wr);
      gain<V, NV, RAG>(p.scale, at.c, sr);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) dw[i][j] = ds[i][j] = 0.f;
    auto turn = [&](int64_t k, bool last) {
      if constexpr (lean<BLK>()) fetch(k);
      // the row as it came, so that it takes half the registers
      Pack<R, V> ch[NV], cr[NV];
      Pack<T, V> cd[NV], cx[NV];
      float s1 = 0.f, s2 = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        ch[i] = qh[i];
        cr[i] = qr[i];
        cd[i] = qd[i];
        cx[i] = qx[i];
        float t1 = 0.f, t2 = 0.f;
        if constexpr (lean<BLK>()) gain_word<V, RAG>(p.w, at.c[i], wr[i]);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float hv = at.counts(i, j) ? to_f32(ch[i].e[j]) : 0.f;
          const float e = at.counts(i, j) ? to_f32(cd[i].e[j]) * wr[i][j] : 0.f;
          t1 = fmaf(hv, hv, t1);
          t2 = fmaf(e, hv, t2);
        }
        s1 += at.in[i] ? t1 : 0.f;
        s2 += at.in[i] ? t2 : 0.f;
      }
      if (!lean<BLK>() && !last) fetch(k + 1);
      team_sum2<BLK>(s1, s2, p.lgteam, red[k & 1]);
      const float r = rsqrtf(s1 * p.inv + p.eps), m = s2 * r * p.inv;
      const int64_t row = at.walker + k * p.walkers;
      if (last && row >= p.M) return;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float o[V], ox[V];
        if constexpr (lean<BLK>()) {
          gain_word<V, RAG>(p.w, at.c[i], wr[i]);
          gain_word<V, RAG>(p.scale, at.c[i], sr[i]);
          afresh(ch[i]);
          afresh(cd[i]);
        }
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float n = to_f32(ch[i].e[j]) * r, d = to_f32(cd[i].e[j]);
          o[j] = to_f32(cr[i].e[j]) + r * (d * wr[i][j] - n * m);
          ox[j] = sr[i][j] * o[j];
          dw[i][j] = fmaf(d, n, dw[i][j]);
          ds[i][j] = fmaf(o[j], to_f32(cx[i].e[j]), ds[i][j]);
        }
        if (dres != nullptr) store_word<R, V, RAG>(col(dres + row * p.D, at.c[i]), o);
        if (dx != nullptr) store_word<T, V, RAG>(col(dx + row * p.D, at.c[i]), ox);
      }
    };
    for (int64_t k = 0; k < whole; ++k) turn(k, false);
    if (whole * p.walkers < p.M) turn(whole, true);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (!at.in[i]) continue;
      if (pw != nullptr) store_word<float, V, RAG>(col(pw, at.c[i]), dw[i]);
      if (ps != nullptr) store_word<float, V, RAG>(col(ps, at.c[i]), ds[i]);
    }
  } else {
    for (int c = at.lane; c < p.D; c += at.team) {
      if (pw != nullptr) pw[c] = 0.f;
      if (ps != nullptr) ps[c] = 0.f;
    }
    for (int64_t row = at.walker, k = 0; row < p.M; row += p.walkers, ++k) {
      const int64_t r0 = row * p.D;
      float s1 = 0.f, s2 = 0.f;
      for (int c = at.lane; c < p.D; c += at.team) {
        const float hv = to_f32(h[r0 + c]);
        s1 = fmaf(hv, hv, s1);
        s2 = fmaf(to_f32(dy[r0 + c]) * (p.w != nullptr ? p.w[c] : 1.f), hv, s2);
      }
      team_sum2<BLK>(s1, s2, p.lgteam, red[k & 1]);
      const float r = rsqrtf(s1 * p.inv + p.eps), m = s2 * r * p.inv;
      for (int c = at.lane; c < p.D; c += at.team) {
        const float n = to_f32(h[r0 + c]) * r, d = to_f32(dy[r0 + c]);
        const float o = (dro != nullptr ? to_f32(dro[r0 + c]) : 0.f) + r * (d * (p.w != nullptr ? p.w[c] : 1.f) - n * m);
        if (dres != nullptr) from_f32(o, dres[r0 + c]);
        if (dx != nullptr) from_f32((p.scale != nullptr ? p.scale[c] : 1.f) * o, dx[r0 + c]);
        if (pw != nullptr) pw[c] = fmaf(d, n, pw[c]);
        if (ps != nullptr) ps[c] = fmaf(o, to_f32(x[row * p.xld + c]), ps[c]);
      }
    }
  }
}

// Lanes for a unit of `width` elements: a part of a wave up to 64 words, wider
// ones over several words per lane or several waves, the loop for what a block
// does not hold in registers (over 2048 words: 16384 bf16 values, 8192 fp32).
// Forward, a unit of 65 to 256 words is one wave's where the units
// fill the card (2048 or more) and a block's otherwise.  The backward holds four
// times the registers per word and takes a block at once: 32768 rows of 2048 bf16
// take 159 us with one word per lane of four waves, and 216 us with four words per
// lane of one wave (216 registers).  Its widest units spill some of them: 4096 rows of
// 8192 fp32 take 135 us gated and 164 us residual, in the loop 310 and 428 us; of
// 16384 bf16 255 and 317 us, in the loop 583 and 777 us.
Geom pick(int64_t units, int width, int in_dtype, bool backward) {
  const int whole = in_dtype == M3_BF16 ? 8 : 4, V = width >= whole ? whole : 1;
  Geom g{V, 1, 0, 6};
  const int64_t words = (int64_t(width) + V - 1) / V;
  if (words <= 64) {
    g.lgteam = 0;
    while ((1 << g.lgteam) < words) ++g.lgteam;
  } else if (words <= 256 && units >= 2048 && !backward) {
    g.nv = words <= 128 ? 2 : 4;
  } else if (words <= 512) {
    g.blk = 256;
    g.nv = words <= 256 ? 1 : 2;
  } else if (words <= 1024) {
    g.blk = backward ? 512 : 256;
    g.nv = backward ? 2 : 4;
  } else if (words <= 2048) {
    g.blk = 1024;
    g.nv = 2;
  } else {
    g.V = 1;
    g.blk = 1024;
    g.nv = 0;
  }
  return g;
}

// Teams of a group, each walking rows that far apart: `waves` waves in all on the
// card's 1024 SIMDs, whole blocks of teams, at most one team per row (rounded up to
// a block's worth).
int64_t pick_walkers(int64_t M, int G, const Geom& g, int64_t waves) {
  const int64_t lanes = g.blk ? g.blk : int64_t(1) << g.lgteam;
  const int64_t per = g.blk ? 1 : 256 >> g.lgteam;  // teams of a block
  int64_t w = waves * 64 / (lanes * G);
  if (w > M) w = M;
  if (w < 1) w = 1;
  return (w + per - 1) / per * per;
}
constexpr int64_t kForwardWaves = 8192, kBackwardWaves = 4096;

// The kernel instance for a geometry: CALL(V, NV, BLK, RAG).
#define M3_NORM_WIDTH(g, V, RAG, CALL)            \
  if ((g).blk == 0) {                             \
    if ((g).nv == 1) return CALL(V, 1, 0, RAG);   \
    if ((g).nv == 2) return CALL(V, 2, 0, RAG);   \
    return CALL(V, 4, 0, RAG);                    \
  }                                               \
  if ((g).blk == 1024) return CALL(V, 2, 1024, RAG); \
  if ((g).nv == 1) return CALL(V, 1, 256, RAG);   \
  if ((g).nv == 2) return CALL(V, 2, 256, RAG);   \
  return CALL(V, 4, 256, RAG);
#define M3_NORM_BACKWARD_WIDTH(g, V, RAG, CALL)   \
  if ((g).blk == 0) return CALL(V, 1, 0, RAG);    \
  if ((g).blk == 512) return CALL(V, 2, 512, RAG); \
  if ((g).blk == 1024) return CALL(V, 2, 1024, RAG); \
  if ((g).nv == 1) return CALL(V, 1, 256, RAG);   \
  return CALL(V, 2, 256, RAG);
#define M3_NORM_DISPATCH(g, vec, VV, WIDTH, CALL) \
  if ((g).nv == 0) return CALL(1, 0, 1024, false); \
  if ((g).V == 1) return CALL(1, 1, 0, false);    \
  if (vec) {                                      \
    WIDTH(g, VV, false, CALL)                     \
  }                                               \
  WIDTH(g, VV, true, CALL)

uint32_t grid_of(const Geom& g, int64_t teams) { return uint32_t(g.blk ? teams : (teams << g.lgteam) / 256); }
bool gain_aligned(const float* w) { return reinterpret_cast<uintptr_t>(w) % 16 == 0; }

template <typename T>
hipError_t run_gated(const m3_gated_norm_args& a, hipStream_t s) {
  constexpr int VV = 16 / int(sizeof(T));
  const int Dg = a.D / a.G;
  const bool vec = Dg % VV == 0 && rows_aligned(a.x, a.x_ld, sizeof(T), 16) && rows_aligned(a.z, a.z_ld, sizeof(T), 16) &&
                   rows_aligned(a.y, a.D, sizeof(T), 16) && gain_aligned(a.w);
  const Geom g = pick(a.M * a.G, Dg, a.in_dtype, false);
  const GatedP p{a.x, a.z, a.w, a.y, a.x_ld, a.z_ld, a.M, pick_walkers(a.M, a.G, g, kForwardWaves), a.D, a.G, Dg, g.lgteam, a.gate_first, a.eps, 1.f / float(Dg)};
#define CALL(V, NV, BLK, RAG) (gated_kernel<T, V, NV, BLK, RAG><<<grid_of(g, p.walkers * p.G), threads<BLK>(), 0, s>>>(p), hipGetLastError())
  M3_NORM_DISPATCH(g, vec, VV, M3_NORM_WIDTH, CALL)
#undef CALL
}

template <typename T>
bool gated_bw_vec(const m3_gated_norm_backward_args& a) {
  constexpr int VV = 16 / int(sizeof(T));
  const m3_gated_norm_args& f = a.fwd;
  return (f.D / f.G) % VV == 0 && rows_aligned(f.x, f.x_ld, sizeof(T), 16) && rows_aligned(f.z, f.z_ld, sizeof(T), 16) &&
         rows_aligned(a.dy, f.D, sizeof(T), 16) && rows_aligned(a.dx, f.D, sizeof(T), 16) &&
         rows_aligned(a.dz, f.D, sizeof(T), 16) && gain_aligned(f.w);
}
template <typename T>
hipError_t launch_gated_bw(const GatedBwP& p, const Geom& g, bool vec, hipStream_t s) {
  constexpr int VV = 16 / int(sizeof(T));
#define CALL(V, NV, BLK, RAG) \
  (gated_backward_kernel<T, V, NV, BLK, RAG><<<grid_of(g, p.walkers * p.G), threads<BLK>(), 0, s>>>(p), hipGetLastError())
  M3_NORM_DISPATCH(g, vec, VV, M3_NORM_BACKWARD_WIDTH, CALL)
#undef CALL
}
template <typename T>
hipError_t run_gated_bw(const m3_gated_norm_backward_args& a, hipStream_t s) {
  const m3_gated_norm_args& f = a.fwd;
  const int Dg = f.D / f.G;
  const Geom g = pick(f.M * f.G, Dg, f.in_dtype, true);
  const GatedBwP p{f.x, f.z, f.w, a.dy, a.dx, a.dz, f.w != nullptr ? static_cast<float*>(a.workspace) : nullptr, f.x_ld, f.z_ld,
                   f.M, pick_walkers(f.M, f.G, g, kBackwardWaves), f.D, f.G, Dg, g.lgteam, f.gate_first, f.eps, 1.f / float(Dg)};
  const hipError_t e = launch_gated_bw<T>(p, g, gated_bw_vec<T>(a), s);
  if (e != hipSuccess || f.w == nullptr) return e;
  ColSum c{};
  c.part = p.part;
  c.P = p.walkers;
  c.ncols = f.D;
  c.dst[0] = a.dw;
  c.n[0] = f.D;
  return launch_colsum(c, s);
}

template <typename T, typename R>
hipError_t run_residual(const m3_residual_norm_args& a, hipStream_t s) {
  constexpr int VV = 16 / int(sizeof(T));
  const bool vec = a.D % VV == 0 && rows_aligned(a.x, a.x_ld, sizeof(T), 16) && rows_aligned(a.y, a.D, sizeof(T), 16) &&
                   rows_aligned(a.residual, a.D, sizeof(R), 16) && rows_aligned(a.residual_out, a.D, sizeof(R), 16) && gain_aligned(a.w) &&
                   gain_aligned(a.scale);
  const Geom g = pick(a.M, a.D, a.in_dtype, false);
  const ResP p{a.x, a.residual, a.scale, a.w, a.y, a.residual_out, a.x_ld, a.M, pick_walkers(a.M, 1, g, kForwardWaves),
               a.D, g.lgteam, a.eps, 1.f / float(a.D)};
#define CALL(V, NV, BLK, RAG) (residual_kernel<T, R, V, NV, BLK, RAG><<<grid_of(g, p.walkers), threads<BLK>(), 0, s>>>(p), hipGetLastError())
  M3_NORM_DISPATCH(g, vec, VV, M3_NORM_WIDTH, CALL)
#undef CALL
}
template <typename T, typename R>
hipError_t launch_residual_bw(const ResBwP& p, const Geom& g, bool vec, hipStream_t s) {
  constexpr int VV = 16 / int(sizeof(T));
#define CALL(V, NV, BLK, RAG) \
  (residual_backward_kernel<T, R, V, NV, BLK, RAG><<<grid_of(g, p.walkers), threads<BLK>(), 0, s>>>(p), hipGetLastError())
  M3_NORM_DISPATCH(g, vec, VV, M3_NORM_BACKWARD_WIDTH, CALL)
#undef CALL
}
template <typename T, typename R>
hipError_t run_residual_bw(const m3_residual_norm_backward_args& a, hipStream_t s) {
  constexpr int VV = 16 / int(sizeof(T));
  const bool vec = a.D % VV == 0 && rows_aligned(a.x, a.x_ld, sizeof(T), 16) && rows_aligned(a.dy, a.D, sizeof(T), 16) &&
                   rows_aligned(a.dx, a.D, sizeof(T), 16) && rows_aligned(a.h, a.D, sizeof(R), 16) &&
                   rows_aligned(a.dresidual_out, a.D, sizeof(R), 16) && rows_aligned(a.dresidual, a.D, sizeof(R), 16) && gain_aligned(a.w) && gain_aligned(a.scale);
  const Geom g = pick(a.M, a.D, a.in_dtype, true);
  const ResBwP p{a.h, a.x, a.scale, a.w, a.dy, a.dresidual_out, a.dx, a.dresidual, static_cast<float*>(a.workspace), a.x_ld, a.M,
                 pick_walkers(a.M, 1, g, kBackwardWaves), a.D, g.lgteam, a.w != nullptr, a.scale != nullptr, a.eps, 1.f / float(a.D)};
  const hipError_t e = launch_residual_bw<T, R>(p, g, vec, s);
  if (e != hipSuccess || (a.w == nullptr && a.scale == nullptr)) return e;
  ColSum c{};
  c.part = p.part;
  c.P = p.walkers;
  c.ncols = int64_t(p.has_dw + p.has_ds) * a.D;
  if (p.has_dw) c.dst[0] = a.dw, c.n[0] = a.D;
  if (p.has_ds) c.dst[1] = a.dscale, c.n[1] = a.D;
  return launch_colsum(c, s);
}

}  // namespace

hipError_t launch_gated_norm(const m3_gated_norm_args& a, hipStream_t s) {
  return a.in_dtype == M3_BF16 ? run_gated<bf16_t>(a, s) : run_gated<float>(a, s);
}
static int64_t gated_bw_walkers(const m3_gated_norm_args& f) {
  return pick_walkers(f.M, f.G, pick(f.M * f.G, f.D / f.G, f.in_dtype, true), kBackwardWaves);
}
bool gated_norm_backward_fits(const m3_gated_norm_backward_args& a) {
  return a.fwd.w == nullptr || launchable(colsum_blocks(gated_bw_walkers(a.fwd), a.fwd.D), 1024);
}
size_t gated_norm_backward_workspace(const m3_gated_norm_backward_args& a) {
  return a.fwd.w == nullptr ? 0 : round256(size_t(gated_bw_walkers(a.fwd)) * a.fwd.D * 4);
}
hipError_t launch_gated_norm_backward(const m3_gated_norm_backward_args& a, hipStream_t s) {
  return a.fwd.in_dtype == M3_BF16 ? run_gated_bw<bf16_t>(a, s) : run_gated_bw<float>(a, s);
}
hipError_t launch_residual_norm(const m3_residual_norm_args& a, hipStream_t s) {
  if (a.in_dtype == M3_F32) return run_residual<float, float>(a, s);
  return a.res_dtype == M3_BF16 ? run_residual<bf16_t, bf16_t>(a, s) : run_residual<bf16_t, float>(a, s);
}
static int64_t residual_bw_walkers(const m3_residual_norm_backward_args& a) {
  return pick_walkers(a.M, 1, pick(a.M, a.D, a.in_dtype, true), kBackwardWaves);
}
bool residual_norm_backward_fits(const m3_residual_norm_backward_args& a) {
  const int64_t ncols = int64_t((a.w != nullptr) + (a.scale != nullptr)) * a.D;
  return launchable(colsum_blocks(residual_bw_walkers(a), ncols), 1024);
}
size_t residual_norm_backward_workspace(const m3_residual_norm_backward_args& a) {
  return round256(size_t(residual_bw_walkers(a)) * ((a.w != nullptr) + (a.scale != nullptr)) * a.D * 4);
}
hipError_t launch_residual_norm_backward(const m3_residual_norm_backward_args& a, hipStream_t s) {
  if (a.in_dtype == M3_F32) return run_residual_bw<float, float>(a, s);
  return a.res_dtype == M3_BF16 ? run_residual_bw<bf16_t, bf16_t>(a, s) : run_residual_bw<bf16_t, float>(a, s);
}

}  // namespace m3
