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
struct Geom {
  bool vec;
  int nv, blk, lgteam;
};

// Sum over the unit's team, in every lane.
template <int BLK>
__device__ __forceinline__ float team_sum(float v, int lgteam, float* red) {
  if constexpr (BLK == 0) {
    if (lgteam == 6) return wave_sum(v);
    for (int m = 1; m < (1 << lgteam); m <<= 1) v += __shfl_xor(v, m);
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

template <int BLK>
constexpr int threads() {
  return BLK == 0 ? 256 : BLK;
}

template <int BLK>
__device__ __forceinline__ int64_t team_index(int lgteam) {
  if constexpr (BLK == 0) return (int64_t(blockIdx.x) * 256 + threadIdx.x) >> lgteam;
  return blockIdx.x;
}
template <int BLK>
__device__ __forceinline__ int team_lane(int lgteam) {
  if constexpr (BLK == 0) return int(threadIdx.x) & ((1 << lgteam) - 1);
  return int(threadIdx.x);
}

struct GatedP {
  const void* x;
  const void* z;
  const float* w;
  void* y;
  int64_t xld, zld, units;
  int D, G, Dg, lgteam, gate_first;
  float eps, inv;
};

template <typename T, int V, int NV, int BLK>
__global__ __launch_bounds__(threads<BLK>()) void gated_kernel(GatedP p) {
  __shared__ float red[16];
  const int64_t unit = team_index<BLK>(p.lgteam);
  const int lane = team_lane<BLK>(p.lgteam), team = BLK ? BLK : 1 << p.lgteam;
  const bool live = unit < p.units;
  const int64_t row = live ? unit / p.G : 0;
  const int g0 = live ? int(unit - row * p.G) * p.Dg : 0;
  const T* x = static_cast<const T*>(p.x) + row * p.xld + g0;
  const T* z = p.z == nullptr ? nullptr : static_cast<const T*>(p.z) + row * p.zld + g0;
  T* y = static_cast<T*>(p.y) + row * p.D + g0;
  const float* w = p.w == nullptr ? nullptr : p.w + g0;
  const bool first = p.gate_first != 0;
  if constexpr (NV > 0) {
    float v[NV][V], gate[NV][V];
    float s = 0.f;
    Pack<T, V> qx[NV], qz[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * team + lane) * V;
      qx[i] = Pack<T, V>{};
      qz[i] = Pack<T, V>{};
      if (live && c < p.Dg) {
        qx[i] = load_pack<T, V>(x + c);
        if (z != nullptr) qz[i] = load_pack<T, V>(z + c);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      unpack<T, V>(qx[i], v[i]);
      unpack<T, V>(qz[i], gate[i]);
#pragma unroll
      for (int j = 0; j < V; ++j) {
        gate[i][j] = z != nullptr ? silu_f(gate[i][j]) : 1.f;
        if (first) v[i][j] *= gate[i][j];
        s = fmaf(v[i][j], v[i][j], s);
      }
    }
    const float r = rsqrtf(team_sum<BLK>(s, p.lgteam, red) * p.inv + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * team + lane) * V;
      if (!live || c >= p.Dg) continue;
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) {
        o[j] = v[i][j] * r * (w != nullptr ? w[c + j] : 1.f);
        if (!first) o[j] *= gate[i][j];
      }
      store_pack<T, V>(y + c, o);
    }
  } else {
    float s = 0.f;
    for (int c = lane; c < p.Dg; c += team) {
      float v = to_f32(x[c]);
      if (first && z != nullptr) v *= silu_f(to_f32(z[c]));
      s = fmaf(v, v, s);
    }
    const float r = rsqrtf(team_sum<BLK>(s, p.lgteam, red) * p.inv + p.eps);
    for (int c = lane; c < p.Dg; c += team) {
      const float gate = z != nullptr ? silu_f(to_f32(z[c])) : 1.f;
      from_f32(to_f32(x[c]) * gate * r * (w != nullptr ? w[c] : 1.f), y[c]);
    }
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
// a row, v^2 and e v, go through one reduction.  A team keeps its group and
// walks rows `walkers` apart, so that its part of dw stays in registers.
template <typename T, int V, int NV, int BLK>
__global__ __launch_bounds__(threads<BLK>()) void gated_backward_kernel(GatedBwP p) {
  __shared__ float red[2][2][16];
  const int64_t slot = team_index<BLK>(p.lgteam);
  const int lane = team_lane<BLK>(p.lgteam), team = BLK ? BLK : 1 << p.lgteam;
  const int64_t walker = slot / p.G;
  const int g0 = int(slot - walker * p.G) * p.Dg;
  const bool live = walker < p.walkers;
  const bool first = p.gate_first != 0, gated = p.z != nullptr;
  const float* w = p.w == nullptr ? nullptr : p.w + g0;
  float* part = p.part == nullptr ? nullptr : p.part + walker * p.D + g0;
  constexpr int NR = NV > 0 ? NV : 1;
  float dw[NR][V], wr[NR][V];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int c = (i * team + lane) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      dw[i][j] = 0.f;
      wr[i][j] = NV > 0 && w != nullptr && live && c < p.Dg ? w[c + j] : 1.f;
    }
  }
  if constexpr (NV == 0) {
    if (part != nullptr && live)
      for (int c = lane; c < p.Dg; c += team) part[c] = 0.f;
  }
  // every team of a block makes the same number of turns (the block's barriers)
  const int64_t turns = (p.M + p.walkers - 1) / p.walkers;
  for (int64_t k = 0; k < turns; ++k) {
    const int64_t row = walker + k * p.walkers;
    const bool on = live && row < p.M;
    const T* x = static_cast<const T*>(p.x) + (on ? row : 0) * p.xld + g0;
    const T* z = gated ? static_cast<const T*>(p.z) + (on ? row : 0) * p.zld + g0 : nullptr;
    const T* dy = static_cast<const T*>(p.dy) + (on ? row : 0) * p.D + g0;
    T* dx = static_cast<T*>(p.dx) + (on ? row : 0) * p.D + g0;
    T* dz = static_cast<T*>(p.dz) + (on ? row : 0) * p.D + g0;
    float s1 = 0.f, s2 = 0.f;
    if constexpr (NV > 0) {
      Pack<T, V> qx[NV], qz[NV], qd[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * team + lane) * V;
        qx[i] = qz[i] = qd[i] = Pack<T, V>{};
        if (on && c < p.Dg) {
          qx[i] = load_pack<T, V>(x + c);
          qd[i] = load_pack<T, V>(dy + c);
          if (gated) qz[i] = load_pack<T, V>(z + c);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float gate = gated ? silu_f(to_f32(qz[i].e[j])) : 1.f;
          const float xv = to_f32(qx[i].e[j]), u = to_f32(qd[i].e[j]) * wr[i][j];
          const float v = first ? xv * gate : xv;
          s1 = fmaf(v, v, s1);
          s2 = fmaf(first ? u : u * gate, v, s2);
        }
      s1 = team_sum<BLK>(s1, p.lgteam, red[k & 1][0]);
      s2 = team_sum<BLK>(s2, p.lgteam, red[k & 1][1]);
      const float r = rsqrtf(s1 * p.inv + p.eps), m = s2 * r * p.inv;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * team + lane) * V;
        if (!on || c >= p.Dg) continue;
        float ox[V], oz[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float zv = to_f32(qz[i].e[j]), xv = to_f32(qx[i].e[j]), d = to_f32(qd[i].e[j]);
          const float sg = gated ? sigmoid_f(zv) : 1.f, gate = gated ? zv * sg : 1.f;
          const float n = (first ? xv * gate : xv) * r;
          const float u = first ? d : d * gate;
          const float dv = r * (u * wr[i][j] - n * m);
          ox[j] = first ? dv * gate : dv;
          oz[j] = (first ? dv * xv : d * n * wr[i][j]) * dsilu_f(zv, sg);
          dw[i][j] = fmaf(u, n, dw[i][j]);
        }
        store_pack<T, V>(dx + c, ox);
        if (gated) store_pack<T, V>(dz + c, oz);
      }
    } else {
      for (int c = lane; on && c < p.Dg; c += team) {
        const float gate = gated ? silu_f(to_f32(z[c])) : 1.f;
        const float xv = to_f32(x[c]), u = to_f32(dy[c]) * (w != nullptr ? w[c] : 1.f);
        const float v = first ? xv * gate : xv;
        s1 = fmaf(v, v, s1);
        s2 = fmaf(first ? u : u * gate, v, s2);
      }
      s1 = team_sum<BLK>(s1, p.lgteam, red[k & 1][0]);
      s2 = team_sum<BLK>(s2, p.lgteam, red[k & 1][1]);
      const float r = rsqrtf(s1 * p.inv + p.eps), m = s2 * r * p.inv;
      for (int c = lane; on && c < p.Dg; c += team) {
        const float zv = gated ? to_f32(z[c]) : 0.f, xv = to_f32(x[c]), d = to_f32(dy[c]);
        const float sg = gated ? sigmoid_f(zv) : 1.f, gate = gated ? zv * sg : 1.f;
        const float wc = w != nullptr ? w[c] : 1.f;
        const float n = (first ? xv * gate : xv) * r;
        const float u = first ? d : d * gate;
        const float dv = r * (u * wc - n * m);
        from_f32(first ? dv * gate : dv, dx[c]);
        if (gated) from_f32((first ? dv * xv : d * n * wc) * dsilu_f(zv, sg), dz[c]);
        if (part != nullptr) part[c] = fmaf(u, n, part[c]);
      }
    }
  }
  if constexpr (NV > 0) {
    if (part == nullptr || !live) return;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * team + lane) * V;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (c + j < p.Dg) part[c + j] = dw[i][j];
    }
  }
}

struct ResP {
  const void* x;
  const void* res;
  const float* scale;
  const float* w;
  void* y;
  void* res_out;
  int64_t xld, M;
  int D, lgteam;
  float eps, inv;
};

template <typename T, typename R, int V, int NV, int BLK>
__global__ __launch_bounds__(threads<BLK>()) void residual_kernel(ResP p) {
  __shared__ float red[16];
  const int64_t unit = team_index<BLK>(p.lgteam);
  const int lane = team_lane<BLK>(p.lgteam), team = BLK ? BLK : 1 << p.lgteam;
  const bool live = unit < p.M;
  const int64_t row = live ? unit : 0;
  const T* x = static_cast<const T*>(p.x) + row * p.xld;
  const R* res = p.res == nullptr ? nullptr : static_cast<const R*>(p.res) + row * p.D;
  R* out = p.res_out == nullptr ? nullptr : static_cast<R*>(p.res_out) + row * p.D;
  T* y = static_cast<T*>(p.y) + row * p.D;
  if constexpr (NV > 0) {
    float h[NV][V];
    float s = 0.f;
    Pack<T, V> qx[NV];
    Pack<R, V> qr[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * team + lane) * V;
      qx[i] = Pack<T, V>{};
      qr[i] = Pack<R, V>{};
      if (live && c < p.D) {
        qx[i] = load_pack<T, V>(x + c);
        if (res != nullptr) qr[i] = load_pack<R, V>(res + c);
      }
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * team + lane) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) {
        const float sc = p.scale != nullptr && c < p.D ? p.scale[c + j] : 1.f;
        h[i][j] = fmaf(sc, to_f32(qx[i].e[j]), to_f32(qr[i].e[j]));
        s = fmaf(h[i][j], h[i][j], s);
      }
      if (out != nullptr && live && c < p.D) store_pack<R, V>(out + c, h[i]);
    }
    const float r = rsqrtf(team_sum<BLK>(s, p.lgteam, red) * p.inv + p.eps);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * team + lane) * V;
      if (!live || c >= p.D) continue;
      float o[V];
#pragma unroll
      for (int j = 0; j < V; ++j) o[j] = h[i][j] * r * (p.w != nullptr ? p.w[c + j] : 1.f);
      store_pack<T, V>(y + c, o);
    }
  } else {
    auto sum = [&](int c) {
      return fmaf(p.scale != nullptr ? p.scale[c] : 1.f, to_f32(x[c]), res != nullptr ? to_f32(res[c]) : 0.f);
    };
    float s = 0.f;
    for (int c = lane; c < p.D; c += team) {
      const float h = sum(c);
      s = fmaf(h, h, s);
    }
    const float r = rsqrtf(team_sum<BLK>(s, p.lgteam, red) * p.inv + p.eps);
    for (int c = lane; c < p.D; c += team) {
      const float h = sum(c);
      if (out != nullptr) from_f32(h, out[c]);
      from_f32(h * r * (p.w != nullptr ? p.w[c] : 1.f), y[c]);
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
// sum dh x; rows walked as in the gated norm's backward.
template <typename T, typename R, int V, int NV, int BLK>
__global__ __launch_bounds__(threads<BLK>()) void residual_backward_kernel(ResBwP p) {
  __shared__ float red[2][2][16];
  const int64_t walker = team_index<BLK>(p.lgteam);
  const int lane = team_lane<BLK>(p.lgteam), team = BLK ? BLK : 1 << p.lgteam;
  const bool live = walker < p.walkers;
  float* pw = nullptr;
  float* ps = nullptr;
  if (live) {
    float* row = p.part + walker * (p.has_dw + p.has_ds) * p.D;
    if (p.has_dw) pw = row;
    if (p.has_ds) ps = row + (p.has_dw ? p.D : 0);
  }
  constexpr int NR = NV > 0 ? NV : 1;
  float dw[NR][V], ds[NR][V], wr[NR][V], sr[NR][V];
#pragma unroll
  for (int i = 0; i < NR; ++i) {
    const int c = (i * team + lane) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) {
      dw[i][j] = ds[i][j] = 0.f;
      wr[i][j] = NV > 0 && p.w != nullptr && c < p.D ? p.w[c + j] : 1.f;
      sr[i][j] = NV > 0 && p.scale != nullptr && c < p.D ? p.scale[c + j] : 1.f;
    }
  }
  if constexpr (NV == 0) {
    for (int c = lane; c < p.D; c += team) {
      if (pw != nullptr) pw[c] = 0.f;
      if (ps != nullptr) ps[c] = 0.f;
    }
  }
  const int64_t turns = (p.M + p.walkers - 1) / p.walkers;
  for (int64_t k = 0; k < turns; ++k) {
    const bool on = live && walker + k * p.walkers < p.M;
    const int64_t row = on ? walker + k * p.walkers : 0;
    const R* h = static_cast<const R*>(p.h) + row * p.D;
    const T* x = static_cast<const T*>(p.x) + row * p.xld;
    const T* dy = static_cast<const T*>(p.dy) + row * p.D;
    const R* dro = p.dro == nullptr ? nullptr : static_cast<const R*>(p.dro) + row * p.D;
    T* dx = p.dx == nullptr ? nullptr : static_cast<T*>(p.dx) + row * p.D;
    R* dres = p.dres == nullptr ? nullptr : static_cast<R*>(p.dres) + row * p.D;
    float s1 = 0.f, s2 = 0.f;
    if constexpr (NV > 0) {
      Pack<R, V> qh[NV], qr[NV];
      Pack<T, V> qd[NV], qx[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * team + lane) * V;
        qh[i] = qr[i] = Pack<R, V>{};
        qd[i] = qx[i] = Pack<T, V>{};
        if (on && c < p.D) {
          qh[i] = load_pack<R, V>(h + c);
          qd[i] = load_pack<T, V>(dy + c);
          if (dro != nullptr) qr[i] = load_pack<R, V>(dro + c);
          if (p.has_ds) qx[i] = load_pack<T, V>(x + c);
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float hv = to_f32(qh[i].e[j]);
          s1 = fmaf(hv, hv, s1);
          s2 = fmaf(to_f32(qd[i].e[j]) * wr[i][j], hv, s2);
        }
      s1 = team_sum<BLK>(s1, p.lgteam, red[k & 1][0]);
      s2 = team_sum<BLK>(s2, p.lgteam, red[k & 1][1]);
      const float r = rsqrtf(s1 * p.inv + p.eps), m = s2 * r * p.inv;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (i * team + lane) * V;
        if (!on || c >= p.D) continue;
        float o[V], ox[V];
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const float n = to_f32(qh[i].e[j]) * r, d = to_f32(qd[i].e[j]);
          o[j] = to_f32(qr[i].e[j]) + r * (d * wr[i][j] - n * m);
          ox[j] = sr[i][j] * o[j];
          dw[i][j] = fmaf(d, n, dw[i][j]);
          ds[i][j] = fmaf(o[j], to_f32(qx[i].e[j]), ds[i][j]);
        }
        if (dres != nullptr) store_pack<R, V>(dres + c, o);
        if (dx != nullptr) store_pack<T, V>(dx + c, ox);
      }
    } else {
      for (int c = lane; on && c < p.D; c += team) {
        const float hv = to_f32(h[c]);
        s1 = fmaf(hv, hv, s1);
        s2 = fmaf(to_f32(dy[c]) * (p.w != nullptr ? p.w[c] : 1.f), hv, s2);
      }
      s1 = team_sum<BLK>(s1, p.lgteam, red[k & 1][0]);
      s2 = team_sum<BLK>(s2, p.lgteam, red[k & 1][1]);
      const float r = rsqrtf(s1 * p.inv + p.eps), m = s2 * r * p.inv;
      for (int c = lane; on && c < p.D; c += team) {
        const float n = to_f32(h[c]) * r, d = to_f32(dy[c]);
        const float o = (dro != nullptr ? to_f32(dro[c]) : 0.f) + r * (d * (p.w != nullptr ? p.w[c] : 1.f) - n * m);
        if (dres != nullptr) from_f32(o, dres[c]);
        if (dx != nullptr) from_f32((p.scale != nullptr ? p.scale[c] : 1.f) * o, dx[c]);
        if (pw != nullptr) pw[c] = fmaf(d, n, pw[c]);
        if (ps != nullptr) ps[c] = fmaf(o, to_f32(x[c]), ps[c]);
      }
    }
  }
  if constexpr (NV > 0) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (i * team + lane) * V;
#pragma unroll
      for (int j = 0; j < V; ++j)
        if (c + j < p.D) {
          if (pw != nullptr) pw[c + j] = dw[i][j];
          if (ps != nullptr) ps[c + j] = ds[i][j];
        }
    }
  }
}

// Lanes for a unit of `width` elements.  Up to 64 words: one wave or a part of
// it.  Up to 256 words: four words per lane of a wave where the units fill the
// card (2048 waves or more), else a block of 256 lanes; then wider blocks, and
// the loop for what no block holds in registers.
Geom pick(int64_t units, int width, int V, bool vec) {
  Geom g{vec, 1, 0, 6};
  const int64_t words = (int64_t(width) + V - 1) / V;
  if (words <= 64) {
    g.lgteam = 0;
    while ((1 << g.lgteam) < words) ++g.lgteam;
  } else if (words <= 128 && units >= 2048) {
    g.nv = 2;
  } else if (words <= 256 && units >= 2048) {
    g.nv = 4;
  } else if (words <= 256) {
    g.blk = 256;
  } else if (words <= 512) {
    g.blk = 256;
    g.nv = 2;
  } else if (words <= 1024) {
    g.blk = 256;
    g.nv = 4;
  } else if (words <= 4096) {
    g.blk = 1024;
    g.nv = 4;
  } else {
    g.vec = false;
    g.blk = 1024;
    g.nv = 0;
  }
  return g;
}

// Rows a team of the backward kernels walks: enough teams for 2048 waves, but
// at least 32 rows each once the card is full (the partial sums of a team cost
// as much as four rows).
int64_t pick_walkers(int64_t M, int G, const Geom& g) {
  const int64_t lanes = g.blk ? g.blk : int64_t(1) << g.lgteam;
  int64_t w = (int64_t(2048) * 64 + lanes * G - 1) / (lanes * G);
  if (w < (M + 31) / 32) w = (M + 31) / 32;
  const int64_t most = (int64_t(16384) * 64 + lanes * G - 1) / (lanes * G);
  if (w > most) w = most;
  return w < M ? w : M;
}

// The kernel instance for a geometry: F<V, NV, BLK>(...).
#define M3_NORM_DISPATCH(g, VV, CALL)                      \
  if ((g).nv == 0) return CALL(1, 0, 1024);                \
  if ((g).vec) {                                           \
    if ((g).blk == 1024) return CALL(VV, 4, 1024);         \
    if ((g).blk == 256) {                                  \
      if ((g).nv == 1) return CALL(VV, 1, 256);            \
      if ((g).nv == 2) return CALL(VV, 2, 256);            \
      return CALL(VV, 4, 256);                             \
    }                                                      \
    if ((g).nv == 1) return CALL(VV, 1, 0);                \
    if ((g).nv == 2) return CALL(VV, 2, 0);                \
    return CALL(VV, 4, 0);                                 \
  }                                                        \
  if ((g).blk == 1024) return CALL(1, 4, 1024);            \
  if ((g).blk == 256) {                                    \
    if ((g).nv == 1) return CALL(1, 1, 256);               \
    if ((g).nv == 2) return CALL(1, 2, 256);               \
    return CALL(1, 4, 256);                                \
  }                                                        \
  if ((g).nv == 1) return CALL(1, 1, 0);                   \
  if ((g).nv == 2) return CALL(1, 2, 0);                   \
  return CALL(1, 4, 0);

uint32_t grid_of(const Geom& g, int64_t teams) {
  return uint32_t(g.blk ? teams : ((teams << g.lgteam) + 255) / 256);
}

template <typename T>
hipError_t run_gated(const m3_gated_norm_args& a, hipStream_t s) {
  constexpr int VV = 16 / int(sizeof(T));
  const int Dg = a.D / a.G;
  const bool vec = Dg % VV == 0 && rows_aligned(a.x, a.x_ld, sizeof(T), 16) && rows_aligned(a.z, a.z_ld, sizeof(T), 16) &&
                   rows_aligned(a.y, a.D, sizeof(T), 16);
  const Geom g = pick(a.M * a.G, Dg, vec ? VV : 1, vec);
  const GatedP p{a.x, a.z, a.w, a.y, a.x_ld, a.z_ld, a.M * a.G, a.D, a.G, Dg, g.lgteam, a.gate_first, a.eps, 1.f / float(Dg)};
#define CALL(V, NV, BLK) (gated_kernel<T, V, NV, BLK><<<grid_of(g, p.units), threads<BLK>(), 0, s>>>(p), hipGetLastError())
  M3_NORM_DISPATCH(g, VV, CALL)
#undef CALL
}

template <typename T>
bool gated_bw_vec(const m3_gated_norm_backward_args& a) {
  constexpr int VV = 16 / int(sizeof(T));
  const m3_gated_norm_args& f = a.fwd;
  return (f.D / f.G) % VV == 0 && rows_aligned(f.x, f.x_ld, sizeof(T), 16) && rows_aligned(f.z, f.z_ld, sizeof(T), 16) &&
         rows_aligned(a.dy, f.D, sizeof(T), 16) && rows_aligned(a.dx, f.D, sizeof(T), 16) &&
         rows_aligned(a.dz, f.D, sizeof(T), 16);
}
template <typename T>
hipError_t launch_gated_bw(const GatedBwP& p, const Geom& g, hipStream_t s) {
  constexpr int VV = 16 / int(sizeof(T));
#define CALL(V, NV, BLK) \
  (gated_backward_kernel<T, V, NV, BLK><<<grid_of(g, p.walkers * p.G), threads<BLK>(), 0, s>>>(p), hipGetLastError())
  M3_NORM_DISPATCH(g, VV, CALL)
#undef CALL
}
template <typename T>
hipError_t run_gated_bw(const m3_gated_norm_backward_args& a, hipStream_t s) {
  constexpr int VV = 16 / int(sizeof(T));
  const m3_gated_norm_args& f = a.fwd;
  const int Dg = f.D / f.G;
  const bool vec = gated_bw_vec<T>(a);
  const Geom g = pick(f.M * f.G, Dg, vec ? VV : 1, vec);
  const GatedBwP p{f.x, f.z, f.w, a.dy, a.dx, a.dz, f.w != nullptr ? static_cast<float*>(a.workspace) : nullptr, f.x_ld, f.z_ld,
                   f.M, pick_walkers(f.M, f.G, g), f.D, f.G, Dg, g.lgteam, f.gate_first, f.eps, 1.f / float(Dg)};
  const hipError_t e = launch_gated_bw<T>(p, g, s);
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
                   rows_aligned(a.residual, a.D, sizeof(R), 16) && rows_aligned(a.residual_out, a.D, sizeof(R), 16);
  const Geom g = pick(a.M, a.D, vec ? VV : 1, vec);
  const ResP p{a.x, a.residual, a.scale, a.w, a.y, a.residual_out, a.x_ld, a.M, a.D, g.lgteam, a.eps, 1.f / float(a.D)};
#define CALL(V, NV, BLK) (residual_kernel<T, R, V, NV, BLK><<<grid_of(g, p.M), threads<BLK>(), 0, s>>>(p), hipGetLastError())
  M3_NORM_DISPATCH(g, VV, CALL)
#undef CALL
}
template <typename T, typename R>
hipError_t launch_residual_bw(const ResBwP& p, const Geom& g, hipStream_t s) {
  constexpr int VV = 16 / int(sizeof(T));
#define CALL(V, NV, BLK) \
  (residual_backward_kernel<T, R, V, NV, BLK><<<grid_of(g, p.walkers), threads<BLK>(), 0, s>>>(p), hipGetLastError())
  M3_NORM_DISPATCH(g, VV, CALL)
#undef CALL
}
template <typename T, typename R>
hipError_t run_residual_bw(const m3_residual_norm_backward_args& a, hipStream_t s) {
  constexpr int VV = 16 / int(sizeof(T));
  const bool vec = a.D % VV == 0 && rows_aligned(a.x, a.x_ld, sizeof(T), 16) && rows_aligned(a.dy, a.D, sizeof(T), 16) &&
                   rows_aligned(a.dx, a.D, sizeof(T), 16) && rows_aligned(a.h, a.D, sizeof(R), 16) &&
                   rows_aligned(a.dresidual_out, a.D, sizeof(R), 16) && rows_aligned(a.dresidual, a.D, sizeof(R), 16);
  const Geom g = pick(a.M, a.D, vec ? VV : 1, vec);
  const ResBwP p{a.h, a.x, a.scale, a.w, a.dy, a.dresidual_out, a.dx, a.dresidual, static_cast<float*>(a.workspace), a.x_ld, a.M,
                 pick_walkers(a.M, 1, g), a.D, g.lgteam, a.w != nullptr, a.scale != nullptr, a.eps, 1.f / float(a.D)};
  const hipError_t e = launch_residual_bw<T, R>(p, g, s);
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
// The sizes cover both widths of the lanes (the addresses are not known here).
size_t gated_norm_backward_workspace(const m3_gated_norm_backward_args& a) {
  const m3_gated_norm_args& f = a.fwd;
  if (f.w == nullptr) return 0;
  const int V = f.in_dtype == M3_BF16 ? 8 : 4, Dg = f.D / f.G;
  int64_t w = pick_walkers(f.M, f.G, pick(f.M * f.G, Dg, 1, false));
  const int64_t v = pick_walkers(f.M, f.G, pick(f.M * f.G, Dg, V, true));
  if (v > w) w = v;
  return round256(size_t(w) * f.D * 4);
}
hipError_t launch_gated_norm_backward(const m3_gated_norm_backward_args& a, hipStream_t s) {
  return a.fwd.in_dtype == M3_BF16 ? run_gated_bw<bf16_t>(a, s) : run_gated_bw<float>(a, s);
}
hipError_t launch_residual_norm(const m3_residual_norm_args& a, hipStream_t s) {
  if (a.in_dtype == M3_F32) return run_residual<float, float>(a, s);
  return a.res_dtype == M3_BF16 ? run_residual<bf16_t, bf16_t>(a, s) : run_residual<bf16_t, float>(a, s);
}
size_t residual_norm_backward_workspace(const m3_residual_norm_backward_args& a) {
  const int V = a.in_dtype == M3_BF16 ? 8 : 4;
  int64_t w = pick_walkers(a.M, 1, pick(a.M, a.D, 1, false));
  const int64_t v = pick_walkers(a.M, 1, pick(a.M, a.D, V, true));
  if (v > w) w = v;
  return round256(size_t(w) * ((a.w != nullptr) + (a.scale != nullptr)) * a.D * 4);
}
hipError_t launch_residual_norm_backward(const m3_residual_norm_backward_args& a, hipStream_t s) {
  if (a.in_dtype == M3_F32) return run_residual_bw<float, float>(a, s);
  return a.res_dtype == M3_BF16 ? run_residual_bw<bf16_t, bf16_t>(a, s) : run_residual_bw<bf16_t, float>(a, s);
}

}  // namespace m3
