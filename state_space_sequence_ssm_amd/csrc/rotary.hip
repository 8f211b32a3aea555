// Norm of queries and keys for each head and their rotation by position, forward and
// backward.  Memory bound: every element is read and written once.
#include "mixer_internal.hpp"
#include "rotary_plan.hpp"

namespace m3 {
namespace {

using namespace rope;

// A wave takes one token: its cosines and sines, which all heads share, are formed once by
// its 64 lanes and handed round through LDS.  Teams of 2^lgteam lanes then take a head each.
// A lane holds NU units of its head, two words of V elements: with rotation the partners of
// V pairs (words R / 2 apart, or with ADJ 2 V adjacent elements), behind R any 2 V elements.
// RAG: words have the alignment of their elements only, and a range's last unit is moved back
// to end with it, its first elements, which the unit before holds too, left out of the sums
// and stored twice with the same value.
// 32768 tokens of 16 + 16 heads of 128 bf16: 104 us, 5.1 TB/s (one token's loads at a time and
// gains read for each head: 157); backward of 16 + 4 heads 152 us, 3.3 TB/s: 198 registers leave
// two waves a SIMD, which wait for memory three quarters of the time (three spill: slower).

// cos and sin of 2 pi r, r in turns: reduced in 64 bits to an eighth of a turn around a
// quarter, then the series of sine and cosine to x^9 and x^10 (off by 2e-9 at pi / 4).
__device__ __forceinline__ float2 turn_of(double r) {
  r -= __builtin_rint(r);
  const double quarter = __builtin_rint(4.0 * r);
  const float x = static_cast<float>((r - 0.25 * quarter) * 6.283185307179586476925);
  const float z = x * x;
  const float s = x * fmaf(z, fmaf(z, fmaf(z, fmaf(z, 2.7557319e-6f, -1.9841270e-4f), 8.3333333e-3f), -0.16666667f), 1.f);
  const float c = fmaf(z, fmaf(z, fmaf(z, fmaf(z, fmaf(z, -2.7557319e-7f, 2.4801587e-5f), -1.3888889e-3f), 4.1666667e-2f), -0.5f), 1.f);
  const int k = static_cast<int>(quarter) & 3;
  const float a = k & 1 ? s : c, b = k & 1 ? c : s;
  return {k == 1 || k == 2 ? -a : a, k >= 2 ? -b : b};
}

// Sum over a team of 2^lg lanes, in every lane.
__device__ __forceinline__ float team_sum(float v, int lg) {
  if (lg >= 1) v += dpp<0xB1, 0xF, true>(v);
  if (lg >= 2) v += dpp<0x4E, 0xF, true>(v);
  if (lg >= 3) v += dpp<0x141, 0xF, true>(v);
  if (lg >= 4) v += dpp<0x140, 0xF, true>(v);
  if (lg >= 5) v = add_x16(v);
  if (lg >= 6) v = add_x32(v);
  return v;
}

// (x0, x1) turned by the angle of (c, s); the transposed turn with the other sign of s.  Where
// `turned` is false they stay, and are not turned by (1, 0): an infinity times 0 is not a number.
// A choice for each element: a branch around them takes 16 registers more and a wave a SIMD.
__device__ __forceinline__ void turn2(float& x0, float& x1, float c, float s, bool turned) {
  const float y0 = fmaf(x0, c, -(x1 * s)), y1 = fmaf(x1, c, x0 * s);
  x0 = turned ? y0 : x0;
  x1 = turned ? y1 : x1;
}
template <int V, bool ADJ>
__device__ __forceinline__ void turn_unit(float (&a)[V], float (&b)[V], const float2 (&cs)[V], float sign, bool turned) {
  if constexpr (!ADJ || V == 1) {
#pragma unroll
    for (int j = 0; j < V; ++j) turn2(a[j], b[j], cs[j].x, sign * cs[j].y, turned);
  } else {
#pragma unroll
    for (int j = 0; j < V / 2; ++j) {
      turn2(a[2 * j], a[2 * j + 1], cs[j].x, sign * cs[j].y, turned);
      turn2(b[2 * j], b[2 * j + 1], cs[V / 2 + j].x, sign * cs[V / 2 + j].y, turned);
    }
  }
}
template <typename T, int V, bool RAG>
__device__ __forceinline__ Pack<T, V> fetch(const T* p) {
  if constexpr (V == 1) {
    Pack<T, 1> q;
    q.e[0] = *p;
    return q;
  } else {
    return load_word<T, V, RAG>(p);
  }
}
template <typename T, int V, bool RAG>
__device__ __forceinline__ void put(T* p, const float (&v)[V]) {
  if constexpr (V == 1) from_f32(v[0], *p);
  else store_word<T, V, RAG>(p, v);
}

// The token's cosines and sines into this wave's part of LDS; no other wave reads them.
// `first`: this lane's first rate in turns, kept from token to token, so that no load of it
// waits for the heads that are on their way.
__device__ __forceinline__ double rate_of(const RopeP& p, int i) { return i < p.R / 2 ? double(p.freqs[i]) * 0.15915494309189533577 : 0.0; }
__device__ __forceinline__ void angles(const RopeP& p, float2* cs, int at, int lane, double first) {
  const double pos = double(at) + (p.positions == nullptr ? double(p.start) : 0.0);  // may pass 32 bits
  if (lane < p.R / 2) cs[lane] = turn_of(pos * first);
  for (int i = lane + 64; i < p.R / 2; i += 64) cs[i] = turn_of(pos * rate_of(p, i));
  __builtin_amdgcn_wave_barrier();
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
}
template <int V, int NU, bool RAG, bool ADJ>
__device__ __forceinline__ void angles_of(const Units<V, NU, RAG, ADJ>& u, const float2* cs, float2 (&o)[NU][V]) {
#pragma unroll
  for (int i = 0; i < NU; ++i)
#pragma unroll
    for (int j = 0; j < V; ++j) o[i][j] = u.pair[i] < 0 ? float2{1.f, 0.f} : cs[u.pair[i] + j];
}

// A lane's gains (1 without them), kept in registers while a wave walks tokens: read anew for
// each head they were half of the loads, and read one by one 8 us of 121.
template <int V, int NU>
struct Gains {
  float a[NU][V], b[NU][V];
  template <bool RAG, bool ADJ>
  __device__ __forceinline__ Gains(const float* w, const Units<V, NU, RAG, ADJ>& u) {
    if (w == nullptr) {
#pragma unroll
      for (int i = 0; i < NU; ++i)
#pragma unroll
        for (int j = 0; j < V; ++j) a[i][j] = b[i][j] = 1.f;
      return;
    }
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      unpack<float, V>(fetch<float, V, true>(w + u.a[i]), a[i]);
      unpack<float, V>(fetch<float, V, true>(w + u.b[i]), b[i]);
    }
  }
};

// Turn `it` of a wave over the heads of a token: q's first, then k's.
struct Head {
  int k, mine, head;
  __device__ __forceinline__ Head(const RopeP& p, int it, int teams, int lane) {
    k = it >= p.its[0] ? 1 : 0;
    mine = (it - (k ? p.its[0] : 0)) * teams + (lane >> p.lgteam);
    head = min(mine, p.heads[k] - 1);
  }
};

// A token: whether its item holds it, and its position (without positions: behind `start`).  A
// wave looks at the next one while it works on one, so that the next one's first heads are on
// their way too.
struct Token {
  int64_t row;
  int pos;
  bool any, held;
  __device__ __forceinline__ Token(const RopeP& p, int64_t r) : row(r), pos(0), any(r < p.rows), held(false) {
    if (!any) return;
    const int t = int(row % p.L);
    held = t < item_length(p.lengths, int(row / p.L), p.L);
    if (held && p.R > 0) pos = p.positions == nullptr ? t : p.positions[row];
  }
};

template <typename T, int V, int NU, bool RAG, bool ADJ>
__global__ __launch_bounds__(256) void rope_kernel(RopeP p) {
  extern __shared__ float2 lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t id = int64_t(blockIdx.x) * 4 + wave, walker = id / p.splits;
  const int split = int(id % p.splits);
  float2* cs = lds + wave * (p.R / 2);
  const int team = 1 << p.lgteam, teams = 64 >> p.lgteam;
  const Units<V, NU, RAG, ADJ> u(p, lane & (team - 1), team);
  const int all = p.its[0] + p.its[1], each = (all + p.splits - 1) / p.splits;
  const Gains<V, NU> wq(p.w[0], u), wk(p.w[1], u);
  const double rate = rate_of(p, lane);
  const int begin = split * each, last = min(all, begin + each);
  if (begin >= last) return;
  Pack<T, V> qa[NU], qb[NU];
  auto load = [&](int64_t row, int it) {
    const Head h(p, it, teams, lane);
    const T* x = static_cast<const T*>(p.x[h.k]) + row * p.ld[h.k] + int64_t(h.head) * p.D;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      qa[i] = fetch<T, V, RAG>(x + u.a[i]);
      qb[i] = fetch<T, V, RAG>(x + u.b[i]);
    }
  };
  Token now(p, walker < p.walkers ? walker : p.rows);
  if (now.held) load(now.row, begin);
  while (now.any) {
    const int64_t row = now.row;
    const Token next(p, row + p.walkers);
    if (!now.held) {
      if (next.held) load(next.row, begin);
      now = next;
      continue;
    }
    if (p.R > 0) angles(p, cs, now.pos, lane, rate);
    float2 turn[NU][V];
    angles_of<V, NU, RAG, ADJ>(u, cs, turn);
    for (int it = begin; it < last; ++it) {
      const Head h(p, it, teams, lane);
      T* y = static_cast<T*>(p.y[h.k]) + (row * p.heads[h.k] + h.head) * p.D;
      float a[NU][V], b[NU][V];
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        unpack<T, V>(qa[i], a[i]);
        unpack<T, V>(qb[i], b[i]);
      }
      // the next heads on their way (in place: other heads than these)
      if (it + 1 < last) load(row, it + 1);
      else if (next.held) load(next.row, begin);
      if (p.norm) {
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const float va = u.in[i] && u.counts_a(i, j) ? a[i][j] : 0.f, vb = u.in[i] && u.counts_b(i, j) ? b[i][j] : 0.f;
            s = fmaf(va, va, fmaf(vb, vb, s));
          }
        const float r = rsqrtf(team_sum(s, p.lgteam) * p.inv + p.eps);
        auto scale = [&](const Gains<V, NU>& w) {
#pragma unroll
          for (int i = 0; i < NU; ++i)
#pragma unroll
            for (int j = 0; j < V; ++j) {
              a[i][j] *= r * w.a[i][j];
              b[i][j] *= r * w.b[i][j];
            }
        };
        if (h.k == 0) scale(wq);
        else scale(wk);
      }
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        turn_unit<V, ADJ>(a[i], b[i], turn[i], 1.f, u.pair[i] >= 0);
        if (NU == 1 || u.in[i]) {
          put<T, V, RAG>(y + u.a[i], a[i]);
          put<T, V, RAG>(y + u.b[i], b[i]);
        }
      }
    }
    now = next;
  }
}

// With n = x r, r = rsqrt(mean(x^2) + eps), d = the output's gradient turned back and
// e = d w:  dw = sum d n,  dx = r (e - n mean(e n)).
template <typename T, int V, int NU, bool RAG, bool ADJ>
__global__ __launch_bounds__(256) void rope_backward_kernel(RopeP p) {
  extern __shared__ float2 lds[];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int64_t id = int64_t(blockIdx.x) * 4 + wave, walker = id / p.splits;
  const int split = int(id % p.splits);
  float2* cs = lds + wave * (p.R / 2);
  const int team = 1 << p.lgteam, teams = 64 >> p.lgteam;
  const Units<V, NU, RAG, ADJ> u(p, lane & (team - 1), team);
  const int all = p.its[0] + p.its[1], each = (all + p.splits - 1) / p.splits;
  const Gains<V, NU> wq(p.w[0], u), wk(p.w[1], u);
  const double rate = rate_of(p, lane);
  float dwa[2][NU][V], dwb[2][NU][V];
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) dwa[k][i][j] = dwb[k][i][j] = 0.f;
  const int begin = split * each, last = min(all, begin + each);
  Pack<T, V> qa[NU], qb[NU], ga[NU], gb[NU];
  auto load = [&](int64_t row, int it) {
    const Head h(p, it, teams, lane);
    const T* x = static_cast<const T*>(p.x[h.k]) + row * p.ld[h.k] + int64_t(h.head) * p.D;
    const T* dy = static_cast<const T*>(p.dy[h.k]) + (row * p.heads[h.k] + h.head) * p.D;
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      qa[i] = fetch<T, V, RAG>(x + u.a[i]);
      qb[i] = fetch<T, V, RAG>(x + u.b[i]);
      ga[i] = fetch<T, V, RAG>(dy + u.a[i]);
      gb[i] = fetch<T, V, RAG>(dy + u.b[i]);
    }
  };
  Token now(p, walker < p.walkers && begin < last ? walker : p.rows);
  if (now.held) load(now.row, begin);
  while (now.any) {
    const int64_t row = now.row;
    const bool held = now.held;
    const Token next(p, row + p.walkers);
    float2 turn[NU][V];
    if (held) {
      if (p.R > 0) angles(p, cs, now.pos, lane, rate);
      angles_of<V, NU, RAG, ADJ>(u, cs, turn);
    }
    for (int it = begin; it < last; ++it) {
      const Head h(p, it, teams, lane);
      T* dx = static_cast<T*>(p.y[h.k]) + (row * p.heads[h.k] + h.head) * p.D;
      float a[NU][V], b[NU][V], da[NU][V], db[NU][V];
      if (!held) {
#pragma unroll
        for (int j = 0; j < V; ++j) a[0][j] = 0.f;
#pragma unroll
        for (int i = 0; i < NU; ++i) {
          put<T, V, RAG>(dx + u.a[i], a[0]);
          put<T, V, RAG>(dx + u.b[i], a[0]);
        }
        if (it + 1 == last && next.held) load(next.row, begin);
        continue;
      }
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        unpack<T, V>(qa[i], a[i]);
        unpack<T, V>(qb[i], b[i]);
        unpack<T, V>(ga[i], da[i]);
        unpack<T, V>(gb[i], db[i]);
      }
      if (it + 1 < last) load(row, it + 1);  // the next heads on their way
      else if (next.held) load(next.row, begin);
#pragma unroll
      for (int i = 0; i < NU; ++i) turn_unit<V, ADJ>(da[i], db[i], turn[i], -1.f, u.pair[i] >= 0);
      auto gradient = [&](const Gains<V, NU>& w, float (&wa)[NU][V], float (&wb)[NU][V]) {
        float s = 0.f, m = 0.f;
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const bool ca = u.in[i] && u.counts_a(i, j), cb = u.in[i] && u.counts_b(i, j);
            const float va = ca ? a[i][j] : 0.f, vb = cb ? b[i][j] : 0.f;
            s = fmaf(va, va, fmaf(vb, vb, s));
            m = fmaf(va, da[i][j] * w.a[i][j], fmaf(vb, db[i][j] * w.b[i][j], m));
          }
        const float r = rsqrtf(team_sum(s, p.lgteam) * p.inv + p.eps);
        m = team_sum(m, p.lgteam) * p.inv * r * r;
        const bool own = h.mine < p.heads[h.k];
#pragma unroll
        for (int i = 0; i < NU; ++i)
#pragma unroll
          for (int j = 0; j < V; ++j) {
            wa[i][j] += own && u.in[i] && u.counts_a(i, j) ? da[i][j] * (a[i][j] * r) : 0.f;
            wb[i][j] += own && u.in[i] && u.counts_b(i, j) ? db[i][j] * (b[i][j] * r) : 0.f;
            da[i][j] = r * (da[i][j] * w.a[i][j] - a[i][j] * m);
            db[i][j] = r * (db[i][j] * w.b[i][j] - b[i][j] * m);
          }
      };
      if (p.norm) {
        if (h.k == 0) gradient(wq, dwa[0], dwb[0]);
        else gradient(wk, dwa[1], dwb[1]);
      }
#pragma unroll
      for (int i = 0; i < NU; ++i) {
        if (NU == 1 || u.in[i]) {
          put<T, V, RAG>(dx + u.a[i], da[i]);
          put<T, V, RAG>(dx + u.b[i], db[i]);
        }
      }
    }
    now = next;
  }
  if (p.part == nullptr) return;
  // over the wave's teams, then over the block's waves, in order
  __syncthreads();
  float* sum = reinterpret_cast<float*>(lds);
#pragma unroll
  for (int k = 0; k < 2; ++k)
#pragma unroll
    for (int i = 0; i < NU; ++i)
#pragma unroll
      for (int j = 0; j < V; ++j) {
        float va = dwa[k][i][j], vb = dwb[k][i][j];
        for (int d = team; d < 64; d *= 2) {
          va += __shfl_xor(va, d);
          vb += __shfl_xor(vb, d);
        }
        if (lane < team && u.in[i]) {
          if (u.counts_a(i, j)) sum[(wave * 2 + k) * p.D + u.a[i] + j] = va;
          if (u.counts_b(i, j)) sum[(wave * 2 + k) * p.D + u.b[i] + j] = vb;
        }
      }
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * p.D; c += 256)
    p.part[int64_t(blockIdx.x) * 2 * p.D + c] = (sum[c] + sum[2 * p.D + c]) + (sum[4 * p.D + c] + sum[6 * p.D + c]);
}

// ---------------------------------------------------------------- launches
bool whole(const void* p, int64_t ld, size_t e) { return p == nullptr || rows_aligned(p, ld, e, 16); }
template <typename T, int V, int NU, bool RAG, bool ADJ>
hipError_t launch_one(const Plan& h, bool backward, hipStream_t s) {
  const dim3 grid(uint32_t(h.blocks)), block(256);
  const size_t table = size_t(4) * (h.p.R / 2) * sizeof(float2);
  if (!backward) {
    rope_kernel<T, V, NU, RAG, ADJ><<<grid, block, table, s>>>(h.p);
  } else {
    const size_t sums = size_t(8) * h.p.D * 4;
    rope_backward_kernel<T, V, NU, RAG, ADJ><<<grid, block, table > sums ? table : sums, s>>>(h.p);
  }
  return hipGetLastError();
}
// The instance that holds V and NU; a plan that none does is an error, never fewer units.
template <typename T, int W, bool ADJ>
hipError_t launch_any(const Plan& h, bool backward, hipStream_t s) {
  if (h.p.units > 64 * h.NU) return hipErrorInvalidValue;
  if (h.V == 1 && h.NU == 1) return launch_one<T, 1, 1, false, ADJ>(h, backward, s);
  if (h.V == 1 && h.NU == 8) return launch_one<T, 1, 8, false, ADJ>(h, backward, s);
  if constexpr (W == 4) {
    if (h.V == W && h.NU == 2) return h.rag ? launch_one<T, W, 2, true, ADJ>(h, backward, s) : launch_one<T, W, 2, false, ADJ>(h, backward, s);
  }
  if (h.V == W && h.NU == 1) return h.rag ? launch_one<T, W, 1, true, ADJ>(h, backward, s) : launch_one<T, W, 1, false, ADJ>(h, backward, s);
  return hipErrorInvalidValue;
}
hipError_t launch(const m3_qk_norm_rope_args& a, const Plan& h, bool backward, hipStream_t s) {
  if (a.in_dtype == M3_BF16) return a.adjacent ? launch_any<bf16_t, 8, true>(h, backward, s) : launch_any<bf16_t, 8, false>(h, backward, s);
  return a.adjacent ? launch_any<float, 4, true>(h, backward, s) : launch_any<float, 4, false>(h, backward, s);
}

}  // namespace

hipError_t launch_rope(const m3_qk_norm_rope_args& a, hipStream_t s) {
  Plan h = plan_of(a, false);
  const size_t e = a.in_dtype == M3_BF16 ? 2 : 4;
  h.p.y[0] = a.q_out;
  h.p.y[1] = a.k_out;
  h.rag = h.rag || (size_t(a.D) * e) % 16 != 0 || !whole(a.q, a.q_ld, e) || !whole(a.k, a.k_ld, e) || !whole(a.q_out, 0, e) ||
          !whole(a.k_out, 0, e);
  return launch(a, h, false, s);
}

size_t rope_backward_workspace(const m3_qk_norm_rope_backward_args& b) {
  const m3_qk_norm_rope_args& a = b.fwd;
  if (!a.norm) return 0;
  return round256(size_t(plan_of(a, true).blocks) * 2 * a.D * 4);
}

hipError_t launch_rope_backward(const m3_qk_norm_rope_backward_args& b, hipStream_t s) {
  const m3_qk_norm_rope_args& a = b.fwd;
  Plan h = plan_of(a, true);
  const size_t e = a.in_dtype == M3_BF16 ? 2 : 4;
  h.p.y[0] = b.dq;
  h.p.y[1] = b.dk;
  h.p.dy[0] = b.dq_out;
  h.p.dy[1] = b.dk_out;
  const bool gains = b.dq_w != nullptr || b.dk_w != nullptr;
  h.p.part = gains ? static_cast<float*>(b.workspace) : nullptr;
  h.rag = h.rag || (size_t(a.D) * e) % 16 != 0 || !whole(a.q, a.q_ld, e) || !whole(a.k, a.k_ld, e) || !whole(b.dq, 0, e) ||
          !whole(b.dk, 0, e) || !whole(b.dq_out, 0, e) || !whole(b.dk_out, 0, e);
  const hipError_t err = launch(a, h, true, s);
  if (err != hipSuccess || !gains) return err;
  ColSum c{};
  c.part = h.p.part;
  c.P = h.blocks;
  c.ncols = 2 * a.D;
  c.dst[0] = b.dq_w;
  c.dst[1] = b.dk_w;
  c.n[0] = c.n[1] = a.D;
  return launch_colsum(c, s);
}

}  // namespace m3
