// Plans of the norm and rotation of queries and keys: into which units a head is cut, which lanes
// hold them and which elements each counts.  No device code, so that every size can be walked on
// the host.
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "m3ssm.h"

namespace m3 {
namespace rope {

struct RopeP {
  const void* x[2];   // q, k
  void* y[2];         // outputs, or in the backward dx
  const void* dy[2];  // backward
  const float* w[2];
  int64_t ld[2];
  int heads[2], its[2];  // turns of a wave over q's and k's heads
  const float* freqs;
  const int32_t* positions;
  const int32_t* lengths;
  float* part;  // backward: [blocks][2 D], or null
  int64_t rows, walkers;
  int L, D, R, start, norm, lgteam, units, rot_units, splits;
  float eps, inv;
};

__host__ __device__ __forceinline__ int least(int a, int b) { return a < b ? a : b; }
__host__ __device__ __forceinline__ int most(int a, int b) { return a > b ? a : b; }

// A lane's units (see rotary.hip).
template <int V, int NU, bool RAG, bool ADJ>
struct Units {
  int a[NU], b[NU];  // the words' columns
  int skip[NU];      // pairs (behind R: elements) at the front that another unit counts
  int pair[NU];      // first pair, or -1 behind R
  bool in[NU], once[NU];  // once: b repeats a
  __host__ __device__ __forceinline__ Units(const RopeP& p, int lane, int team) {
#pragma unroll
    for (int i = 0; i < NU; ++i) {
      int u = lane + i * team;
      in[i] = u < p.units;
      u = in[i] ? u : 0;
      once[i] = false;
      if (u < p.rot_units) {
        const int half = p.R / 2, s = RAG ? least(u * V, half - V) : u * V;
        skip[i] = u * V - s;
        pair[i] = s;
        a[i] = ADJ ? 2 * s : s;
        b[i] = ADJ ? 2 * s + V : half + s;
      } else {
        const int rest = p.D - p.R, at = (u - p.rot_units) * 2 * V, s = RAG || V == 1 ? most(0, least(at, rest - 2 * V)) : at;
        skip[i] = at - s;
        pair[i] = -1;
        a[i] = p.R + s;
        b[i] = a[i] + V;
        if (V == 1 && rest == 1) {
          b[i] = a[i];
          once[i] = true;
        }
      }
    }
  }
  // whether element j of word a (of word b) is this unit's to count
  __host__ __device__ __forceinline__ bool counts_a(int i, int j) const {
    if (V > 1 && !RAG) return true;
    return pair[i] < 0 || !ADJ ? j >= skip[i] : j / 2 >= skip[i];
  }
  __host__ __device__ __forceinline__ bool counts_b(int i, int j) const {
    if (V > 1 && !RAG) return true;
    if (once[i]) return false;
    if (pair[i] < 0) return V + j >= skip[i];
    return ADJ ? (V + j) / 2 >= skip[i] : j >= skip[i];
  }
};

struct Plan {
  int V, NU;
  bool rag;
  RopeP p;
  int64_t blocks;
};
inline int lg2_up(int v) {
  int l = 0;
  while ((1 << l) < v) ++l;
  return l;
}
// The units that a lane of the kernels holds at most: of words of 16 bytes one in bf16 and two in
// fp32; of single elements eight, which is every head.
inline int most_units(int V) { return V == 1 ? 8 : V == 4 ? 2 : 1; }
inline void cut(RopeP& p, int V) {
  p.rot_units = (p.R / 2 + V - 1) / V;
  p.units = p.rot_units + (p.D - p.R + 2 * V - 1) / (2 * V);
}

// The words: 16 bytes wherever both ranges of a head hold a unit of them and a wave's lanes hold
// all units, else single elements (heads of 1011 elements and more of which both ranges end
// inside a word are 65 units in bf16 and 129 in fp32).  Tokens over waves; with few tokens,
// their heads over several.
inline Plan plan_of(const m3_qk_norm_rope_args& a, bool backward) {
  Plan h{};
  RopeP& p = h.p;
  const size_t e = a.in_dtype == M3_BF16 ? 2 : 4;
  const int word = int(16 / e), rest = a.D - a.R;
  p.D = a.D;
  p.R = a.R;
  h.V = (a.R == 0 || a.R >= 2 * word) && (rest == 0 || rest >= 2 * word) ? word : 1;
  cut(p, h.V);
  if (p.units > 64 * most_units(h.V)) {
    h.V = 1;
    cut(p, h.V);
  }
  h.rag = (a.R / 2) % word != 0 || rest % (2 * word) != 0;
  p.lgteam = lg2_up(p.units < 64 ? p.units : 64);
  h.NU = p.units <= 64 ? 1 : most_units(h.V);
  p.x[0] = a.q;
  p.x[1] = a.k;
  p.w[0] = a.q_w;
  p.w[1] = a.k_w;
  p.ld[0] = a.q_ld;
  p.ld[1] = a.k_ld;
  p.heads[0] = a.H;
  p.heads[1] = a.Hk;
  const int teams = 64 >> p.lgteam;
  for (int i = 0; i < 2; ++i) p.its[i] = (p.heads[i] + teams - 1) / teams;
  p.freqs = a.freqs;
  p.positions = a.positions;
  p.lengths = a.lengths;
  p.rows = int64_t(a.Bt) * a.L;
  p.L = a.L;
  p.start = a.start;
  p.norm = a.norm;
  p.eps = a.eps;
  p.inv = 1.f / float(a.D);
  const int all = p.its[0] + p.its[1];
  const int64_t want = (2048 + p.rows - 1) / p.rows;
  p.splits = int(want < all ? want : all);
  // A wave's start (gains, rates) is worth a few tokens' time: four tokens each where that still
  // leaves two waves a SIMD (7685 tokens of 9 heads of 80, fp32, uneven: 13 us, one each 16).
  const int64_t most = backward ? 4096 : 8192, few = p.rows / 4 < 2048 ? 2048 : p.rows / 4;
  p.walkers = p.rows < few ? p.rows : few;
  if (p.walkers > most) p.walkers = most;
  h.blocks = (p.walkers * p.splits + 3) / 4;
  return h;
}

}  // namespace rope
}  // namespace m3
