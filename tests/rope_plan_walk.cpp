// Walks the plans of the norm and rotation of queries and keys over every head size and
// rotated part: each element of a head is counted exactly once, written, and no place
// outside of the head or of the table of angles is touched.  Prints what is wrong.
#include <cstdio>
#include <cstring>
#include <initializer_list>

#include "rotary_plan.hpp"

using namespace m3::rope;

static long wrong = 0, walked = 0;
static void say(const char* what, const RopeP& p, int V, int NU, bool rag, bool adj, int at) {
  if (++wrong <= 20) std::printf("%s: D %d R %d V %d NU %d rag %d adjacent %d at %d\n", what, p.D, p.R, V, NU, rag, adj, at);
}

template <int V, int NU, bool RAG, bool ADJ>
static void walk(const RopeP& p) {
  static int counted[1024];
  static bool written[1024];
  std::memset(counted, 0, sizeof counted);
  std::memset(written, 0, sizeof written);
  ++walked;
  const int team = 1 << p.lgteam, half = p.R / 2;
  for (int lane = 0; lane < team; ++lane) {
    const Units<V, NU, RAG, ADJ> u(p, lane, team);
    for (int i = 0; i < NU; ++i) {
      if (u.a[i] < 0 || u.b[i] < 0 || u.a[i] + V > p.D || u.b[i] + V > p.D) {
        say("outside", p, V, NU, RAG, ADJ, u.a[i]);
        continue;
      }
      if (u.pair[i] >= 0 && u.pair[i] + V > half) say("angles", p, V, NU, RAG, ADJ, u.pair[i]);
      if (!u.in[i]) continue;
      for (int j = 0; j < V; ++j) {
        const int a = u.a[i] + j, b = u.b[i] + j;
        written[a] = written[b] = true;
        counted[a] += u.counts_a(i, j);
        counted[b] += u.counts_b(i, j);
        if ((a < p.R) != (u.pair[i] >= 0) || (b < p.R) != (u.pair[i] >= 0)) say("range", p, V, NU, RAG, ADJ, a);
        if (u.pair[i] >= 0 && !ADJ && (a != u.pair[i] + j || b != half + u.pair[i] + j)) say("partners", p, V, NU, RAG, ADJ, a);
        if (u.pair[i] >= 0 && ADJ && (a != 2 * u.pair[i] + j || b != 2 * u.pair[i] + V + j)) say("partners", p, V, NU, RAG, ADJ, a);
      }
    }
  }
  for (int c = 0; c < p.D; ++c)
    if (counted[c] != 1 || !written[c]) say("counted", p, V, NU, RAG, ADJ, c);
}
template <int V, int NU>
static void both(const Plan& h) {
  if constexpr (V == 1) {
    walk<V, NU, false, false>(h.p);
    walk<V, NU, false, true>(h.p);
  } else {
    if (!h.rag) {
      walk<V, NU, false, false>(h.p);
      walk<V, NU, false, true>(h.p);
    }
    walk<V, NU, true, false>(h.p);  // also by alignment
    walk<V, NU, true, true>(h.p);
  }
}

int main() {
  for (int dtype : {int(M3_F32), int(M3_BF16)})
    for (int D = 1; D <= 1024; ++D)
      for (int R = 0; R <= D; R += 2) {
        m3_qk_norm_rope_args a{};
        a.Bt = 1, a.L = 3, a.H = 5, a.Hk = 2, a.D = D, a.R = R, a.in_dtype = dtype, a.norm = 1;
        const Plan h = plan_of(a, false);
        if (h.p.units > 64 * h.NU || h.p.units < 1 || (1 << h.p.lgteam) * h.NU < h.p.units) say("units", h.p, h.V, h.NU, h.rag, false, h.p.units);
        const int word = dtype == M3_BF16 ? 8 : 4;
        // the kernels' instances
        if (h.V == 1 && h.NU == 1) both<1, 1>(h);
        else if (h.V == 1 && h.NU == 8) both<1, 8>(h);
        else if (h.V == 4 && word == 4 && h.NU == 1) both<4, 1>(h);
        else if (h.V == 4 && word == 4 && h.NU == 2) both<4, 2>(h);
        else if (h.V == 8 && word == 8 && h.NU == 1) both<8, 1>(h);
        else say("no instance", h.p, h.V, h.NU, h.rag, false, 0);
      }
  std::printf("%ld plans walked, %ld wrong\n", walked, wrong);
  return wrong != 0;
}
