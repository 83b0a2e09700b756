// Walks every item of packed batches as the backward's kernels do (var_split.h) and
// checks that each chunk of each key tile is one item, whichever way items are numbered,
// and that the bounds the host relies on hold.  Input, a batch a line: causal, Hq, Hkv,
// SMs, B, then B query and B key lengths.  Output, a line each: items, parts, CTAs.
#include <cstdio>
#include <cstdlib>
#include <set>
#include <utility>
#include <vector>

#include "var_split.h"

using namespace attn;

#define CHECK(x)                                              \
  do {                                                        \
    if (!(x)) {                                               \
      std::fprintf(stderr, "line %d: %s\n", __LINE__, #x);    \
      std::exit(1);                                           \
    }                                                         \
  } while (0)

int main() {
  int causal, Hq, Hkv, sms, B;
  while (std::scanf("%d %d %d %d %d", &causal, &Hq, &Hkv, &sms, &B) == 5) {
    std::vector<int> lq(B), lk(B);
    for (int& x : lq) CHECK(std::scanf("%d", &x) == 1);
    for (int& x : lk) CHECK(std::scanf("%d", &x) == 1);
    const int G = Hq / Hkv;
    long long Tq = 0, Tk = 0, steps = 0, items = 0, parts = 0;
    for (int b = 0; b < B; ++b) {
      Tq += lq[b];
      Tk += lk[b];
      steps += var_steps(lq[b], lk[b], causal);
    }
    const int a = var_chunk(steps, Hq, G);
    for (int b = 0; b < B; ++b) {
      if (lq[b] == 0) continue;
      const VarSplit sp(lq[b], lk[b], a, causal);
      long long per_head = 0;
      for (int tk = 0; tk < sp.nkt; ++tk) {
        const int nqs = (lq[b] + 63) / 64, n = causal && 2 * tk + 2 < nqs ? 2 * tk + 2 : nqs;
        CHECK(sp.items(tk) == (n + 2 * a - 1) / (2 * a));
        CHECK(sp.items_before(tk) == per_head);
        CHECK((sp.items(tk) > 1) == (tk >= sp.first_split()));
        if (sp.items(tk) > 1) CHECK(sp.parts_before(tk) == per_head - sp.items_before(sp.first_split()));
        per_head += sp.items(tk);
      }
      CHECK(sp.count(-1) == per_head);
      int tk = 0, chunk = 0;
      for (int by_class = 0; by_class < 2; ++by_class) {
        std::set<std::pair<int, int>> seen;
        for (int c = by_class ? 0 : -1; c < (by_class ? kVarClasses : 0); ++c)
          for (int e = 0, n = sp.count(c); e < n; ++e) {
            sp.pick(c, e, &tk, &chunk);
            CHECK(tk >= 0 && tk < sp.nkt && chunk >= 0 && chunk < sp.items(tk));
            CHECK(seen.insert({tk, chunk}).second);
          }
        CHECK((long long)seen.size() == per_head);
      }
      items += per_head * Hkv;
      parts += (long long)sp.parts_before(sp.nkt) * Hkv;
    }
    const int ctas = bwd_varlen_grid(B, Tq, Tk, G, Hkv, sms);
    CHECK(parts <= kVarMaxParts);
    CHECK(parts == 0 || var_may_split(Tq, G));
    CHECK(ctas >= 1 && ctas <= sms);
    CHECK(ctas == sms || ctas >= items);
    std::printf("%lld %lld %d\n", items, parts, ctas);
  }
  return 0;
}
