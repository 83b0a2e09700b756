// Walks the ranges of every CTA of a decode from a paged cache as the split kernels do (kv_split.h) and checks that each
// tile of each segment is walked once, that no CTA of the deal is without a range, and that the merge kernel looks for
// every part where it was written and for no other.  Input, a call a line: TS, SC, heads times row blocks, grid,
// CTAs with a full share, B, then B lengths.  Output, a line each: units, CTAs, segments that are cut, 32-bit divisions.
#include <cstdio>
#include <cstdlib>
#include <map>
#include <utility>
#include <vector>

#include "kv_split.h"

using namespace attn;

#define CHECK(x)                                              \
  do {                                                        \
    if (!(x)) {                                               \
      std::fprintf(stderr, "line %d: %s\n", __LINE__, #x);    \
      std::exit(1);                                           \
    }                                                         \
  } while (0)

struct Args {
  const int* lens;
  int width, page_shift, grid, full;
};

template <int TS, int SC>
void check(int Hr, int grid, int full, const std::vector<int>& lens) {
  const Args p = {lens.data(), (int)((1ll << 31) / 128 - 2), 7, grid, full};
  const int B = (int)lens.size();
  long long total = 0;
  for (int b = 0; b < B; ++b) total += seg_units<SC>(kv_tiles<TS>(kv_len(p, b)));
  const Deal deal(p, total * Hr);
  CHECK(deal.n <= grid && deal.n <= deal.units && (deal.n == grid || deal.n == deal.units));
  struct Piece {
    int c, slot, t0, t1;
  };
  std::map<std::pair<int, int>, std::vector<Piece>> pieces;
  std::map<std::pair<int, int>, int> written;  // (CTA, slot)
  long long at = 0;                            // first unit of request b
  int b = 0;
  for (long long c = 0; c < deal.n; ++c) {
    const long long u0 = deal.start(c), u1 = deal.start(c + 1);
    CHECK(u0 < u1 && (c > 0 || u0 == 0) && (c + 1 < deal.n || u1 == deal.units));
    CHECK(deal.owner(u0) == c && deal.owner(u1 - 1) == c && deal.owner((u0 + u1) / 2) == c);
    int n = seg_units<SC>(kv_tiles<TS>(kv_len(p, b)));
    while (u0 >= at + (long long)n * Hr) {
      at += (long long)n * Hr;
      n = seg_units<SC>(kv_tiles<TS>(kv_len(p, ++b)));
    }
    Walk w = {b, (int)((u0 - at) / n), (int)((u0 - at) % n), u1 - u0};
    Seg s;
    for (int k = 0; next_seg<TS, SC>(p, Hr, w, s); ++k) {
      CHECK(s.b < B && s.hr < Hr && s.t0 < s.t1 && s.t1 <= s.nt && s.len == kv_len(p, s.b));
      const int slot = k > 0 ? 1 : 0;
      if (s.t1 - s.t0 < s.nt) CHECK((++written[{(int)c, slot}] == 1));
      pieces[{s.b, s.hr}].push_back({(int)c, slot, s.t0, s.t1});
    }
  }
  long long first = 0, cut = 0;
  for (int q = 0; q < B; ++q) {
    const int nt = kv_tiles<TS>(kv_len(p, q));
    for (int hr = 0; nt && hr < Hr; ++hr) {
      const std::vector<Piece>& v = pieces[{q, hr}];
      const Parts m = kv_parts<SC>(deal, first + (long long)hr * seg_units<SC>(nt), nt);
      CHECK(m.c1 - m.c0 + 1 == (int)v.size());
      int t = 0;
      for (size_t i = 0; i < v.size(); ++i) {
        CHECK(v[i].c == m.c0 + (int)i && v[i].t0 == t);
        if (v.size() > 1) CHECK(v[i].slot == (i == 0 ? m.s0 : 0));
        t = v[i].t1;
      }
      CHECK(t == nt);
      cut += v.size() > 1;
    }
    first += (long long)seg_units<SC>(nt) * Hr;
  }
  std::printf("%lld %lld %lld %d\n", deal.units, deal.n, cut, (int)deal.small);
}

int main() {
  int TS, SC, Hr, grid, full, B;
  while (std::scanf("%d %d %d %d %d %d", &TS, &SC, &Hr, &grid, &full, &B) == 6) {
    std::vector<int> lens(B);
    for (int& x : lens) CHECK(std::scanf("%d", &x) == 1);
    CHECK((TS == 7 || TS == 8) && (SC == 1 || SC == 2));
    if (TS == 7) SC == 1 ? check<7, 1>(Hr, grid, full, lens) : check<7, 2>(Hr, grid, full, lens);
    else SC == 1 ? check<8, 1>(Hr, grid, full, lens) : check<8, 2>(Hr, grid, full, lens);
  }
}
