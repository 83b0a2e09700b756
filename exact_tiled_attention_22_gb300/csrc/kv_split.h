// kv_split.h -- how decoding from a paged cache deals its work to the CTAs and
// where the merge kernel finds their parts: plain arithmetic, checked by itself on the CPU.
//
// All tiles (2^TS tokens of one head group of one request) are numbered and every
// CTA takes an equal consecutive range, whatever the lengths are; the range may
// begin and end inside a (request, head), whose parts then meet in the merge
// kernel.
#pragma once

#include <cstdint>

#include "var_split.h"

namespace attn {

// What a segment (a request's tiles of one head group) costs besides its tiles, SC
// in tiles: its query terms, the first S and the last O^T, during which nothing
// else of the CTA runs.  Units are counted with it, tile t of a segment being
// unit SC + t, so that a CTA with many short requests gets fewer tiles.  Both
// caches' figures stand at kKv8SegCost and kv4_seg_cost.
template <int SC>
ATTN_HD inline int seg_units(int nt) { return nt > 0 ? nt + SC : 0; }

// The units are dealt to n = min(grid, units) CTAs, so that none of those has an empty range (the merge
// kernel reads a part from each CTA of a segment): in equal shares, or, where `full` says so and there
// are units enough, with shares of kFull to the first `full` CTAs and of kLate to the others.
// (Divisions in 32 bits where the products fit: 64-bit ones took 0.3 us of a short decoding step.)
constexpr int kFull = 8, kLate = 7;
struct Deal {
  long long units, n, all;  // all: the sum of the shares
  long long full;           // 0: equal shares of 1
  bool small;
  template <typename Args>
  ATTN_HD Deal(const Args& p, long long units_) : units(units_), n(var_min((long long)p.grid, units_)) {
    full = p.full && units >= 4ll * p.grid ? p.full : 0;
    all = full ? full * kFull + (n - full) * kLate : n;
    small = units <= 0xffffffffll / var_max(all, 1ll);
  }
  // The first unit of CTA c's range.
  ATTN_HD long long start(long long c) const {
    const long long x = !full ? c : (c < full ? c * kFull : full * kFull + (c - full) * kLate);
    return small ? (long long)((uint32_t)x * (uint32_t)units / (uint32_t)all) : x * units / all;
  }
  // The CTA whose range holds unit u: the last one that starts at u or before.
  ATTN_HD long long owner(long long u) const {
    const long long y = small ? (long long)((((uint32_t)u + 1) * (uint32_t)all - 1) / (uint32_t)units) : ((u + 1) * all - 1) / units;
    if (!full) return y;
    return y < full * kFull ? (uint32_t)y / kFull : full + (uint32_t)(y - full * kFull) / kLate;
  }
};

template <typename Args>
ATTN_HD inline int kv_len(const Args& p, int b) {
  const long long cap = (long long)p.width << p.page_shift;
  return (int)var_min(var_max((long long)p.lens[b], 0ll), cap);
}

// Tiles of a request of `len` tokens.
template <int TS>
ATTN_HD inline int kv_tiles(int len) { return (len + (1 << TS) - 1) >> TS; }

// Walks the (request, head, row block) segments of a CTA's range: `left` units
// from unit v of segment (b, hr) on.
struct Walk {
  int b, hr, v;
  long long left;
};
// The next segment of which the range holds tiles [t0, t1); false at the end.
struct Seg {
  int b, hr, len, nt, t0, t1;
};
template <int TS, int SC, typename Args>
ATTN_HD inline bool next_seg(const Args& p, int Hr, Walk& w, Seg& s) {
  while (w.left > 0) {
    s.len = kv_len(p, w.b);
    s.nt = kv_tiles<TS>(s.len);
    const int n = seg_units<SC>(s.nt);
    if (n == 0) {  // (a request without tokens has no units)
      ++w.b;
      w.hr = 0;
      w.v = 0;
      continue;
    }
    const int end = (int)var_min((long long)n, w.v + w.left);
    s.b = w.b;
    s.hr = w.hr;
    s.t0 = var_max(0, w.v - SC);
    s.t1 = var_max(0, end - SC);
    w.left -= end - w.v;
    w.v = 0;
    if (++w.hr == Hr) {
      w.hr = 0;
      ++w.b;
    }
    if (s.t0 < s.t1) return true;
  }
  return false;
}

// Where the merge kernel finds a segment of nt > 0 tiles whose units begin at u0: in the parts of CTAs c0 .. c1, the
// first one's in its second slot if its range began earlier, all others' in their first.  (c0 == c1: that CTA wrote
// the result itself.)
struct Parts {
  int c0, c1, s0;
};
template <int SC>
ATTN_HD inline Parts kv_parts(const Deal& deal, long long u0, int nt) {
  Parts r;
  r.c0 = (int)deal.owner(u0 + SC);
  r.c1 = (int)deal.owner(u0 + SC + nt - 1);
  r.s0 = deal.start(r.c0) < u0 ? 1 : 0;
  return r;
}

}  // namespace attn
