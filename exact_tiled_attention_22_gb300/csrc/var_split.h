// var_split.h -- how the work of a packed batch's backward is cut into items: pure
// arithmetic on lengths, shared by the kernels and the host code that sizes grids and
// workspaces, and checked by itself on the CPU.
#pragma once

#ifdef __CUDACC__
#define ATTN_HD __host__ __device__
#else
#define ATTN_HD
#endif

namespace attn {

// SMs of a GB300, for what must not depend on the device of a call: sizes of workspaces,
// the split of the work (and with it the order of sums).
constexpr int kSms = 152;

constexpr int kVarClasses = 9;                // classes of items by length: whole chunks, eighths of one
constexpr int kVarChunks = 2 * kSms;          // equal chunks a batch's steps are cut into
constexpr int kVarMaxParts = 2 * kVarChunks;  // a split tile of n steps has < 2 n / (all steps / kVarChunks) parts

template <typename T>
ATTN_HD constexpr T var_min(T x, T y) { return y < x ? y : x; }
template <typename T>
ATTN_HD constexpr T var_max(T x, T y) { return x < y ? y : x; }

// How a packed batch's key tiles are cut into items.  Tile tk (from the end) of a
// sequence has G min(nqs, 2 tk + 2) steps (causal; else G nqs); an item takes
// 2 G a of them, so tile tk has tk / a + 1 items while the causal limit binds
// (tk < n1) and C above, and the items before a tile have a closed form.  `a`
// comes from the whole batch's steps (var_chunk): about kVarChunks equal chunks,
// twice the SMs, and never fewer than 32 steps in one, so that the longest item
// is a fraction of the kernel's time however the lengths are spread (without
// the cut the first tile of the longest sequence took as long as the rest of
// the batch: 4096 tokens, 4 heads to a key head, 256 steps, 0.24 ms).
// With heads that share a key head, where most of the work is in split tiles, items
// are numbered by classes of their length, kVarClasses in all: whole chunks of 2 G a
// steps first, then what is left of the tiles, by eighths of a chunk from the longest
// on.  (The blocks take two or three items each, so a chunk that is claimed after
// short rests makes the last ones late: 8192 tokens, 8 / 2 heads, d 128, 291 us tile by
// tile, 249 by classes; three texts of 3000 141 and 124.)  Others are numbered tile by
// tile, which are found sooner: few of their tiles are split, and the classes gained them
// nothing (4096 tokens, 12 heads with keys of their own, d 64: 88 us, 90 by classes).
struct VarSplit {
  int nkt, n1, a, C, nqs;
  ATTN_HD VarSplit(int lq, int lk, int a_, int causal) {
    nqs = (lq + 63) >> 6;
    nkt = (lk + 127) >> 7;
    n1 = causal ? var_min(nkt, nqs >> 1) : 0;
    a = a_;
    C = (nqs + 2 * a - 1) / (2 * a);
  }
  // of a tile beyond the causal limit: whole chunks, and the eighths (1 .. 8) of its rest or 0
  ATTN_HD int fC() const { return nqs == C * 2 * a ? C : C - 1; }
  ATTN_HD int lC() const { return ((nqs - fC() * 2 * a) * 4 + a - 1) / a; }
  // whole chunks of the tiles before tile n
  ATTN_HD int full_before(int n) const {
    const int m = var_min(n, n1), k = m / a, r = m - k * a;
    return a * (k * (k - 1) / 2) + k * (r + 1) + (n - m) * fC();
  }
  ATTN_HD int full(int tk) const { return tk < n1 ? (tk + 1) / a : fC(); }
  // rests of class c: (tk + 1) % a in (lo, hi], l = 9 - c eighths
  ATTN_HD int lo(int l) const { return (l - 1) * a / 8; }
  ATTN_HD int hi(int l) const { return l == 8 ? a - 1 : l * a / 8; }
  ATTN_HD int count1(int l) const {  // of the tiles at the causal limit
    const int w = hi(l) - lo(l), k = n1 / a, r = n1 - k * a;
    return k * w + var_min(var_max(r - lo(l), 0), w);
  }
  // items of class c, or of all (c = -1)
  ATTN_HD int count(int c) const {
    if (c < 0) return items_before(nkt);
    return c == 0 ? full_before(nkt) : count1(9 - c) + (nkt > n1 && lC() == 9 - c ? nkt - n1 : 0);
  }
  // tile and chunk of the e-th of them, the first tiles first
  ATTN_HD void pick(int c, int e, int* tk, int* chunk) const {
    if (c <= 0) {
      int at = 0, end = nkt - 1;
      while (at < end) {
        const int mid = (at + end + 1) >> 1;
        if ((c < 0 ? items_before(mid) : full_before(mid)) <= e) at = mid; else end = mid - 1;
      }
      *tk = at;
      *chunk = e - (c < 0 ? items_before(at) : full_before(at));
    } else {
      const int l = 9 - c, n = count1(l), w = hi(l) - lo(l);
      *tk = e < n ? e / w * a + lo(l) + e % w : n1 + e - n;
      *chunk = full(*tk);
    }
  }
  ATTN_HD int items(int tk) const { return tk < n1 ? tk / a + 1 : C; }
  ATTN_HD int items_before(int n) const {
    const int m = var_min(n, n1), k = m / a, r = m - k * a;
    return a * (k * (k + 1) / 2) + r * (k + 1) + (n - m) * C;
  }
  // tiles from here on have several items
  ATTN_HD int first_split() const { return C >= 2 ? var_min(a, n1) : nkt; }
  ATTN_HD int parts_before(int n) const {
    const int f = first_split();
    return n > f ? items_before(n) - items_before(f) : 0;
  }
};

// Steps (64 query rows on a key tile) of one query head in a sequence.
ATTN_HD inline long long var_steps(int lq, int lk, int causal) {
  const int nqs = (lq + 63) >> 6, nkt = (lk + 127) >> 7, n1 = causal ? var_min(nkt, nqs >> 1) : 0;
  return (long long)n1 * (n1 + 1) + (long long)(nkt - n1) * nqs;
}

// Least `a`: 32 steps to a chunk, or two per head of the group.
ATTN_HD inline long long var_chunk_min(int G) { return (16ll + G - 1) / G; }

// `a` of a batch of `steps` steps to each of H query heads, G to a key head (no
// more than the 2^20 steps of the longest sequence).
ATTN_HD inline int var_chunk(long long steps, int H, int G) {
  const long long total = steps * H, unit = 2ll * G * kVarChunks;
  return (int)var_min(1ll << 19, var_max(var_chunk_min(G), (total + unit - 1) / unit));
}

// Whether any tile can be split: not while a sequence of all Tq queries has no more
// than one chunk of steps.
inline bool var_may_split(long long Tq, int G) { return (Tq + 63) / 64 > 2 * var_chunk_min(G); }

// CTAs of the persistent main kernel: no more than there can be items, which are the
// tiles of the worst split of the keys into sequences and the parts of those that are cut.
// (The tiles alone are too few where there are few keys or heads: first to last kernel,
// d 128, one causal text of 8192 tokens with one head 57 us, 105 with a block for every
// tile; 65536 queries on 128 keys, 4 heads, 161 and 707; 16384 on 128, 8 heads, 96 and 201.)
inline int bwd_varlen_grid(int B, long long Tq, long long Tk, int G, int Hkv, int sms) {
  const long long items = (Tk / 128 + B) * Hkv + (var_may_split(Tq, G) ? kVarMaxParts : 0);
  return (int)var_min((long long)sms, items);
}

}  // namespace attn
