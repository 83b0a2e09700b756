// kv4_rules.h -- how attn_kv4_decode takes a call: rows of a block, clusters or dealt tiles, grid and
// shares.  Plain arithmetic on sizes, checked by itself on the CPU.
#pragma once

namespace attn {

constexpr int kKvMaxCtas = 640;  // workspace bound of the decode grids

// Row blocks of 4, 8 or, in bf16, 16 rows, a warpgroup for every four: what a thread does for a tile does not
// grow, and a block of 16 rows is one CTA's (32 requests of 1000 to 16384 tokens, 64 query and 4 key heads: 55 us,
// with 8 rows, 64 and 8 heads, 55; one warpgroup for all of a block's rows 57 and 53, but 19.8 us against 18.1 for 912
// heads of 128 tokens in groups of 8).  (16 rows of fp16 in three terms would take P rows of 192 bytes.)
inline int kv4_rows(int R, bool bf16) { return R <= 4 ? 4 : (R <= 8 || !bf16 ? 8 : 16); }

// CTAs that the GPU holds at once.
inline long long kv4_resident(int rp, bool bf16, int sms) { return (rp == 16 ? 1ll : (rp == 4 && bf16 ? 3ll : 2ll)) * sms; }

// CTAs of the cluster that takes a segment, of `tiles` tiles at most, or 0: the tiles of all
// requests are dealt to all CTAs, and a second kernel joins the parts.  A cluster saves that
// kernel and the sums over the lengths, but a long request among short ones is its few CTAs'
// alone: four tiles to a CTA, eight where there is one request.  (The tiles are the block table's: the
// lengths are on the device.  A table with room for long requests is dealt, however short they are.)  Up to 8 CTAs; 16 where that is one to an
// SM (more such clusters do not fit at once: 24 segments of 4096 tokens 14 us, 9 with 8) and a
// CTA would have more than two tiles.
// Requests of equal length, us by clusters and dealt (bf16, 8 heads, groups of 4, d = 128): one of 1000 tokens
// 5.5 and 8.0, of 8192 8.9 and 11.9, of 16384 13.5 and 13.3; 12 of 2048 10.1 and 13.5; 24 of 1024 10.7 and
// 13.9.  Of 1 to 2048 tokens, 12: 9.2 and 10.0; of 1 to 4096, eight tiles to a CTA: 12.6 and 11.2.
// `most`: 16, or 8 where the GPU (a part of it) has no 16 SMs together.
constexpr int kKv4MaxCluster = 16;
inline int kv4_cluster(int rp, bool bf16, int sms, int B, long long segs, long long tiles, int most) {
  int c = most > 8 && segs * 16 <= sms && tiles > 16 ? kKv4MaxCluster : 8;
  while (c > 1 && (segs * c > kv4_resident(rp, bf16, sms) || c / 2 >= tiles)) c /= 2;
  return c > 1 && tiles <= (B == 1 ? 8 : 4) * c ? c : 0;
}

// All CTAs resident at once, no more than there can be tiles.
inline int kv4_grid(int rp, bool bf16, int sms, long long max_units) {
  long long g = kv4_resident(rp, bf16, sms);
  if (g > kKvMaxCtas) g = kKvMaxCtas;
  if (g > max_units) g = max_units;
  return (int)(g < 1 ? 1 : g);
}

// Of three CTAs to an SM the last one starts a microsecond after the others and goes 5 % slower:
// four long requests, equal shares: the first two thirds of the CTAs end at 68 us, the others at 73.  Shares
// of 8 and 7: 75.8 us in all, 78.6 with equal ones, 76.7 with 9 and 8, 75.9 with 7 and 6 (64 ragged
// requests 31.7, 32.9, 31.8, 31.5).
inline int kv4_full(int rp, bool bf16, int sms, int grid) { return kv4_resident(rp, bf16, sms) == 3ll * sms && grid == 3 * sms ? 2 * sms : 0; }

}  // namespace attn
