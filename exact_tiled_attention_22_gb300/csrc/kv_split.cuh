// kv_split.cuh -- how decoding from a paged cache deals its work to the CTAs:
// shared by the cache in 8 bits (attn_kv8.cu) and in 4 bits (attn_kv4.cu), whose
// parts one merge kernel joins.
//
// All tiles (2^TS tokens of one head group of one request) are numbered and every
// CTA takes an equal consecutive range, whatever the lengths are; the range may
// begin and end inside a (request, head), whose parts then meet in the merge
// kernel.
#pragma once

#include "kernels.h"

namespace attn {
namespace {

// What a segment (a request's tiles of one head group) costs besides its tiles, SC
// in tiles: its query terms, the first S and the last O^T, during which nothing
// else of the CTA runs.  Units are counted with it, tile t of a segment being
// unit SC + t, so that a CTA with many short requests gets fewer tiles.  Both
// caches' figures stand at kKv8SegCost and kv4_seg_cost.
template <int SC>
__device__ __forceinline__ int seg_units(int nt) { return nt > 0 ? nt + SC : 0; }

// The units are dealt to n = min(grid, units) CTAs, so that none of those has an empty range (the merge
// kernel reads a part from each CTA of a segment): in equal shares, or, where `full` says so and there
// are units enough, with shares of kFull to the first `full` CTAs and of kLate to the others.
// (Divisions in 32 bits where the products fit: 64-bit ones took 0.3 us of a short decoding step.)
constexpr int kFull = 8, kLate = 7;
struct Deal {
  long long units, n, all;  // all: the sum of the shares
  long long full;           // 0: equal shares of 1
  bool small;
  __device__ __forceinline__ Deal(const KvDecArgs& p, long long units_) : units(units_), n(min((long long)p.grid, units_)) {
    full = p.full && units >= 4ll * p.grid ? p.full : 0;
    all = full ? full * kFull + (n - full) * kLate : n;
    small = units <= 0xffffffffll / max(all, 1ll);
  }
  // The first unit of CTA c's range.
  __device__ __forceinline__ long long start(long long c) const {
    const long long x = !full ? c : (c < full ? c * kFull : full * kFull + (c - full) * kLate);
    return small ? (long long)((uint32_t)x * (uint32_t)units / (uint32_t)all) : x * units / all;
  }
  // The CTA whose range holds unit u: the last one that starts at u or before.
  __device__ __forceinline__ long long owner(long long u) const {
    const long long y = small ? (long long)((((uint32_t)u + 1) * (uint32_t)all - 1) / (uint32_t)units) : ((u + 1) * all - 1) / units;
    if (!full) return y;
    return y < full * kFull ? (uint32_t)y / kFull : full + (uint32_t)(y - full * kFull) / kLate;
  }
};

__device__ __forceinline__ int kv_len(const KvDecArgs& p, int b) {
  const long long cap = (long long)p.width << p.page_shift;
  return (int)min(max((long long)p.lens[b], 0ll), cap);
}

// Tiles of a request of `len` tokens.
template <int TS>
__device__ __forceinline__ int kv_tiles(int len) { return (len + (1 << TS) - 1) >> TS; }

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
template <int TS, int SC>
__device__ __forceinline__ bool next_seg(const KvDecArgs& p, int Hr, Walk& w, Seg& s) {
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
    const int end = (int)min((long long)n, w.v + w.left);
    s.b = w.b;
    s.hr = w.hr;
    s.t0 = max(0, w.v - SC);
    s.t1 = max(0, end - SC);
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

// The CTA's range of units [u0, u1) and where it starts: every thread sums the units
// of a run of requests, a scan finds the thread whose run holds u0.  wsum: [THREADS / 32]
// and st: [4] in shared memory; st is valid behind the caller's next barrier.
template <int TS, int SC, int THREADS>
__device__ __forceinline__ void deal_range(const KvDecArgs& p, int Hr, long long* wsum, long long* st) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int per = (p.B + THREADS - 1) / THREADS;
  const int b0 = min(p.B, (int)threadIdx.x * per), b1 = min(p.B, b0 + per);
  long long mine = 0;
  for (int b = b0; b < b1; ++b) mine += seg_units<SC>(kv_tiles<TS>(kv_len(p, b)));
  long long inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long a = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += a;
  }
  if (lane == 31) wsum[warp] = inc;
  __syncthreads();
  long long before = inc - mine, total = 0;
  for (int w = 0; w < THREADS / 32; ++w) {
    if (w < warp) before += wsum[w];
    total += wsum[w];
  }
  const long long units = total * Hr;
  const Deal deal(p, units);
  const bool has = blockIdx.x < deal.n;
  const long long u0 = has ? deal.start(blockIdx.x) : 0;
  const long long u1 = has ? deal.start(blockIdx.x + 1ll) : 0;
  if (threadIdx.x == 0) {
    st[0] = u0;
    st[1] = u1;
  }
  if (u0 < u1 && before * Hr <= u0 && u0 < (before + mine) * Hr) {
    long long at = before;
    for (int b = b0; b < b1; ++b) {
      const int n = seg_units<SC>(kv_tiles<TS>(kv_len(p, b)));
      if (u0 < (at + n) * Hr) {
        const long long in = u0 - at * Hr;  // (below n Hr)
        int* w = reinterpret_cast<int*>(st + 2);
        w[0] = b;
        w[1] = in <= 0xffffffffll ? (int)((uint32_t)in / (uint32_t)n) : (int)(in / n);
        w[2] = (int)(in - (long long)w[1] * n);
        break;
      }
      at += n;
    }
  }
}
// The same by a warp alone, for at most kWarpDealB requests: no barrier, so that a warp that
// copies can begin (17 drafts of 5 tokens: 14.8 -> 14.4 us, 38 x 4096 tokens 39.3 -> 38.9).
constexpr int kWarpDealB = 128;
template <int TS, int SC>
__device__ __forceinline__ Walk deal_warp(const KvDecArgs& p, int Hr) {
  const int lane = threadIdx.x & 31, per = (p.B + 31) / 32, b0 = lane * per;
  uint32_t n[kWarpDealB / 32], mine = 0;  // (units of 128 requests fit 31 bits)
#pragma unroll
  for (int i = 0; i < kWarpDealB / 32; ++i) {
    n[i] = i < per && b0 + i < p.B ? seg_units<SC>(kv_tiles<TS>(kv_len(p, b0 + i))) : 0;
    mine += n[i];
  }
  uint32_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint32_t a = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += a;
  }
  const Deal deal(p, (long long)__shfl_sync(0xffffffffu, inc, 31) * Hr);
  Walk w = {0, 0, 0, 0};
  if (blockIdx.x >= deal.n) return w;
  const long long u0 = deal.start(blockIdx.x);
  long long at = (long long)(inc - mine) * Hr;
  const bool here = at <= u0 && u0 < (long long)inc * Hr;
  if (here) {
#pragma unroll
    for (int i = 0; i < kWarpDealB / 32; ++i) {
      const long long in = u0 - at, all = (long long)n[i] * Hr;
      if (in >= 0 && in < all) {
        w.b = b0 + i;
        w.hr = in <= 0xffffffffll ? (int)((uint32_t)in / n[i]) : (int)(in / n[i]);
        w.v = (int)(in - (long long)w.hr * n[i]);
      }
      at += all;
    }
  }
  const int src = __ffs(__ballot_sync(0xffffffffu, here)) - 1;
  w.b = __shfl_sync(0xffffffffu, w.b, src);
  w.hr = __shfl_sync(0xffffffffu, w.hr, src);
  w.v = __shfl_sync(0xffffffffu, w.v, src);
  w.left = deal.start(blockIdx.x + 1ll) - u0;
  return w;
}
__device__ __forceinline__ Walk first_walk(const long long* st) {
  const int* w = reinterpret_cast<const int*>(st + 2);
  Walk w0;
  w0.left = st[1] - st[0];
  w0.b = w[0];
  w0.hr = w[1];
  w0.v = w[2];
  return w0;
}

}  // namespace
}  // namespace attn
