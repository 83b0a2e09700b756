// kv_split.cuh -- how a block of a decode from a paged cache finds its range of the work (kv_split.h):
// shared by the cache in 8 bits (attn_kv8.cu) and in 4 bits (attn_kv4.cu).
#pragma once

#include "kernels.h"
#include "kv_split.h"

namespace attn {
namespace {

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
