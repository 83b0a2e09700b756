// attn_kv8.cu -- a paged key/value cache held in 8 bits, for sm_103a.
//
// The cache holds codes [P][H][page][d] in e4m3 and one scale per page and
// key head, K and V each: a key is k = ks * kcode.  Scales written here are
// powers of two, so scaling is exact, the codes lose nothing but e4m3's own
// rounding, and a page whose scale must grow is rounded again from its codes
// (exactly, but where they fall among the subnormal ones).
//
// attn_kv8_append_kernel   rounds new keys and values into their slots.
// attn_kv8_split_kernel    O = softmax(s q K^T) V over the cache, split.
// attn_kv_merge_kernel     joins the parts of a split (request, head), of this cache
//                          and of the one in 4 bits.
//
// Decoding streams the codes once, 2 d bytes a key and head, and is bound by
// HBM.  The codes go from TMA to shared memory to the tensor core as they
// are: no thread ever converts a cached value.  What makes that possible is
// that the *other* operand of each product is written as a short sum of e4m3
// values,
//   q 2^-e = q1 + q2 / 16 [+ q3 / 256],   p = p1 + p2 / 16 [+ p3 / 256],
// each term the rounding of what the ones before it leave: four significant
// bits a term.  Two terms hold a bf16 q exactly (8 bits) and p to 2^-9 of its
// value; three hold an fp16 q exactly (11 bits) and p to 2^-14.  (Elements
// below 2^-13 of their row's largest lose bits, none more than 2^-21 of that
// largest.)  The terms are rows of one operand, so they cost columns of an
// MMA that is nearly empty anyway:
//   S^T [128 keys x N]  = K [128 x d]  (q terms)^T,   N = rows x terms
//   O^T [d x N]         = V^T [d x 128] (p terms)^T
// with K and V the A operands straight from shared memory (K rows K-major, V
// MN-major) and keys, then d, along the 128 TMEM lanes.  A thread owns a key
// and all query rows of the head group: masks, scales of pages and the
// exponentials need no exchange; the row maximum is one redux per row and
// warp and one shared-memory exchange per tile.
//
// The value scale enters the exponent: with w = s + log2 vs and the tile's
// row maximum m_t of w, p = 2^(w - m_t + 8) fills e4m3's range whatever the
// pages' scales are; l sums p / vs, O^T of the tile comes out of TMEM and is
// added to fp32 registers with the usual running-maximum factors.  p is
// normalised per tile, so a tile far below the running maximum keeps its
// precision, and what a key loses is at most 2^-22 of its own tile's largest.
//
// Work split: all tiles (128 keys of one head group of one request) are
// numbered and every CTA takes an equal consecutive range, whatever the
// lengths are; the range may begin and end inside a (request, head), whose
// parts then meet in the merge kernel.
//
// Measured (graph replay, split and merge kernel; 16-bit q, d = 128, page 64 /
// 128): four requests of 50001 to 131072 tokens, 32 query and 4 key heads, 341 MB:
// 60 us, the split kernel by itself 55 us or 6.2 TB/s, 93 % of the measured copy
// bandwidth; 64 requests of 100 to 8192 tokens, 32 and 8 heads, 246 MB: 51 us, the
// split kernel 45 us or 5.5 TB/s; one request of 1000 tokens: 9.4 us, two launches
// and the chain lengths, page ids, keys, scores, parts.  DRAM reads are the codes,
// once (340.9 MB); the tensor pipe is 4 % busy, the warp schedulers 36 %.
// What it took, on the 64 requests: 79 us with O^T waited for in its own tile and
// two CTAs to an SM, 65 us with it added a tile later, blocks of 4 rows and three
// CTAs, 52 us with the segments' cost counted in the shares.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "kv_split.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

// ------------------------------------------------------------------ append
// Exponent of the smallest power of two s with amax <= 448 s, in [-64, 60]
// (amax = 1.75 2^8 s at most: adding 2^21 - 1 to the bits carries into the
// exponent exactly when the mantissa is above 1.75).
__device__ __forceinline__ int scale_exp(float amax) {
  const int e = (int)((__float_as_uint(amax) + 0x1FFFFFu) >> 23) - 135;
  return min(max(e, -64), 60);
}
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// Pairwise max(a, |w|) of two 16-bit values.
template <bool BF16>
__device__ __forceinline__ uint32_t max2_abs(uint32_t a, uint32_t w) {
  uint32_t r;
  if constexpr (BF16)
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(w & 0x7fff7fffu));
  else
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(w & 0x7fff7fffu));
  return r;
}

constexpr int kAppThreads = 128;

// One warp per (chunk of `chunk` tokens, head, K or V): it takes the runs of
// consecutive slots in one page that begin in its chunk.  Two passes over a
// run: largest magnitude, then codes; the first 16 (d = 128) or 32 (d = 64)
// tokens stay in registers between them.  Bound by its own instructions for prompts
// (conversions and the search for runs: issue slots 58 %, DRAM 25 %), by latency for a
// decoding step: the chain slot, values and old scale, codes.  Blocks of 128 threads,
// six to an SM at 80 registers: a block whose warps have done their runs makes room
// sooner than a larger one.
// Measured: 31749 tokens of 4 heads, d = 64, page 16 (49 MB) 11.1 us or 4.4 TB/s (12.0
// with blocks of 256, three to an SM; 11.6 with eight at 64 registers), 15 us with
// the values in HBM, the schedulers 58 % busy; one token of each of 256 requests, 8
// heads, d = 128, 4.3 us.
template <int D, bool BF16>
__global__ void __launch_bounds__(kAppThreads, 6) attn_kv8_append_kernel(const __grid_constant__ Kv8AppendArgs p,
                                                                     int chunk) {
  griddep_wait();
  constexpr int kLanes = D / 8;          // lanes of 16 bytes to a token
  constexpr int kTok = 32 / kLanes;      // tokens per warp load
  constexpr int kU = 8;
  const int lane = threadIdx.x & 31, sub = lane / kLanes, part = lane % kLanes;
  // (T H < 2^30: the warp's number has 31 bits; pages are powers of two)
  const unsigned gw = (unsigned)(((unsigned long long)blockIdx.x * blockDim.x + threadIdx.x) >> 5);
  const int kv = (int)(gw & 1);
  const unsigned ci = (gw >> 1) / (unsigned)p.H;
  const int h = (int)((gw >> 1) - ci * (unsigned)p.H);
  const long long t0 = (long long)ci * chunk;
  const int ps = 1 << p.page_shift;
  auto slot_at = [&](long long t) -> long long {
    const long long s = t >= 0 && t < p.T ? p.slots[t] : -1;
    return s >= 0 && s < p.n_slots ? s : -1;
  };
  // A lane looks at one token: whether it goes on with the run of the token
  // before it, or begins one (only the chunk's own beginnings are taken).
  const long long my_slot = slot_at(t0 + lane);
  long long prev = __shfl_up_sync(0xffffffffu, my_slot, 1);
  if (lane == 0) prev = slot_at(t0 - 1);
  const bool goes_on = my_slot >= 0 && prev == my_slot - 1 && (my_slot & (ps - 1)) != 0;
  const uint32_t on = __ballot_sync(0xffffffffu, goes_on);
  uint32_t starts = __ballot_sync(0xffffffffu, my_slot >= 0 && !goes_on && lane < chunk);
  const uint8_t* x = static_cast<const uint8_t*>(p.x[kv]);
  while (starts) {
    const int bit = __ffs(starts) - 1;
    starts &= starts - 1;
    const long long t = t0 + bit, slot = __shfl_sync(0xffffffffu, my_slot, bit);
    const long long page = slot >> p.page_shift;
    const int first = (int)(slot & (ps - 1));
    // length of the run: seen above, or beyond the 32 tokens
    int n = 1 + __ffs(~(on >> bit >> 1)) - 1;
    if (bit + n >= 32) {
      n = 32 - bit;
      for (; first + n < ps; n += 32) {
        const int i = n + lane;
        const uint32_t in = __ballot_sync(0xffffffffu, first + i < ps && slot_at(t + i) == slot + i);
        if (in != 0xffffffffu) {
          n += __ffs(~in) - 1;
          break;
        }
      }
      n = min(n, ps - first);
    }
    const uint8_t* src = x + ((t * p.x_stride[kv]) + (long long)h * D) * 2 + part * 16;
    const long long row_bytes = p.x_stride[kv] * 2;
    float* scale = p.scale[kv] + page * p.H + h;
    uint8_t* dst = p.cache[kv] + ((page * p.H + h) << p.page_shift) * D;
    const float old = first > 0 ? *scale : 0.f;
    uint4 v[kU];
    uint32_t top = 0;  // largest magnitudes, a pair of 16-bit values (NaN ignored)
    auto load = [&](int i0) {
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = i0 + u * kTok + sub;
        v[u] = i < n ? *reinterpret_cast<const uint4*>(src + i * row_bytes) : make_uint4(0, 0, 0, 0);
      }
    };
    for (int i0 = 0; i0 < n; i0 += kU * kTok) {
      load(i0);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const uint32_t* w = &v[u].x;
#pragma unroll
        for (int j = 0; j < 4; ++j) top = max2_abs<BF16>(top, w[j]);
      }
    }
    const float2 top2 = unpack2<BF16>(top);
    const float amax = warp_max(fmaxf(top2.x, top2.y));
    const float now = fmaxf(pow2f(scale_exp(amax)), old);
    const float inv = 1.f / now;
    if (first > 0 && now > old) {  // the tokens before the run, rounded again
      const float ratio = old / now;
      for (int o = lane * 16; o < first * D; o += 32 * 16) {
        uint4 c = *reinterpret_cast<const uint4*>(dst + o);
        uint32_t* w = &c.x;
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 lo = unpack_e4m3(w[j] & 0xffffu), hi = unpack_e4m3(w[j] >> 16);
          w[j] = pack_e4m3(lo.x * ratio, lo.y * ratio) | (pack_e4m3(hi.x * ratio, hi.y * ratio) << 16);
        }
        *reinterpret_cast<uint4*>(dst + o) = c;
      }
    }
    for (int i0 = 0; i0 < n; i0 += kU * kTok) {
      if (n > kU * kTok) load(i0);
#pragma unroll
      for (int u = 0; u < kU; ++u) {
        const int i = i0 + u * kTok + sub;
        const uint32_t* w = &v[u].x;
        uint32_t c[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const float2 f = unpack2<BF16>(w[j]);
          c[j] = pack_e4m3(f.x * inv, f.y * inv);
        }
        if (i < n)
          *reinterpret_cast<uint2*>(dst + (first + i) * D + part * 8) = make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
      }
    }
    __syncwarp();
    if (lane == 0 && now != old) *scale = now;
  }
  if (threadIdx.x == 0) griddep_launch_dependents();
}

// ------------------------------------------------------------------ decode
constexpr int kDecThreads = 192;  // warps 0-3 softmax, 4 producer, 5 MMA
constexpr int kWarpProd = 4, kWarpMma = 5;
constexpr uint32_t kWgBar = 1;    // named barrier of the softmax warps

__host__ __device__ constexpr int up1024(int x) { return (x + 1023) / 1024 * 1024; }

template <int D, int RP, int NP>
struct Kv8Layout {
  static constexpr int N = (RP * NP + 15) / 16 * 16;  // MMA columns (M = 128 needs a multiple of 16)
  static constexpr int kTile = 128 * D;
  // CTAs to an SM: 3 with 4 rows (94 registers, two stages each), 2 with more, whose
  // rows need the registers (8 rows: 60 us on four long requests, 63 with 3).
  static constexpr int kCtas = RP <= 4 ? 3 : 2;
  static constexpr int kStages = (D == 128 ? 1 : 2) * (kCtas == 3 ? 2 : 3);
  static constexpr int kQ = 0;
  static constexpr int kP = kQ + up1024(N * D);
  static constexpr int kKV = kP + up1024(N * 128);    // stage s: K at + s * 2 kTile, V behind it
  static constexpr int kScale = kKV + kStages * 2 * kTile;  // [stages][K, V][8] fp32
  static constexpr int kXm = kScale + kStages * 64;   // [2][4][RP] fp32 row maxima of the warps
  static constexpr int kXl = kXm + 2 * 4 * RP * 4;    // [4][RP] fp32 row sums
  static constexpr int kQs = kXl + 4 * RP * 4;        // [RP] fp32 row factors
  static constexpr int kQi = kQs + RP * 4;            // [RP] int query index of the row
  static constexpr int kBar = kQi + RP * 4;
  static constexpr int kBarKFull = 0;
  static constexpr int kBarVFull = kBarKFull + kStages;
  static constexpr int kBarEmpty = kBarVFull + kStages;
  static constexpr int kBarSFull = kBarEmpty + kStages;  // [2]
  static constexpr int kBarPFull = kBarSFull + 2;
  static constexpr int kBarOFull = kBarPFull + 1;
  static constexpr int kBarQFull = kBarOFull + 1;
  static constexpr int kBarDrain = kBarQFull + 1;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kStart = kTmemSlot + 16;       // start of the CTA's range: long long u0, u1; int b, hr, t
  static constexpr int kScan = kStart + 32;           // [6] warp sums
  static constexpr int kBytes = kScan + 8 * 8;
  static constexpr int kSmem = kBytes + 1024;
  static constexpr int kCols = 4 * N <= 64 ? 64 : (4 * N <= 128 ? 128 : 256);  // S x 2, O x 2, a power of two
  static constexpr int kColS = 0, kColO = 2 * N;
  static_assert(4 * N <= kCols && kCols * kCtas <= 512, "TMEM budget");
  static_assert((kSmem + 1024) * kCtas <= 228 * 1024, "shared memory budget");
  static_assert(kBar % 8 == 0 && kStart % 8 == 0 && kScan % 8 == 0, "alignment");
};

template <int D, int RP, int NP>
__global__ void __launch_bounds__(kDecThreads, Kv8Layout<D, RP, NP>::kCtas) attn_kv8_split_kernel(const __grid_constant__ KvDecArgs p) {
  using L = Kv8Layout<D, RP, NP>;
  constexpr bool BF16 = NP == 2;
  constexpr int N = L::N;
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t base = (raw + 1023u) & ~1023u;
  uint8_t* sbase = smem_raw + (base - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hr = p.H * p.n_rb;
  const WaitCtl wc{p.wait.status, p.wait.limit_ns};
  auto bar = [&](int i) -> uint32_t { return base + L::kBar + 8u * i; };

  if (warp == kWarpProd && lane == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar(L::kBarKFull + s), 33);  // the copies' arrival and one per lane (scales)
      mbar_init(bar(L::kBarVFull + s), 1);
      mbar_init(bar(L::kBarEmpty + s), 1);
    }
    mbar_init(bar(L::kBarSFull), 1);
    mbar_init(bar(L::kBarSFull + 1), 1);
    mbar_init(bar(L::kBarPFull), 128);
    mbar_init(bar(L::kBarOFull), 1);
    mbar_init(bar(L::kBarQFull), 128);
    mbar_init(bar(L::kBarDrain), 1);
    fence_mbar_init();
    tma_prefetch(&p.tm_k);
    tma_prefetch(&p.tm_v);
  }
  if (warp == kWarpMma) {
    tmem_alloc(base + L::kTmemSlot, L::kCols);
    tmem_relinquish();
  }
  griddep_wait();
  deal_range<7, kKv8SegCost, kDecThreads>(p, Hr, reinterpret_cast<long long*>(sbase + L::kScan),
                             reinterpret_cast<long long*>(sbase + L::kStart));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sbase + L::kTmemSlot);
  const Walk w0 = first_walk(reinterpret_cast<const long long*>(sbase + L::kStart));
  const int page_rows = 1 << p.page_shift;
  const int tile_pages = 128 >> p.page_shift;

  if (warp == kWarpProd) {
    // ------------------------------------------------------------ producer
    // Lane i takes page i of a tile: its id (read a tile ahead), its K and V
    // copies and its two scales.
    if (!(p.debug_flags & 16)) {
      int g = 0;
      bool ok = true;
      Walk w = w0;
      Seg sg;
      while (ok && next_seg<7, kKv8SegCost>(p, Hr, w, sg)) {
        const int len = sg.len;
        const int h = sg.hr / p.n_rb;
        const int pages = (len + page_rows - 1) >> p.page_shift;
        const int* row = p.table + (size_t)sg.b * p.width;
        auto page_id = [&](int t) -> int {
          const int j = t * tile_pages + lane;
          return lane < tile_pages && j < pages ? row[j] : -1;
        };
        int id = page_id(sg.t0);
        for (int t = sg.t0; t < sg.t1; ++t, ++g) {
          const int here = id;
          const int n_here = min(tile_pages, pages - t * tile_pages);
          if (t + 1 < sg.t1) id = page_id(t + 1);
          const int s = g % L::kStages;
          const uint32_t ph = (g / L::kStages) & 1;
          ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarEmpty + s), ph ^ 1, wc));
          if (!ok) break;
          const uint32_t bytes = (uint32_t)(n_here * page_rows * D);
          if (lane == 0) {
            mbar_expect_tx(bar(L::kBarKFull + s), bytes);
            mbar_expect_tx(bar(L::kBarVFull + s), bytes);
          }
          __syncwarp();
          if (lane < n_here) {
            const uint32_t k = base + L::kKV + s * 2 * L::kTile + lane * page_rows * D;
            // (a page id outside the cache reads as zeros, its scales too)
            const bool in = here >= 0 && here < p.P;
            const int c2 = in ? here * p.H + h : -1;
            const size_t si = in ? (size_t)here * p.H + h : 0;
            const uint32_t sn = in ? 4 : 0;  // bytes read; the rest of the four are zeros
            tma_load_3d(k, &p.tm_k, bar(L::kBarKFull + s), 0, 0, c2);
            const uint32_t sc = base + L::kScale + s * 64 + lane * 4;
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(sc), "l"(p.k_scale + si), "r"(sn)
                         : "memory");
            asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(sc + 32), "l"(p.v_scale + si), "r"(sn)
                         : "memory");
            tma_load_3d(k + L::kTile, &p.tm_v, bar(L::kBarVFull + s), 0, 0, c2);
          }
          asm volatile("cp.async.mbarrier.arrive.noinc.shared.b64 [%0];" ::"r"(bar(L::kBarKFull + s)) : "memory");
        }
      }
      if (!ok) {
        for (int i = max(0, g - L::kStages); i < g; ++i) {
          mbar_wait_drain(bar(L::kBarKFull + i % L::kStages), (i / L::kStages) & 1, wc.limit_ns);
          mbar_wait_drain(bar(L::kBarVFull + i % L::kStages), (i / L::kStages) & 1, wc.limit_ns);
        }
      }
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA warp
    constexpr uint32_t idesc_s = make_idesc_e4m3(128, N, false, false);
    constexpr uint32_t idesc_o = make_idesc_e4m3(128, N, true, false);
    auto wt = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar(i), parity, wc)); };
    auto kaddr = [&](int g) { return base + L::kKV + (g % L::kStages) * 2 * L::kTile; };
    auto issue_s = [&](int g) {  // S^T = K (q terms)^T over d
      const uint32_t k = kaddr(g), d_t = tmem + L::kColS + (g & 1) * N;
#pragma unroll
      for (int ks = 0; ks < D / 32; ++ks) {
        const uint64_t a = D == 128 ? make_sdesc(k + ks * 32, 16, 1024) : make_sdesc64(k + ks * 32, 16, 512);
        const uint64_t b = D == 128 ? make_sdesc(base + L::kQ + ks * 32, 16, 1024)
                                    : make_sdesc64(base + L::kQ + ks * 32, 16, 512);
        mma_ss_f8(d_t, a, b, idesc_s, ks > 0);
      }
      tc_commit(bar(L::kBarSFull + (g & 1)));
    };
    auto issue_o = [&](int g) {  // O^T = V^T (p terms)^T over the tile's keys
      const uint32_t v = kaddr(g) + L::kTile;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks) {
        // V is MN-major: 32 keys are four 8-key groups of 8 D bytes; for
        // d = 64 a zero block offset makes rows 64-127 of V^T repeat 0-63
        const uint64_t a = D == 128 ? make_sdesc(v + ks * 32 * D, 16, 1024) : make_sdesc64(v + ks * 32 * D, 0, 512);
        mma_ss_f8(tmem + L::kColO + (g & 1) * N, a, make_sdesc(base + L::kP + ks * 32, 16, 1024), idesc_o, ks > 0);
      }
      tc_commit(bar(L::kBarEmpty + g % L::kStages));
      tc_commit(bar(L::kBarOFull));
    };
    bool ok = true;
    int g = 0, seg = 0;
    Walk w = w0;
    Seg sg;
    while (ok && next_seg<7, kKv8SegCost>(p, Hr, w, sg)) {
      const int cnt = sg.t1 - sg.t0;
      ok = wt(L::kBarQFull, seg & 1) && wt(L::kBarKFull + g % L::kStages, (g / L::kStages) & 1);
      if (!ok) break;
      tc_fence_after();
      issue_s(g);
      for (int i = 0; i < cnt; ++i, ++g) {
        if (i + 1 < cnt) {
          ok = wt(L::kBarKFull + (g + 1) % L::kStages, ((g + 1) / L::kStages) & 1);
          if (!ok) break;
          tc_fence_after();
          issue_s(g + 1);
        }
        ok = wt(L::kBarPFull, g & 1) && wt(L::kBarVFull + g % L::kStages, (g / L::kStages) & 1);
        if (!ok) break;
        tc_fence_after();
        issue_o(g);
      }
      ++seg;
    }
    tc_commit(bar(L::kBarDrain));
    mbar_wait_drain(bar(L::kBarDrain), 0, wc.limit_ns);
  } else {
    // ------------------------------------------------------------ softmax
    const int kl = threadIdx.x;  // key of the tile = TMEM lane of S^T; d index = lane of O^T
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t tS = tmem + lane_off + L::kColS, tO = tmem + lane_off + L::kColO;
    float* xm = reinterpret_cast<float*>(sbase + L::kXm);
    float* xl = reinterpret_cast<float*>(sbase + L::kXl);
    float* qs_s = reinterpret_cast<float*>(sbase + L::kQs);
    int* qi_s = reinterpret_cast<int*>(sbase + L::kQi);
    const int R = p.Nq * p.G;
    uint8_t* prow = sbase + L::kP;
    const uint32_t pcol = (uint32_t)kl;
    bool ok = true;
    int g = 0, seg = 0;
    Walk w = w0;
    Seg sg;
    while (ok && next_seg<7, kKv8SegCost>(p, Hr, w, sg)) {
      const int len = sg.len;
      const int h = sg.hr / p.n_rb, rb = sg.hr % p.n_rb;
      // ---- the q terms of the row block: eight lanes to a row
      if (kl < RP * 8) {
        constexpr int E = D / 8;  // elements per lane
        const int r = kl >> 3, c = kl & 7, idx = rb * RP + r;
        const int i = idx / p.G, hq = h * p.G + idx % p.G;
        float f[E];
        if (idx < R) {
          const uint4* src = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.q) +
                                                            ((((size_t)sg.b * p.Nq + i) * p.Hq + hq) * D + c * E) * 2);
#pragma unroll
          for (int j = 0; j < E / 8; ++j) {
            const uint4 v = src[j];
            const uint32_t* wv = &v.x;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float2 x = unpack2<BF16>(wv[e]);
              f[j * 8 + 2 * e] = x.x;
              f[j * 8 + 2 * e + 1] = x.y;
            }
          }
        } else {
#pragma unroll
          for (int j = 0; j < E; ++j) f[j] = 0.f;
        }
        uint32_t top = 0;  // largest magnitude, as bits (inf and NaN above all numbers)
#pragma unroll
        for (int j = 0; j < E; ++j) top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        // 2^-e brings the row's largest into [128, 256)
        const int e = min(max((int)(top >> 23) - 127 - 7, -100), 120);
        const float mul = pow2f(-e);
        const bool bad = top >= 0x7f800000u;
#pragma unroll
        for (int j = 0; j < E; ++j) f[j] *= mul;
#pragma unroll
        for (int t = 0; t < NP; ++t) {
          uint32_t cw[E / 4];
#pragma unroll
          for (int j = 0; j < E; j += 4) {
            const uint32_t lo = pack_e4m3(f[j], f[j + 1]), hi = pack_e4m3(f[j + 2], f[j + 3]);
            const float2 a = unpack_e4m3(lo), b = unpack_e4m3(hi);
            f[j] = (f[j] - a.x) * 16.f;  // exact: what the term leaves, for the next one
            f[j + 1] = (f[j + 1] - a.y) * 16.f;
            f[j + 2] = (f[j + 2] - b.x) * 16.f;
            f[j + 3] = (f[j + 3] - b.y) * 16.f;
            cw[j / 4] = lo | (hi << 16);
          }
          const uint32_t off = (uint32_t)((t * RP + r) * D + c * E);
          const uint32_t swz = D == 128 ? off ^ (((off >> 7) & 7u) << 4) : off ^ (((off >> 7) & 3u) << 4);
          if constexpr (E == 16)
            *reinterpret_cast<uint4*>(sbase + L::kQ + swz) = make_uint4(cw[0], cw[1], cw[2], cw[3]);
          else
            *reinterpret_cast<uint2*>(sbase + L::kQ + swz) = make_uint2(cw[0], cw[1]);
        }
        if (c == 0) {
          qs_s[r] = bad ? __uint_as_float(0x7fc00000u) : pow2f(e) * p.scale * kLog2e;
          qi_s[r] = i;
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(L::kBarQFull));
      ok = named_bar_and(kWgBar, 128, ok);
      if (!ok) break;
      float m[RP], l[RP], acc[RP];
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
        acc[r] = 0.f;
      }
      const int lim0 = p.causal ? len - p.Nq : len - 1;  // keys <= lim0 are seen by every row
      // O^T of a tile is added a tile later, while the tensor core works on the
      // next one: be is the factor of the tile whose O^T is outstanding (acc is
      // already on that tile's scale).
      float be[RP];
      auto add_o = [&](int go) {
        tc_fence_after();
        uint32_t r_[N];
#pragma unroll
        for (int c = 0; c < N; c += 16) tmem_ld16(tO + (go & 1) * N + c, r_ + c);
        tmem_ld_wait();
        reg_fence<N>(r_);
        tc_fence_before();
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          float o = __uint_as_float(r_[r]), c = __uint_as_float(r_[RP + r]);
          if constexpr (NP == 3) c = fmaf(__uint_as_float(r_[2 * RP + r]), 0.0625f, c);
          o = fmaf(c, 0.0625f, o);
          acc[r] = fmaf(o, be[r], acc[r]);
        }
      };
      for (int t = sg.t0; t < sg.t1; ++t, ++g) {
        const int st = g % L::kStages, kv0 = t * 128;
        const bool later = t > sg.t0;  // the tile before is of this segment, its O^T outstanding
        ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarSFull + (g & 1)), (g >> 1) & 1, wc) &&
                                         mbar_wait(bar(L::kBarKFull + st), (g / L::kStages) & 1, wc));
        float x[RP];
        float inv_vs = 1.f, lv = 0.f;
        if (ok) {
          tc_fence_after();
          uint32_t r_[N];
#pragma unroll
          for (int c = 0; c < N; c += 16) tmem_ld16(tS + (g & 1) * N + c, r_ + c);
          const float* sc = reinterpret_cast<const float*>(sbase + L::kScale + st * 64);
          const bool live = kv0 + kl < len;
          const float ks = sc[kl >> p.page_shift], vs_ = sc[8 + (kl >> p.page_shift)];
          const float vs = live && vs_ != 0.f ? vs_ : 1.f;
          lv = __log2f(vs);
          inv_vs = 1.f / vs;
          tmem_ld_wait();
          reg_fence<N>(r_);
#pragma unroll
          for (int r0 = 0; r0 < RP; r0 += 4) {
            const float4 q4 = *reinterpret_cast<const float4*>(qs_s + r0);
            const float qs[4] = {q4.x, q4.y, q4.z, q4.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int r = r0 + j;
              float s = __uint_as_float(r_[r]);
              float c = __uint_as_float(r_[RP + r]);
              if constexpr (NP == 3) c = fmaf(__uint_as_float(r_[2 * RP + r]), 0.0625f, c);
              s = fmaf(c, 0.0625f, s);
              x[r] = fmaf(s, ks * qs[j], lv);  // w = s + log2 vs
            }
          }
          if (kv0 + 127 > lim0) {
#pragma unroll
            for (int r = 0; r < RP; ++r) {
              const int lim = p.causal ? len - p.Nq + qi_s[r] : len - 1;
              if (kv0 + kl > lim || !live) x[r] = -INFINITY;
            }
          }
          float* mine = xm + ((g & 1) * 4 + warp) * RP;
#pragma unroll
          for (int r = 0; r < RP; r += 4) {
            const float4 v = make_float4(warp_max(x[r]), warp_max(x[r + 1]), warp_max(x[r + 2]), warp_max(x[r + 3]));
            if (lane == 0) *reinterpret_cast<float4*>(mine + r) = v;
          }
        }
        if (ok && kv0 + 128 > len) {
          // the last tile: values behind the request's end become zeros
          ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarVFull + st), (g / L::kStages) & 1, wc));
          if (ok && kv0 + kl >= len) {
            uint4* z = reinterpret_cast<uint4*>(sbase + L::kKV + st * 2 * L::kTile + L::kTile + kl * D);
#pragma unroll
            for (int j = 0; j < D / 16; ++j) z[j] = make_uint4(0, 0, 0, 0);
          }
        }
        // (the O^T outstanding is complete: its MMA has read P, which is
        // written again below)
        if (ok && later) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarOFull), (g - 1) & 1, wc));
        ok = named_bar_and(kWgBar, 128, ok);
        if (!ok) break;
        float al_t[RP], be_t[RP];
#pragma unroll
        for (int r0 = 0; r0 < RP; r0 += 4) {
          float4 v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const float4*>(xm + ((g & 1) * 4 + q) * RP + r0);
          const float mt4[4] = {fmaxf(fmaxf(v[0].x, v[1].x), fmaxf(v[2].x, v[3].x)),
                                fmaxf(fmaxf(v[0].y, v[1].y), fmaxf(v[2].y, v[3].y)),
                                fmaxf(fmaxf(v[0].z, v[1].z), fmaxf(v[2].z, v[3].z)),
                                fmaxf(fmaxf(v[0].w, v[1].w), fmaxf(v[2].w, v[3].w))};
          uint32_t code[NP][2];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = r0 + j;
            const float mt = mt4[j];
            // running maximum: one of the factors of the old and the new part is 1
            const float e = ex2(mt > m[r] ? m[r] - mt : mt - m[r]);
            al_t[r] = mt > m[r] ? e : 1.f;
            be_t[r] = (mt < m[r] ? e : 1.f) * 0.00390625f;  // p below carries 2^8
            m[r] = fmaxf(m[r], mt);
            x[r] = ex2(x[r] - (mt == -INFINITY ? 0.f : mt - 8.f));  // p 2^8
            l[r] = fmaf(x[r], be_t[r] * inv_vs, l[r] * al_t[r]);
          }
#pragma unroll
          for (int q = 0; q < 2; ++q) {
            float a = x[r0 + 2 * q], b = x[r0 + 2 * q + 1];
#pragma unroll
            for (int t2 = 0; t2 < NP; ++t2) {
              code[t2][q] = pack_e4m3(a, b);
              if (t2 + 1 < NP) {
                const float2 d = unpack_e4m3(code[t2][q]);
                a = (a - d.x) * 16.f;
                b = (b - d.y) * 16.f;
              }
            }
          }
          // byte of this key in row n of the P tile: 128 n, 16-byte chunk XOR n % 8
#pragma unroll
          for (int t2 = 0; t2 < NP; ++t2)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const int n = t2 * RP + r0 + j;
              prow[n * 128 + (pcol ^ ((n & 7) << 4))] = (uint8_t)(code[t2][j >> 1] >> (8 * (j & 1)));
            }
        }
        fence_proxy_async_smem();
        tc_fence_before();
        mbar_arrive(bar(L::kBarPFull));
        if (later) add_o(g - 1);
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          acc[r] *= al_t[r];
          be[r] = be_t[r];
        }
      }
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarOFull), (g - 1) & 1, wc));
      if (ok) add_o(g - 1);
      // ---- end of the segment: row sums over the 128 keys, then O
#pragma unroll
      for (int r = 0; r < RP; ++r) {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) l[r] += __shfl_xor_sync(0xffffffffu, l[r], o);
        if (lane == 0) xl[warp * RP + r] = l[r];
      }
      ok = named_bar_and(kWgBar, 128, ok);
      if (!ok) break;
      const bool whole = sg.t1 - sg.t0 == sg.nt;
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        const int idx = rb * RP + r;
        if (idx >= R) break;
        const float lt = (xl[r] + xl[RP + r]) + (xl[2 * RP + r] + xl[3 * RP + r]);
        if (whole) {
          const int i = idx / p.G, hq = h * p.G + idx % p.G;
          const float v = lt != 0.f ? acc[r] / lt : 0.f;
          if (kl < D) {
            const uint32_t c = pack2<BF16>(v, 0.f);
            reinterpret_cast<uint16_t*>(p.o)[(((size_t)sg.b * p.Nq + i) * p.Hq + hq) * D + kl] = (uint16_t)c;
          }
          if (kl == 0)
            p.lse[((size_t)sg.b * p.Hq + hq) * p.Nq + i] = lt != 0.f ? (m[r] + __log2f(lt)) * kLn2 : -INFINITY;
        } else {
          const size_t part = ((size_t)blockIdx.x * 2 + (seg > 0 ? 1 : 0)) * RP + r;
          if (kl < D) p.ws_o[part * D + kl] = acc[r];
          if (kl == 0) {
            p.ws_ml[part * 2] = m[r];
            p.ws_ml[part * 2 + 1] = lt;
          }
        }
      }
      ++seg;
    }
  }
  if (threadIdx.x == 0) griddep_launch_dependents();
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

// Joins the parts of a segment that several CTAs share; requests without keys get
// O = 0, LSE = -inf.  A lane holds D / 32 columns, eight parts' loads in flight.
// WPR = 4: a block per query row, whose parts are dealt to its four warps (few
// rows, many parts: one row of four long requests has 19 parts each).  WPR = 1: a
// warp per row, four rows of a segment at a time, p.merge_run times (many rows: most
// segments are one CTA's, and their blocks only find that out).  Always in the same
// order.
template <int D, bool BF16, int WPR, int TS, int SC>
__global__ void __launch_bounds__(128) attn_kv_merge_kernel(const __grid_constant__ KvDecArgs p) {
  __shared__ long long sums[4][2];
  __shared__ float xo[4][D];
  __shared__ float xml[4][2];
  // (Before the wait only what the split kernel reads as well, which waited for the kernels before it.)
  constexpr int kPer = D / 32, kU = 8;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int Hr = p.H * p.n_rb, R = p.Nq * p.G;
  // a block's units: one row, or p.merge_run times four rows of one row block
  const unsigned per = WPR == 4 ? 1 : 4, n_in = (p.rp + per - 1) / per;
  const unsigned run = WPR == 4 ? 1 : p.merge_run, units_all = (unsigned)p.B * Hr * n_in;
  const unsigned first = blockIdx.x * run;
  int b = (int)(first / n_in / (unsigned)Hr);
  long long before = 0, total = 0;
  for (int i = threadIdx.x; i < p.B; i += 128) {
    const int n = seg_units<SC>(kv_tiles<TS>(kv_len(p, i)));
    total += n;
    if (i < b) before += n;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    before += __shfl_xor_sync(0xffffffffu, before, o);
    total += __shfl_xor_sync(0xffffffffu, total, o);
  }
  if (lane == 0) {
    sums[warp][0] = before;
    sums[warp][1] = total;
  }
  __syncthreads();
  before = sums[0][0] + sums[1][0] + sums[2][0] + sums[3][0];
  total = sums[0][1] + sums[1][1] + sums[2][1] + sums[3][1];
  const Deal deal(p, total * Hr);
  int nt = kv_tiles<TS>(kv_len(p, b));
  bool waited = false;
  for (unsigned unit = first; unit < min(first + run, units_all); ++unit) {
    const unsigned blk = unit / n_in;  // (b, head, row block)
    if ((int)(blk / (unsigned)Hr) != b) {
      before += seg_units<SC>(nt);
      nt = kv_tiles<TS>(kv_len(p, ++b));
    }
    const int hr = (int)(blk - (unsigned)b * Hr);
    const int h = hr / p.n_rb, rb = hr - h * p.n_rb;
    const int r = (int)((unit - blk * n_in) * per) + (WPR == 4 ? 0 : warp), idx = rb * p.rp + r;
    const long long u0 = before * Hr + (long long)hr * seg_units<SC>(nt);
    Parts at = {0, 0, 0};
    if (nt) at = kv_parts<SC>(deal, u0, nt);
    const int c0 = at.c0, c1 = at.c1, s0 = at.s0;
    if ((nt == 0 || c0 != c1) && (WPR == 1 || idx < R)) {
      auto part = [&](int c) -> size_t { return ((size_t)c * 2 + (c == c0 ? s0 : 0)) * p.rp + r; };
      const bool live = idx < R;  // (WPR = 1: a warp may have no row)
      if (!waited) griddep_wait();
      waited = true;
      float acc[kPer];
#pragma unroll
      for (int k = 0; k < kPer; ++k) acc[k] = 0.f;
      float M = -INFINITY, Ls = 0.f;
      if (nt && live) {
        // eight parts from cb on: maximum and sum of one a lane, columns of all
        float mc, lc;
        float4 v[kU];
        auto fetch = [&](int cb) {
          mc = -INFINITY;
          lc = 0.f;
          if (lane < kU && cb + lane <= c1) {
            const float2 ml = *reinterpret_cast<const float2*>(p.ws_ml + part(cb + lane) * 2);
            mc = ml.x;
            lc = ml.y;
          }
#pragma unroll
          for (int k = 0; k < kU; ++k) {
            v[k] = make_float4(0.f, 0.f, 0.f, 0.f);
            if (cb + k <= c1) {
              const float* o = p.ws_o + part(cb + k) * D + lane * kPer;
              if constexpr (kPer == 4) {
                v[k] = *reinterpret_cast<const float4*>(o);
              } else {
                const float2 v2 = *reinterpret_cast<const float2*>(o);
                v[k].x = v2.x;
                v[k].y = v2.y;
              }
            }
          }
        };
        const int cb0 = c0 + (WPR == 4 ? warp * kU : 0);
        fetch(cb0);  // (on its way while the maximum is looked for)
        for (int c = c0 + (WPR == 4 ? (int)threadIdx.x : lane); c <= c1; c += 32 * WPR) M = fmaxf(M, p.ws_ml[part(c) * 2]);
        M = warp_max(M);
        if constexpr (WPR == 4) {
          if (lane == 0) xml[warp][0] = M;
          __syncthreads();
          M = fmaxf(fmaxf(xml[0][0], xml[1][0]), fmaxf(xml[2][0], xml[3][0]));
        }
        for (int cb = cb0; cb <= c1; cb += WPR * kU) {
          if (cb != cb0) fetch(cb);
          float wgt = 0.f;
          if (lane < kU && cb + lane <= c1) {
            wgt = mc == -INFINITY ? 0.f : ex2(mc - M);
            // (a part whose every score is NaN has m = -inf and a NaN sum)
            Ls += lc != lc ? lc : wgt * lc;
          }
#pragma unroll
          for (int k = 0; k < kU; ++k) {
            const float wk = __shfl_sync(0xffffffffu, wgt, k);
            acc[0] = fmaf(wk, v[k].x, acc[0]);
            acc[1] = fmaf(wk, v[k].y, acc[1]);
            if constexpr (kPer == 4) {
              acc[2] = fmaf(wk, v[k].z, acc[2]);
              acc[3] = fmaf(wk, v[k].w, acc[3]);
            }
          }
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) Ls += __shfl_xor_sync(0xffffffffu, Ls, o);
        if constexpr (WPR == 4) {
          if (lane == 0) xml[warp][1] = Ls;
#pragma unroll
          for (int k = 0; k < kPer; ++k) xo[warp][lane * kPer + k] = acc[k];
          __syncthreads();
          Ls = (xml[0][1] + xml[1][1]) + (xml[2][1] + xml[3][1]);
#pragma unroll
          for (int k = 0; k < kPer; ++k) {
            const int c = lane * kPer + k;
            acc[k] = (xo[0][c] + xo[1][c]) + (xo[2][c] + xo[3][c]);
          }
        }
      }
      if (live && (WPR == 1 || warp == 0)) {
        const int i = idx / p.G, hq = h * p.G + idx - i * p.G;
        const float inv = Ls != 0.f ? 1.f / Ls : 0.f;
        uint32_t wv[kPer / 2];
#pragma unroll
        for (int k = 0; k < kPer / 2; ++k) wv[k] = pack2<BF16>(acc[2 * k] * inv, acc[2 * k + 1] * inv);
        uint8_t* dst = static_cast<uint8_t*>(p.o) + ((((size_t)b * p.Nq + i) * p.Hq + hq) * D + lane * kPer) * 2;
        if constexpr (kPer == 4) *reinterpret_cast<uint2*>(dst) = make_uint2(wv[0], wv[1]);
        else *reinterpret_cast<uint32_t*>(dst) = wv[0];
        if (lane == 0) p.lse[((size_t)b * p.Hq + hq) * p.Nq + i] = Ls != 0.f ? (M + __log2f(Ls)) * kLn2 : -INFINITY;
      }
    }
  }
  if (!waited) griddep_wait();  // (so that whoever waits for this kernel has waited for the split)
  griddep_launch_dependents();
}

template <int D, int RP, int NP>
cudaError_t launch_split_t(const KvDecArgs& a, cudaStream_t stream) {
  using L = Kv8Layout<D, RP, NP>;
  auto* k = attn_kv8_split_kernel<D, RP, NP>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, (unsigned)a.grid, kDecThreads, L::kSmem, stream, a);
}

template <int D, int RP>
cudaError_t launch_split_n(const KvDecArgs& a, cudaStream_t stream) {
  return a.bf16 ? launch_split_t<D, RP, 2>(a, stream) : launch_split_t<D, RP, 3>(a, stream);
}

}  // namespace

// Row blocks of 4, 8 or 16 rows: the work per tile grows with the rows.
int kv8_rows(int R) { return R <= 4 ? 4 : (R <= 8 ? 8 : 16); }

// All CTAs resident at once, no more than there can be tiles.
int kv8_grid(int rp, int sms, long long max_units) {
  long long g = (rp <= 4 ? 3ll : 2ll) * sms;
  if (g > kKvMaxCtas) g = kKvMaxCtas;
  if (g > max_units) g = max_units;
  return (int)(g < 1 ? 1 : g);
}

cudaError_t launch_kv8_split(const KvDecArgs& a, cudaStream_t stream) {
  if (a.d == 128)
    return a.rp == 4 ? launch_split_n<128, 4>(a, stream)
                     : (a.rp == 8 ? launch_split_n<128, 8>(a, stream) : launch_split_n<128, 16>(a, stream));
  return a.rp == 4 ? launch_split_n<64, 4>(a, stream)
                   : (a.rp == 8 ? launch_split_n<64, 8>(a, stream) : launch_split_n<64, 16>(a, stream));
}

constexpr long long kMergeBlocks = 2 * 8 * kSms;  // two waves of eight blocks to an SM

template <int D, bool BF16, int TS, int SC>
static cudaError_t launch_merge_t(KvDecArgs a, cudaStream_t stream) {
  const long long segs = (long long)a.B * a.H * a.n_rb;
  // parts of a segment: about a.grid / segs + 1 (64 requests of 8 heads: 51 us with a
  // warp per row, 52 with a block; 17 requests of 2 heads and 3 row blocks: 20 and 19)
  if (a.grid >= 2 * segs)
    return launch_pdl(attn_kv_merge_kernel<D, BF16, 4, TS, SC>, (unsigned)(segs * a.rp), 128, 0, stream, a);
  // Every block sums all the lengths, so with many rows a block takes several, two
  // waves of blocks in all (4096 requests of 30 to 60 tokens, 8 heads: the merge 43 us, 127
  // with a block for every four rows).
  const long long rows4 = segs * ((a.rp + 3) / 4);
  a.merge_run = (int)((rows4 + kMergeBlocks - 1) / kMergeBlocks);
  return launch_pdl(attn_kv_merge_kernel<D, BF16, 1, TS, SC>, (unsigned)((rows4 + a.merge_run - 1) / a.merge_run), 128, 0, stream, a);
}

template <bool BF16>
static cudaError_t launch_merge_b(const KvDecArgs& a, cudaStream_t stream) {
  if (a.k_scale16) {  // the cache in 4 bits
    if (a.rp == 4)
      return a.d == 128 ? launch_merge_t<128, BF16, 7, kv4_seg_cost(4, BF16)>(a, stream)
                        : launch_merge_t<64, BF16, 8, kv4_seg_cost(4, BF16)>(a, stream);
    return a.d == 128 ? launch_merge_t<128, BF16, 7, kv4_seg_cost(8, BF16)>(a, stream)
                      : launch_merge_t<64, BF16, 8, kv4_seg_cost(8, BF16)>(a, stream);
  }
  return a.d == 128 ? launch_merge_t<128, BF16, 7, kKv8SegCost>(a, stream) : launch_merge_t<64, BF16, 7, kKv8SegCost>(a, stream);
}

cudaError_t launch_kv_merge(const KvDecArgs& a, cudaStream_t stream) {
  return a.bf16 ? launch_merge_b<true>(a, stream) : launch_merge_b<false>(a, stream);
}

cudaError_t launch_kv8_append(const Kv8AppendArgs& a, int sms, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  // A warp per token, head and tensor while that is few warps, a warp per 32 tokens
  // above.  The rule sees how many tokens there are, not whether they are prompts, whose
  // runs a warp takes whole, or single tokens of many requests, which it takes one after
  // the other.  Prompts, us with 1 and with 32 (8 heads, d = 128, page 64): 300 tokens 5.5
  // and 5.3, 608 (the last with 1) 7.2 and 5.5, 2000 13.1 and 6.4; 31749 of 4 heads, d = 64,
  // page 16: 66 and 10.7 (12.8 with 32 when 16 took 13.8 and 8 took 17.3).  Single tokens:
  // 256 requests 4.2 and 25.6, 608 7.2 and 25.5, 640 (the first with 32) 7.6 and 25.6, 1024
  // 10.9 and 25.6, 4096 38 and 41, 8192 75 and 69: steps of 608 to about 4500 requests of 8
  // heads pay for the prompts.
  const int chunk = a.T * a.H * 2 <= 64ll * sms ? 1 : 32;
  const long long warps = (a.T + chunk - 1) / chunk * a.H * 2;
  const unsigned grid = (unsigned)((warps * 32 + kAppThreads - 1) / kAppThreads);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = dim3(kAppThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.d == 128)
    return a.bf16 ? cudaLaunchKernelEx(&cfg, attn_kv8_append_kernel<128, true>, a, chunk)
                  : cudaLaunchKernelEx(&cfg, attn_kv8_append_kernel<128, false>, a, chunk);
  return a.bf16 ? cudaLaunchKernelEx(&cfg, attn_kv8_append_kernel<64, true>, a, chunk)
                : cudaLaunchKernelEx(&cfg, attn_kv8_append_kernel<64, false>, a, chunk);
}

}  // namespace attn
