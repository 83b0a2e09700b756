// attn_kv4.cu -- a paged key/value cache held in 4 bits, for sm_103a.
//
// A cached value is s * c: c an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives), s a bf16 scale shared by 32 consecutive channels of one token
// and head.  4.5 bits a value; a token is rounded by itself, so nothing that is
// in the cache is ever rounded again.
//
// attn_kv4_append_kernel   rounds new keys and values into their slots.
// attn_kv4_split_kernel    O = softmax(s q K^T) V over the cache, split (joined by
//                          attn_kv_merge_kernel).
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "kv_split.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

// ------------------------------------------------------------------ append
constexpr int kAppThreads = 256;

constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kLog2e = 1.44269504088896340736f;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A thread rounds 8 channels (16 bytes in, 4 out), four neighbours share a scale.
// A block takes p.tok tokens of K or of V (blockIdx.y), all their heads, U items of a
// thread at a time.
template <int D, bool BF16, int U>
__global__ void __launch_bounds__(kAppThreads) attn_kv4_append_kernel(const __grid_constant__ Kv4AppendArgs p) {
  griddep_wait();
  constexpr int kParts = D / 8;  // threads to a token and head
  const int kv = blockIdx.y;
  const long long t0 = (long long)blockIdx.x * p.tok;
  const int n_tok = (int)min((long long)p.tok, p.T - t0);
  const int items = n_tok * p.H * kParts;
  const uint8_t* x = static_cast<const uint8_t*>(p.x[kv]);
  const int ps = 1 << p.page_shift;
  for (int i0 = threadIdx.x; i0 - (int)threadIdx.x < items; i0 += kAppThreads * U) {
    uint4 v[U];
    long long at[U];  // (page, head, place) of the item, -1: none
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kAppThreads;
      const int row = i / kParts, part = i % kParts;
      const int tl = (int)__umulhi((uint32_t)row * 2, p.h_magic), h = row - tl * p.H;
      at[u] = -1;
      v[u] = make_uint4(0, 0, 0, 0);
      if (i < items) {
        const long long t = t0 + tl, slot = p.slots[t];
        v[u] = *reinterpret_cast<const uint4*>(x + (t * p.x_stride[kv] + (long long)h * D + part * 8) * 2);
        if (slot >= 0 && slot < p.n_slots)
          at[u] = ((((slot >> p.page_shift) * p.H + h) << p.page_shift) + (slot & (ps - 1))) * kParts + part;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const uint32_t* w = &v[u].x;
      // largest magnitude as the 16 bits of it: ordered as numbers, infinity and NaN above all
      uint32_t top = max_u16x2(max_u16x2(w[0] & 0x7fff7fffu, w[1] & 0x7fff7fffu),
                               max_u16x2(w[2] & 0x7fff7fffu, w[3] & 0x7fff7fffu));
      top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, 1));
      top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, 2));
      top = max(top & 0xffffu, top >> 16);
      const float amax = unpack2<BF16>(top).x;
      // s = amax / 6 rounded to bf16.  (The quotient of 11 bits by 6 is exact in 32 bits where
      // it lies half-way between two bf16 values, so rounding it twice is rounding it once.)
      // fminf and fmaxf pass a NaN over, so a NaN is put back.
      const float f = fminf(fmaxf(__fdiv_rn(amax, 6.f), 0x1p-64f), 0x1p60f);
      const uint32_t sb = amax != amax ? 0x7fc0u : (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(f));
      const float s = __uint_as_float(sb << 16), inv = 1.f / s;
      uint32_t code = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float2 n = unpack2<BF16>(w[j] ^ 0x80008000u);  // -x
        if (amax > 0x1p63f) {  // (beyond the largest scale: saturated below; an infinity has no residual)
          n.x = fminf(fmaxf(n.x, -0x1p63f), 0x1p63f);
          n.y = fminf(fmaxf(n.y, -0x1p63f), 0x1p63f);
        }
        // x / s to 32 bits: the product with 1 / s, corrected by its residual.  A quotient of 11 by 8
        // bits that is no border between two codes is at least 2^-12 of its value away from it; one
        // that is comes out exactly.  (From -x, so that a zero keeps its sign.)
        float2 y = mul2(n, make_float2(-inv, -inv));
        const float2 r = fma2(y, make_float2(s, s), n);
        y = fma2(r, make_float2(-inv, -inv), y);
        code |= pack_e2m1(y.x, y.y) << (8 * j);
      }
      if (at[u] >= 0) {
        *reinterpret_cast<uint32_t*>(p.cache[kv] + at[u] * 4) = code;
        if ((i0 & 3) == 0) p.scale[kv][at[u] >> 2] = (uint16_t)sb;
      }
    }
  }
  if (threadIdx.x == 0) griddep_launch_dependents();
}

// ------------------------------------------------------------------ decode
constexpr int kDecThreads = 192;  // warps 0-3 softmax, 4 producer, 5 MMA, query terms and scales
constexpr int kWarpProd = 4, kWarpMma = 5;
constexpr uint32_t kWgBar = 1;    // named barrier of the softmax warps

__host__ __device__ constexpr int up1024(int x) { return (x + 1023) / 1024 * 1024; }

// A row is 128 channels: a token (d = 128) or two (d = 64).  A tile is 128 rows.
template <int D, int RP, int NP>
struct Kv4Layout {
  static constexpr int TPR = 128 / D;                 // tokens to a row
  static constexpr int kTileShift = D == 128 ? 7 : 8; // tokens to a tile
  static constexpr int NG = RP * NP;                  // operand rows: query rows times terms
  // S^T has a set of NG columns for each group of 32 channels.  M = 128 takes columns by 16: eight are
  // written by twos, a set with the next one (the other's rows of the query operand are zeros there).
  static constexpr bool kPair = NG == 8;
  static constexpr int NS = kPair ? 16 : (NG + 15) / 16 * 16;  // MMA columns
  static constexpr int kSet = kPair ? 8 : NS;         // columns from one set to the next
  static constexpr int NO = 4 * NG;                   // O^T: likewise a set for each group
  static constexpr int PW = NO <= 32 ? 32 : (NO <= 64 ? 64 : 128);  // bytes of a P row, and its swizzle
  // CTAs to an SM, by what shared memory, TMEM and registers leave
  static constexpr int kCtas = PW == 32 ? 3 : 2;
  static constexpr int kStages = PW == 64 ? 3 : 2;
  static constexpr int kCode = 128 * 128;             // bytes of a tile's codes: 16 to 16 bytes, 8 of them filled
  static constexpr int kScl = 128 * 8;                // bytes of its scales: four bf16 a row
  static constexpr int kQ = 0;
  static constexpr int kP = kQ + up1024(NS * 128);
  // three rings: K codes, V codes, scales (stage s: K's at + s * 2 kScl, V's behind them)
  static constexpr int kK = kP + up1024(128 * PW);
  static constexpr int kV = kK + kStages * kCode;
  static constexpr int kSc = kV + kStages * kCode;
  static constexpr int kNorm = kSc + kStages * 2 * kScl;  // [stages][4] 2^-e, [4] 2^e: powers above the groups' largest V scale
  static constexpr int kXm = kNorm + kStages * 32;    // [2][4][RP] fp32 row maxima of the warps
  static constexpr int kXl = kXm + 2 * 4 * RP * 4;    // [RP][4] fp32 row sums of the warps
  static constexpr int kQs = kXl + 4 * RP * 4;        // [RP] fp32 row factors
  // what the MMA warp tells the softmax warps of a segment, for two of them in turn: int4 (length, tiles
  // t0 .. t1 - 1 of nt); of a row int2 (place in o, in lse; -1: no row) and the index of its query, a byte
  static constexpr int kInfo = kQs + RP * 4;
  static constexpr int kRow = kInfo + 2 * 16;
  static constexpr int kQi = kRow + 2 * RP * 8;
  static constexpr int kBar = kQi + 2 * RP;
  static constexpr int kBarKFull = 0;
  static constexpr int kBarKEmpty = kBarKFull + kStages;
  static constexpr int kBarVFull = kBarKEmpty + kStages;
  static constexpr int kBarVEmpty = kBarVFull + kStages;
  static constexpr int kBarCFull = kBarVEmpty + kStages;   // scales
  static constexpr int kBarCEmpty = kBarCFull + kStages;
  static constexpr int kBarSFull = kBarCEmpty + kStages;   // [2] S^T and the scales' maxima
  static constexpr int kBarPFull = kBarSFull + 2;
  static constexpr int kBarOFull = kBarPFull + 1;
  static constexpr int kBarQFull = kBarOFull + 1;
  static constexpr int kBarDrain = kBarQFull + 1;
  static constexpr int kNumBars = kBarDrain + 1;
  static constexpr int kTmemSlot = kBar + kNumBars * 8;
  static constexpr int kStart = kTmemSlot + 16;       // start of the CTA's range: long long u0, u1; int b, hr, t
  static constexpr int kScan = kStart + 32;           // [6] warp sums
  static constexpr int kSmem = kScan + 6 * 8;
  // TMEM: two buffers of S^T and of O^T where the columns are there, else one
  static constexpr int kMaxCols = kCtas == 3 ? 128 : 256;
  static constexpr int kBufs = 2 * (4 * kSet + NO) <= kMaxCols ? 2 : 1;
  static constexpr int kCols = kBufs * (4 * kSet + NO) <= 128 ? 128 : 256;
  static constexpr int kColS = 0, kColO = kBufs * 4 * kSet;
  static_assert(kBufs * (4 * kSet + NO) <= kCols && kCols * kCtas <= 512, "TMEM budget");
  static_assert((kSmem + 1024) * kCtas <= 228 * 1024, "shared memory budget");
  static_assert(NO % 16 == 0 && NO <= PW, "P rows");
  static_assert(kBar % 8 == 0 && kNorm % 16 == 0 && kXm % 16 == 0 && kStart % 8 == 0 && kScan % 8 == 0, "alignment");
};

// Descriptor of the MN-major P operand: rows (keys) of PW bytes, PW-byte swizzle, 8-key
// groups 8 PW bytes apart.
template <int PW>
__device__ __forceinline__ uint64_t make_pdesc(uint32_t saddr) {
  constexpr uint64_t layout = PW == 128 ? 2 : (PW == 64 ? 4 : 6);
  return (uint64_t)((saddr >> 4) & 0x3FFFu) | ((uint64_t)(8 * PW >> 4) << 16) | ((uint64_t)(8 * PW >> 4) << 32) |
         (1ull << 46) | (layout << 61);
}

// Byte of 16-byte chunk c in P row k.
template <int PW>
__device__ __forceinline__ uint32_t p_off(uint32_t k, uint32_t c) {
  const uint32_t x = PW == 128 ? (k & 7) : (PW == 64 ? ((k >> 1) & 3) : ((k >> 2) & 1));
  return k * PW + ((c ^ x) << 4);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }
__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// e4m3 of (h16 - 16 t) for a pair: h16 fp16, t the e4m3 pair in the low 16 bits of w.
__device__ __forceinline__ uint32_t rest_e4m3(uint32_t h16, uint32_t w) {
  uint16_t r;
  asm("{\n\t.reg .b32 t, m;\n\t"
      "cvt.rn.f16x2.e4m3x2 t, %2;\n\t"
      "mov.b32 m, 0xcc00cc00;\n\t"  // -16
      "fma.rn.f16x2 t, t, m, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 %0, t;\n\t}"
      : "=h"(r) : "r"(h16), "h"((uint16_t)w));
  return r;
}

template <int D, int RP, int NP>
__global__ void __launch_bounds__(kDecThreads, Kv4Layout<D, RP, NP>::kCtas) attn_kv4_split_kernel(const __grid_constant__ KvDecArgs p) {
  using L = Kv4Layout<D, RP, NP>;
  constexpr bool BF16 = NP == 2;
  constexpr int TPR = L::TPR, TS = L::kTileShift, NB = L::kBufs;
  // (dynamic shared memory begins behind the 1024 bytes the system keeps: aligned as declared.
  // Three CTAs leave no room to align it here; a launch that it does not hold for gives up.)
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const uint32_t base = smem_u32(smem_raw);
  uint8_t* sbase = smem_raw;
  if (base & 1023u) {
    if (threadIdx.x == 0) atomicCAS(p.wait.status, kDevOk, kDevTimeout);
    return;
  }
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int Hr = p.H * p.n_rb;
  const WaitCtl wc{p.wait.status, p.wait.limit_ns};
  auto bar = [&](int i) -> uint32_t { return base + L::kBar + 8u * i; };

  if (warp == kWarpProd && lane == 0) {
    for (int s = 0; s < L::kStages; ++s) {
      mbar_init(bar(L::kBarKFull + s), 1);
      mbar_init(bar(L::kBarKEmpty + s), 1);
      mbar_init(bar(L::kBarVFull + s), 1);
      mbar_init(bar(L::kBarVEmpty + s), 1);
      mbar_init(bar(L::kBarCFull + s), 32);
      mbar_init(bar(L::kBarCEmpty + s), 1);
    }
    mbar_init(bar(L::kBarSFull), 2);
    mbar_init(bar(L::kBarSFull + 1), 2);
    mbar_init(bar(L::kBarPFull), 4);
    mbar_init(bar(L::kBarOFull), 1);
    mbar_init(bar(L::kBarQFull), 1);
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
  deal_range<TS, kDecThreads>(p, Hr, reinterpret_cast<long long*>(sbase + L::kScan),
                              reinterpret_cast<long long*>(sbase + L::kStart));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t*>(sbase + L::kTmemSlot);
  const Walk w0 = first_walk(reinterpret_cast<const long long*>(sbase + L::kStart));

  if (warp == kWarpProd) {
    // ------------------------------------------------------------ producer
    // Lane i takes page i of a tile: its id (read a tile ahead) and the copies of its
    // codes.  K is let go when S is there, V and the scales a tile's softmax later: K runs
    // a tile ahead of them.
    const int tile_pages = 1 << (TS - p.page_shift);
    const int row_shift = p.page_shift - (TPR - 1), page_rows = 1 << row_shift;
    if (!(p.debug_flags & 16)) {
      int gk = 0, gv = 0;  // tiles whose K, whose V and scales were asked for
      bool ok = true;
      int ph = -1, n_pages = 0;  // the tile whose V is next: (page, head) of the lane's page, pages
      auto load_k = [&] {
        const int s = gk % L::kStages;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarKEmpty + s), ((gk / L::kStages) & 1) ^ 1, wc));
        if (!ok) return;
        // (a row of codes counts as its 64 bytes in memory)
        if (lane == 0) mbar_expect_tx(bar(L::kBarKFull + s), n_pages * page_rows * 64);
        __syncwarp();
        if (lane < n_pages)
          tma_load_3d(base + L::kK + s * L::kCode + lane * page_rows * 128, &p.tm_k, bar(L::kBarKFull + s), 0, 0, ph);
        __syncwarp();
        ++gk;
      };
      auto load_v = [&](int ph_v, int n_v) {
        const int s = gv % L::kStages;
        const uint32_t par = ((gv / L::kStages) & 1) ^ 1;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarCEmpty + s), par, wc));
        if (!ok) return;
        // scales, two rows (16 bytes) a lane and copy; of pages that are not there zeros
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int row = 2 * (i * 32 + lane), pg = row >> row_shift;
          const int at_page = __shfl_sync(0xffffffffu, ph_v, pg);
          if (pg < n_v) {
            const size_t at = at_page < 0 ? 0 : (((size_t)at_page << row_shift) + (row & (page_rows - 1))) * 4;
            const uint32_t n = at_page < 0 ? 0 : 16, dst = base + L::kSc + s * 2 * L::kScl + row * 8;
            cp_async16(dst, p.k_scale16 + at, n);
            cp_async16(dst + L::kScl, p.v_scale16 + at, n);
          }
        }
        cp_async_arrive(bar(L::kBarCFull + s));
        ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarVEmpty + s), par, wc));
        if (!ok) return;
        if (lane == 0) mbar_expect_tx(bar(L::kBarVFull + s), n_v * page_rows * 64);
        __syncwarp();
        if (lane < n_v)
          tma_load_3d(base + L::kV + s * L::kCode + lane * page_rows * 128, &p.tm_v, bar(L::kBarVFull + s), 0, 0, ph_v);
        __syncwarp();
        ++gv;
      };
      Walk w = w0;
      Seg sg;
      while (ok && next_seg<TS>(p, Hr, w, sg)) {
        const int h = sg.hr / p.n_rb;
        const int pages = (sg.len + (1 << p.page_shift) - 1) >> p.page_shift;
        const int* row = p.table + (size_t)sg.b * p.width;
        auto page_id = [&](int t) -> int {
          const int j = t * tile_pages + lane;
          return lane < tile_pages && j < pages ? row[j] : -1;
        };
        int id = page_id(sg.t0);
        for (int t = sg.t0; t < sg.t1; ++t) {
          const int here = id, ph_v = ph, n_v = n_pages;
          if (t + 1 < sg.t1) id = page_id(t + 1);
          n_pages = min(tile_pages, pages - t * tile_pages);
          // (a page id outside the cache reads as zeros: the copies fill with them)
          ph = lane < n_pages && here >= 0 && here < p.P ? here * p.H + h : -1;
          load_k();
          if (ok && gk > 1) load_v(ph_v, n_v);
          if (!ok) break;
        }
      }
      if (ok && gk > gv) load_v(ph, n_pages);
      if (!ok) {  // copies in flight end before shared memory is left
        for (int i = max(0, gk - L::kStages); i < gk; ++i)
          mbar_wait_drain(bar(L::kBarKFull + i % L::kStages), (i / L::kStages) & 1, wc.limit_ns);
        for (int i = max(0, gv - L::kStages); i < gv; ++i)
          mbar_wait_drain(bar(L::kBarVFull + i % L::kStages), (i / L::kStages) & 1, wc.limit_ns);
        cp_async_wait_all();
      }
    }
  } else if (warp == kWarpMma) {
    // ------------------------------------------------------------ MMA warp
    constexpr uint32_t idesc_s = make_idesc_e2m1_e4m3(128, L::NS, false, false);
    constexpr uint32_t idesc_o = make_idesc_e2m1_e4m3(128, L::NO, true, true);
    auto wt = [&](int i, uint32_t parity) { return __all_sync(0xffffffffu, mbar_wait(bar(i), parity, wc)); };
    auto issue_s = [&](int g) {  // S^T = K (q terms)^T, the four groups of 32 channels apart
      const uint32_t k = base + L::kK + (g % L::kStages) * L::kCode, d_t = tmem + L::kColS + (g % NB) * 4 * L::kSet;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        mma_ss_f8(d_t + (L::kPair ? ks / 2 * L::NS : ks * L::NS), make_sdesc(k + ks * 32, 16, 1024),
                  make_sdesc(base + L::kQ + ks * 32, 16, 1024), idesc_s, L::kPair ? ks & 1 : 0);
      tc_commit(bar(L::kBarSFull + (g & 1)));
      tc_commit(bar(L::kBarKEmpty + g % L::kStages));
    };
    auto issue_o = [&](int g) {  // O^T = V^T (p terms)^T over the tile's rows
      const uint32_t v = base + L::kV + (g % L::kStages) * L::kCode, d_t = tmem + L::kColO + (g % NB) * L::NO;
#pragma unroll
      for (int ks = 0; ks < 4; ++ks)
        mma_ss_f8(d_t, make_sdesc(v + ks * 32 * 128, 16, 1024), make_pdesc<L::PW>(base + L::kP + ks * 32 * L::PW), idesc_o,
                  ks > 0);
      tc_commit(bar(L::kBarOFull));
      tc_commit(bar(L::kBarVEmpty + g % L::kStages));
    };
    // The power of two above the largest V scale of each group of channels in tile t.
    // (Rows behind the request's end hold anything.)
    auto norms = [&](int g, const Seg& sg, int t) {
      const int s = g % L::kStages;
      if (!wt(L::kBarCFull + s, (g / L::kStages) & 1)) return false;
      const uint4* sc = reinterpret_cast<const uint4*>(sbase + L::kSc + s * 2 * L::kScl + L::kScl);
      const int live = sg.len - (t << TS);  // tokens of the tile that there are, or more
      uint32_t a = 0, b = 0;                // largest magnitudes of groups 0 and 1, 2 and 3, as bits
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 v = sc[i * 32 + lane];  // rows 2 (32 i + lane) and the next
        const int tok = 2 * (i * 32 + lane) * TPR;
        if (tok < live) a = max_u16x2(a, v.x & 0x7fff7fffu);
        if (tok + TPR - 1 < live) b = max_u16x2(b, v.y & 0x7fff7fffu);
        if (tok + TPR < live) a = max_u16x2(a, v.z & 0x7fff7fffu);
        if (tok + 2 * TPR - 1 < live) b = max_u16x2(b, v.w & 0x7fff7fffu);
      }
      const uint32_t top[4] = {__reduce_max_sync(0xffffffffu, a & 0xffffu), __reduce_max_sync(0xffffffffu, a >> 16),
                               __reduce_max_sync(0xffffffffu, b & 0xffffu), __reduce_max_sync(0xffffffffu, b >> 16)};
      if (lane < 4) {
        const uint32_t m = lane == 0 ? top[0] : (lane == 1 ? top[1] : (lane == 2 ? top[2] : top[3]));
        // (a NaN among them says nothing of the others: its own scale makes its group a NaN)
        const int e = min(max((int)(m >> 7) - 126, -100), 100);
        float* n = reinterpret_cast<float*>(sbase + L::kNorm + s * 32);
        n[lane] = pow2f(-e);
        n[4 + lane] = pow2f(e);
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kBarSFull + (g & 1)));
      return true;
    };
    // The q terms of a segment's row block, eight lanes to a row: loaded (early), then
    // written where the last segment's products are done.
    constexpr int E = D / 8, kPass = RP / 4;  // elements per lane; four rows a pass
    uint4 qv[kPass][E / 8];
    auto load_q = [&](const Seg& sg) {
      const int h = sg.hr / p.n_rb, rb = sg.hr % p.n_rb;
#pragma unroll
      for (int ps = 0; ps < kPass; ++ps) {
        const int idx = rb * RP + ps * 4 + (lane >> 3), i = idx / p.G, hq = h * p.G + idx % p.G;
#pragma unroll
        for (int j = 0; j < E / 8; ++j) {
          qv[ps][j] = make_uint4(0, 0, 0, 0);
          if (idx < p.Nq * p.G)
            qv[ps][j] = reinterpret_cast<const uint4*>(static_cast<const uint8_t*>(p.q) +
                                                       ((((size_t)sg.b * p.Nq + i) * p.Hq + hq) * D + (lane & 7) * E) * 2)[j];
        }
      }
    };
    auto put_info = [&](int seg, int len, int t0, int t1, int nt) {
      if (lane == 0) *reinterpret_cast<int4*>(sbase + L::kInfo + (seg & 1) * 16) = make_int4(len, t0, t1, nt);
    };
    auto put_q = [&](const Seg& sg, int seg) {
      const int h = sg.hr / p.n_rb, rb = sg.hr % p.n_rb, c = lane & 7;
#pragma unroll
      for (int ps = 0; ps < kPass; ++ps) {
        const int r = ps * 4 + (lane >> 3);
        float f[E];
#pragma unroll
        for (int j = 0; j < E / 8; ++j) {
          const uint32_t* wv = &qv[ps][j].x;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float2 x = unpack2<BF16>(wv[e]);
            f[j * 8 + 2 * e] = x.x;
            f[j * 8 + 2 * e + 1] = x.y;
          }
        }
        uint32_t top = 0;  // largest magnitude, as bits (inf and NaN above all numbers)
#pragma unroll
        for (int j = 0; j < E; ++j) top = max(top, __float_as_uint(f[j]) & 0x7fffffffu);
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
        // 2^-e brings the row's largest into [128, 256)
        const int e = min(max((int)(top >> 23) - 127 - 7, -100), 119);
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
#pragma unroll
          for (int half = 0; half < TPR; ++half) {  // (d = 64: against both tokens of a row)
            const uint32_t byte = half * 64 + c * E;
            // (sets by twos: rows 0-7 hold the even groups, 8-15 the odd ones)
            const uint32_t row = t * RP + r + (L::kPair ? ((byte >> 5) & 1) * 8 : 0);
            uint32_t off = row * 128 + byte;
            off ^= ((off >> 7) & 7u) << 4;
            if constexpr (E == 16)
              *reinterpret_cast<uint4*>(sbase + L::kQ + off) = make_uint4(cw[0], cw[1], cw[2], cw[3]);
            else
              *reinterpret_cast<uint2*>(sbase + L::kQ + off) = make_uint2(cw[0], cw[1]);
          }
        }
        if (c == 0) {
          reinterpret_cast<float*>(sbase + L::kQs)[r] = bad ? __uint_as_float(0x7fc00000u) : pow2f(e) * p.scale * kLog2e;
          const int idx = rb * RP + r, i = idx / p.G, hq = h * p.G + idx % p.G;
          reinterpret_cast<int2*>(sbase + L::kRow)[(seg & 1) * RP + r] =
              idx < p.Nq * p.G ? make_int2((sg.b * p.Nq + i) * p.Hq + hq, (sg.b * p.Hq + hq) * p.Nq + i) : make_int2(-1, -1);
          sbase[L::kQi + (seg & 1) * RP + r] = (uint8_t)min(i, 127);
        }
      }
      put_info(seg, sg.len, sg.t0, sg.t1, sg.nt);
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kBarQFull));
    };
    if constexpr (L::kPair) {  // (the zeros of the sets by twos stay)
      for (int i = lane; i < L::NS * 128 / 16; i += 32) reinterpret_cast<uint4*>(sbase + L::kQ)[i] = make_uint4(0, 0, 0, 0);
      __syncwarp();
    }
    bool ok = true;
    int g = 0, seg = 0;
    Walk w = w0;
    Seg sg;
    bool more = next_seg<TS>(p, Hr, w, sg);
    if (more) load_q(sg);
    while (more) {
      put_q(sg, seg++);
      ok = wt(L::kBarKFull + g % L::kStages, (g / L::kStages) & 1);
      if (!ok) break;
      tc_fence_after();
      issue_s(g);
      ok = norms(g, sg, sg.t0);
      if (!ok) break;
      const Seg now = sg;
      more = next_seg<TS>(p, Hr, w, sg);
      if (more) load_q(sg);
      for (int t = now.t0; t < now.t1; ++t, ++g) {
        auto next_s = [&] {
          if (t + 1 < now.t1) {
            ok = wt(L::kBarKFull + (g + 1) % L::kStages, ((g + 1) / L::kStages) & 1);
            if (!ok) return;
            tc_fence_after();
            issue_s(g + 1);
            ok = norms(g + 1, now, t + 1);
          }
        };
        if (NB == 2) next_s();  // (with one buffer S of this tile has to be read first: P says so)
        if (!ok) break;
        ok = wt(L::kBarPFull, g & 1) && wt(L::kBarVFull + g % L::kStages, (g / L::kStages) & 1);
        if (!ok) break;
        tc_fence_after();
        issue_o(g);
        if (NB == 1) next_s();
        if (!ok) break;
      }
      if (!ok) break;
    }
    if (ok) {  // no more segments
      put_info(seg, 0, 0, 0, 0);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(L::kBarQFull));
    }
    tc_commit(bar(L::kBarDrain));
    mbar_wait_drain(bar(L::kBarDrain), 0, wc.limit_ns);
  } else {
    // ------------------------------------------------------------ softmax
    const int kl = threadIdx.x;  // row of the tile = TMEM lane of S^T; channel of the row = lane of O^T
    const uint32_t lane_off = (uint32_t)(warp * 32) << 16;
    const uint32_t tS = tmem + lane_off + L::kColS, tO = tmem + lane_off + L::kColO + warp * L::NG;
    float* xm = reinterpret_cast<float*>(sbase + L::kXm);
    float* xl = reinterpret_cast<float*>(sbase + L::kXl);
    float* qs_s = reinterpret_cast<float*>(sbase + L::kQs);
    uint8_t* prow = sbase + L::kP;
    bool ok = true;
    int g = 0;
    for (int seg = 0;; ++seg) {
      ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarQFull), seg & 1, wc));
      if (!named_bar_and(kWgBar, 128, ok)) break;
      const int4 info = *reinterpret_cast<const int4*>(sbase + L::kInfo + (seg & 1) * 16);
      const int len = info.x, t0 = info.y, t1 = info.z;
      if (t0 == t1) break;
      const int2* rows = reinterpret_cast<const int2*>(sbase + L::kRow) + (seg & 1) * RP;
      const uint8_t* qi = sbase + L::kQi + (seg & 1) * RP;
      float m[RP], l[RP], acc[RP];
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        m[r] = -INFINITY;
        l[r] = 0.f;
        acc[r] = 0.f;
      }
      const int lim0 = p.causal ? len - p.Nq : len - 1;  // tokens <= lim0 are seen by every row
      // O^T of a tile is added a tile later, while the tensor core works on the
      // next one: be is the factor of the tile whose O^T is outstanding (acc is
      // already on that tile's scale), the power of two of its V scales in it.
      float be[RP];
      auto add_o = [&](int go) {
        tc_fence_after();
        uint32_t r_[L::NG];
        tmem_ld_n<L::NG>(tO + (go % NB) * L::NO, r_);
        tmem_ld_wait();
        reg_fence<L::NG>(r_);
        tc_fence_before();
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          float o = __uint_as_float(r_[r]), c = __uint_as_float(r_[RP + r]);
          if constexpr (NP == 3) c = fmaf(__uint_as_float(r_[2 * RP + r]), 0.0625f, c);
          o = fmaf(c, 0.0625f, o);
          acc[r] = fmaf(o, be[r], acc[r]);
        }
      };
      for (int t = t0; t < t1; ++t, ++g) {
        const int st = g % L::kStages, kv0 = (t << TS) + kl * TPR;  // first token of this row
        const bool later = t > t0;  // the tile before is of this segment, its O^T outstanding
        // S^T, and with the scales' maxima the scales: the MMA warp has waited for them
        ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarSFull + (g & 1)), (g >> 1) & 1, wc));
        __align__(8) float x[TPR][RP];  // scores in log2 units
        float f[4], lv[TPR], mul = 0.f;
        if (ok) {
          tc_fence_after();
          const uint2 kw = *reinterpret_cast<const uint2*>(sbase + L::kSc + st * 2 * L::kScl + kl * 8);
          const uint2 vw = *reinterpret_cast<const uint2*>(sbase + L::kSc + st * 2 * L::kScl + L::kScl + kl * 8);
          const float4 inv = *reinterpret_cast<const float4*>(sbase + L::kNorm + st * 32);
          mul = *reinterpret_cast<const float*>(sbase + L::kNorm + st * 32 + 16 + warp * 4);
          const float ks[4] = {bf16_lo(kw.x), bf16_hi(kw.x), bf16_lo(kw.y), bf16_hi(kw.y)};
          f[0] = bf16_lo(vw.x) * inv.x;
          f[1] = bf16_hi(vw.x) * inv.y;
          f[2] = bf16_lo(vw.y) * inv.z;
          f[3] = bf16_hi(vw.y) * inv.w;
#pragma unroll
          for (int k = 0; k < 4; ++k)  // (a token behind the end has no weight, whatever its scales hold)
            if (kv0 + k * TPR / 4 >= len) f[k] = 0.f;
          // the largest weight of each token's value, at most 1
          if constexpr (TPR == 1) {
            lv[0] = __log2f(fmaxf(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])), 0x1p-30f));
          } else {
            lv[0] = __log2f(fmaxf(fmaxf(f[0], f[1]), 0x1p-30f));
            lv[1] = __log2f(fmaxf(fmaxf(f[2], f[3]), 0x1p-30f));
          }
          constexpr int kAt = L::NG <= 12 ? 4 : (L::NG <= 16 ? 2 : 1);  // groups loaded at a time
#pragma unroll
          for (int k0 = 0; k0 < 4; k0 += kAt) {
            uint32_t r_[kAt * L::NG];
            const uint32_t from = tS + (g % NB) * 4 * L::kSet + k0 * L::kSet;
            if constexpr (L::kSet == L::NG) {
              tmem_ld_n<kAt * L::NG>(from, r_);
            } else {
#pragma unroll
              for (int k = 0; k < kAt; ++k) tmem_ld_n<L::NG>(from + k * L::kSet, r_ + k * L::NG);
            }
            tmem_ld_wait();
            reg_fence<kAt * L::NG>(r_);
            constexpr int per = 4 / TPR;
#pragma unroll
            for (int k = 0; k < kAt; ++k) {
              const int j = (k0 + k) / per;
              const float2 k2 = make_float2(ks[k0 + k], ks[k0 + k]);
#pragma unroll
              for (int r = 0; r < RP; r += 2) {
                auto term = [&](int t2) {
                  const uint32_t* z = r_ + k * L::NG + t2 * RP + r;
                  return make_float2(__uint_as_float(z[0]), __uint_as_float(z[1]));
                };
                const float2 sixteenth = make_float2(0.0625f, 0.0625f);
                float2 c = term(1);
                if constexpr (NP == 3) c = fma2(term(2), sixteenth, c);
                const float2 s2 = fma2(c, sixteenth, term(0));
                float2* to = reinterpret_cast<float2*>(&x[j][r]);
                *to = (k0 + k) % per == 0 ? mul2(s2, k2) : fma2(s2, k2, *to);
              }
            }
          }
          tc_fence_before();
#pragma unroll
          for (int r = 0; r < RP; r += 2) {
            const float2 q2 = *reinterpret_cast<const float2*>(qs_s + r);
#pragma unroll
            for (int j = 0; j < TPR; ++j) {
              float2* to = reinterpret_cast<float2*>(&x[j][r]);
              *to = mul2(*to, q2);
            }
          }
          if ((t << TS) + (1 << TS) - 1 > lim0) {
#pragma unroll
            for (int r = 0; r < RP; ++r) {
              const int lim = p.causal ? min(len - 1, len - p.Nq + (int)qi[r]) : len - 1;
#pragma unroll
              for (int j = 0; j < TPR; ++j)
                if (kv0 + j > lim) x[j][r] = -INFINITY;
            }
          }
          float* mine = xm + ((g & 1) * 4 + warp) * RP;
#pragma unroll
          for (int r0 = 0; r0 < RP; r0 += 4) {
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              float y = x[0][r0 + j] + lv[0];
              if constexpr (TPR == 2) y = fmaxf(y, x[1][r0 + j] + lv[1]);
              v[j] = warp_max(y);
            }
            if (lane == 0) *reinterpret_cast<float4*>(mine + r0) = make_float4(v[0], v[1], v[2], v[3]);
          }
        }
        // (the O^T outstanding is complete: its MMA has read P, which is written again below)
        if (ok && later) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarOFull), (g - 1) & 1, wc));
        ok = named_bar_and(kWgBar, 128, ok);
        if (!ok) break;
        if (threadIdx.x == 0) mbar_arrive(bar(L::kBarCEmpty + st));  // (every warp has its scales)
        if (NB == 1 && later) add_o(g - 1);  // (before P lets the next O^T overwrite it)
        float al_t[RP], be_t[RP];
        uint32_t code[4][NP][RP / 4];  // terms of p f for the four groups, four rows to a word
#pragma unroll
        for (int r0 = 0; r0 < RP; r0 += 4) {
          float4 v[4];
#pragma unroll
          for (int q = 0; q < 4; ++q) v[q] = *reinterpret_cast<const float4*>(xm + ((g & 1) * 4 + q) * RP + r0);
          const float mt4[4] = {fmaxf(fmaxf(v[0].x, v[1].x), fmaxf(v[2].x, v[3].x)),
                                fmaxf(fmaxf(v[0].y, v[1].y), fmaxf(v[2].y, v[3].y)),
                                fmaxf(fmaxf(v[0].z, v[1].z), fmaxf(v[2].z, v[3].z)),
                                fmaxf(fmaxf(v[0].w, v[1].w), fmaxf(v[2].w, v[3].w))};
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int r = r0 + j;
            const float mt = mt4[j];
            // running maximum: one of the factors of the old and the new part is 1
            const float e = ex2(mt > m[r] ? m[r] - mt : mt - m[r]);
            al_t[r] = mt > m[r] ? e : 1.f;
            be_t[r] = (mt < m[r] ? e : 1.f) * 0.00390625f;  // p below carries 2^8
            m[r] = fmaxf(m[r], mt);
            const float ref = mt == -INFINITY ? 0.f : mt - 8.f;
            float sum = 0.f;
#pragma unroll
            for (int k = 0; k < TPR; ++k) {
              x[k][r] = ex2(x[k][r] - ref);  // p 2^8
              sum += x[k][r];
            }
            l[r] = fmaf(sum, be_t[r], l[r] * al_t[r]);
            be_t[r] *= mul;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2* pr = reinterpret_cast<const float2*>(&x[k * TPR / 4][r0]);
            const float2 f2 = make_float2(f[k], f[k]);
            float2 a = mul2(pr[0], f2), b = mul2(pr[1], f2);
            uint32_t lo = pack_e4m3(a.x, a.y), hi = pack_e4m3(b.x, b.y);
            code[k][0][r0 / 4] = lo | (hi << 16);
            if constexpr (NP == 2) {
              // (what the first term leaves, in fp16: 16 p f to 2^-11 less 16 times the term)
              const float2 g2 = make_float2(16.f * f[k], 16.f * f[k]);
              a = mul2(pr[0], g2);
              b = mul2(pr[1], g2);
              lo = rest_e4m3(pack2<false>(a.x, a.y), lo);
              hi = rest_e4m3(pack2<false>(b.x, b.y), hi);
              code[k][1][r0 / 4] = lo | (hi << 16);
            } else {
#pragma unroll
              for (int t2 = 1; t2 < NP; ++t2) {
                const float2 d0 = unpack_e4m3(lo), d1 = unpack_e4m3(hi), mul16 = make_float2(16.f, 16.f);
                a = mul2(sub2(a, d0), mul16);
                b = mul2(sub2(b, d1), mul16);
                lo = pack_e4m3(a.x, a.y);
                hi = pack_e4m3(b.x, b.y);
                code[k][t2][r0 / 4] = lo | (hi << 16);
              }
            }
          }
        }
        // row kl of P: column (group, term, row) one byte each
        const uint32_t* cw = &code[0][0][0];
#pragma unroll
        for (int c = 0; c < L::NO / 16; ++c)
          *reinterpret_cast<uint4*>(prow + p_off<L::PW>(kl, c)) = make_uint4(cw[4 * c], cw[4 * c + 1], cw[4 * c + 2], cw[4 * c + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kBarPFull));
        if (NB == 2 && later) add_o(g - 1);
#pragma unroll
        for (int r = 0; r < RP; ++r) {
          acc[r] *= al_t[r];
          be[r] = be_t[r];
        }
      }
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarOFull), (g - 1) & 1, wc));
      if (ok) add_o(g - 1);
      // ---- end of the segment: row sums over the tile's rows, then O.  A lane keeps half of its rows and
      // sends the others, until it has one, whose sum over the lanes that hold it goes on.
      {
        int row = 0;
#pragma unroll
        for (int n = RP / 2, o = 16; n > 0; n >>= 1, o >>= 1) {
          const bool up = lane & o;
          row = row * 2 + (up ? 1 : 0);
#pragma unroll
          for (int r = 0; r < n; ++r) {
            const float keep = up ? l[n + r] : l[r], send = up ? l[r] : l[n + r];
            l[r] = keep + __shfl_xor_sync(0xffffffffu, send, o);
          }
        }
#pragma unroll
        for (int o = 16 / RP; o > 0; o >>= 1) l[0] += __shfl_xor_sync(0xffffffffu, l[0], o);
        if (lane % (32 / RP) == 0) xl[row * 4 + warp] = l[0];
      }
      // (d = 64: lanes 64 to 127 hold the second token's part; P's rows are free)
      float* half = reinterpret_cast<float*>(prow);
      if (TPR == 2 && kl >= 64) {
#pragma unroll
        for (int r = 0; r < RP; ++r) half[r * 64 + kl - 64] = acc[r];
      }
      ok = named_bar_and(kWgBar, 128, ok);
      if (!ok) break;
      const bool whole = t1 - t0 == info.w;
#pragma unroll
      for (int r = 0; r < RP; ++r) {
        const int2 at = rows[r];
        const float4 l4 = *reinterpret_cast<const float4*>(xl + r * 4);
        const float lt = (l4.x + l4.y) + (l4.z + l4.w);
        const float sum = TPR == 2 && kl < 64 ? acc[r] + half[r * 64 + kl] : acc[r];
        if (at.x < 0) continue;
        if (whole) {
          const float v = lt != 0.f ? __fdividef(sum, lt) : 0.f;
          if (kl < D) reinterpret_cast<uint16_t*>(p.o)[(size_t)at.x * D + kl] = (uint16_t)pack2<BF16>(v, 0.f);
          if (kl == 0) p.lse[at.y] = lt != 0.f ? (m[r] + __log2f(lt)) * kLn2 : -INFINITY;
        } else {
          const size_t part = ((size_t)blockIdx.x * 2 + (seg > 0 ? 1 : 0)) * RP + r;
          if (kl < D) p.ws_o[part * D + kl] = sum;
          if (kl == 0) {
            p.ws_ml[part * 2] = m[r];
            p.ws_ml[part * 2 + 1] = lt;
          }
        }
      }
      // (the next segment's P and row sums are written behind the barrier of its first tile)
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

template <int D, int RP, int NP>
cudaError_t launch_split_t(const KvDecArgs& a, cudaStream_t stream) {
  using L = Kv4Layout<D, RP, NP>;
  auto* k = attn_kv4_split_kernel<D, RP, NP>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, (unsigned)a.grid, kDecThreads, L::kSmem, stream, a);
}

template <int D>
cudaError_t launch_split_d(const KvDecArgs& a, cudaStream_t stream) {
  if (a.bf16)
    return a.rp == 4 ? launch_split_t<D, 4, 2>(a, stream)
                     : (a.rp == 8 ? launch_split_t<D, 8, 2>(a, stream) : launch_split_t<D, 16, 2>(a, stream));
  return a.rp == 4 ? launch_split_t<D, 4, 3>(a, stream) : launch_split_t<D, 8, 3>(a, stream);
}

}  // namespace

template <int U>
static cudaError_t launch_append_u(const Kv4AppendArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.T + a.tok - 1) / a.tok), 2);
  cfg.blockDim = dim3(kAppThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (a.d == 128)
    return a.bf16 ? cudaLaunchKernelEx(&cfg, attn_kv4_append_kernel<128, true, U>, a)
                  : cudaLaunchKernelEx(&cfg, attn_kv4_append_kernel<128, false, U>, a);
  return a.bf16 ? cudaLaunchKernelEx(&cfg, attn_kv4_append_kernel<64, true, U>, a)
                : cudaLaunchKernelEx(&cfg, attn_kv4_append_kernel<64, false, U>, a);
}

cudaError_t launch_kv4_append(Kv4AppendArgs a, int sms, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  const long long per_tok = (long long)a.H * (a.d / 8);
  const int u = a.T * per_tok * 2 > 4ll * sms * 2048 ? 4 : 1;
  kv_rows(&a, (long long)kAppThreads * u / per_tok);
  return u == 4 ? launch_append_u<4>(a, stream) : launch_append_u<1>(a, stream);
}

// Row blocks of 4, 8 or, in bf16, 16 rows: the work per tile grows with the rows.  (16 rows of
// fp16 in three terms would take 384 columns of TMEM.)
int kv4_rows(int R, bool bf16) { return R <= 4 ? 4 : (R <= 8 || !bf16 ? 8 : 16); }

// All CTAs resident at once, no more than there can be tiles.
int kv4_grid(int rp, bool bf16, int sms, long long max_units) {
  long long g = (rp == 4 && bf16 ? 3ll : 2ll) * sms;
  if (g > kKvMaxCtas) g = kKvMaxCtas;
  if (g > max_units) g = max_units;
  return (int)(g < 1 ? 1 : g);
}

cudaError_t launch_kv4_split(const KvDecArgs& a, cudaStream_t stream) {
  return a.d == 128 ? launch_split_d<128>(a, stream) : launch_split_d<64>(a, stream);
}

}  // namespace attn
