// attn_kv4.cu -- a paged key/value cache held in 4 bits, for sm_103a.
//
// A cached value is s * c: c an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives), s a bf16 scale shared by 32 consecutive channels of one token
// and head.  4.5 bits a value; a token is rounded by itself, so nothing that is
// in the cache is ever rounded again.
//
// attn_kv4_append_kernel   rounds new keys and values into their slots.
// attn_kv4_split_kernel    O = softmax(s q K^T) V over the cache, split (joined by
//                          attn_kv_merge_kernel or within clusters).
//
// Decoding streams the codes and scales once, 1.125 d bytes a key and head.  As in the
// cache in 8 bits no thread converts a cached value: TMA copies the packed codes and
// spreads them over shared memory as the tensor core takes e2m1 (16 codes in 8 bytes,
// 8 bytes unused), and the *other* operand of each product is a short sum of e4m3
// terms (see attn_kv8.cu).  What is new is that the scales change along d and from token
// to token.  With groups g of 32 channels, which is one k-step of the MMA,
//   s_j      = sum_g ks[j][g] (K_g q_g^T)_j           the four k-steps of S^T go to columns of their own
//                                                     and are added by the thread that owns the key
//   O[c in g] = sum_j code[j][c] (p_j vs[j][g])       P has a set of columns for each group, with the
//                                                     scale multiplied in; a warp of the accumulator's
//                                                     lanes, 32 channels, reads its own group's set
// A row of an operand is 128 channels: a token at d = 128, two at d = 64 (the query then stands twice in
// its row, and P's sets belong to the first and the second token), so both sizes are one kernel.
//
// P's numbers fill e4m3's range whatever the scales are: group g is measured by a power of two above the
// largest vs[.][g] of the tile (at d = 64 of both tokens of its rows: measured apart, the other one's P could
// fall among e4m3's subnormals), found by the MMA warp while it waits, and the row's reference is
// the maximum of s_j + log2 u_j, u_j the token's largest measured scale (or 2^-80).  l sums 2^(s - m) without the scales.
//
// Work: deal and merge as attn_kv8.cu, or, for few or short requests, a cluster of CTAs to a segment
// (kv4_cluster), which joins its parts through shared memory.  Three rings of stages, for K, V and scales:
// K is let go when S is there, a softmax earlier than V, which keeps twice as much in flight (with one ring
// for all, four long requests took 107 us, 86 with one CTA less and a stage more, 80 with three rings).
//
// Measured (graph replay, bf16, d = 128): four requests of 50001 to 131072 tokens, 32 query and 8 key heads, 450 MB:
// 75.8 us or 5.9 TB/s, 88 % of the measured copy bandwidth (from tile to tile 97 %; the rest is the start, the
// uneven ends and the merge); 64 requests of 100 to 8192 tokens, 130 MB: 31.7 us; one of 1000 tokens: 5.3 us behind
// a table of that length, 8.0 behind a wide one (kv4_cluster).
// The tensor pipe is 9 % busy, the warp schedulers 47 %.  With 8 and 16 query rows the conversions and
// the softmax bound it: 0.6 and 1.2 us a tile and SM, 0.43 with 4 rows, which is the memory's rate.
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

__device__ __forceinline__ uint32_t max_s16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.s16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// Bound by memory for long prompts (256k tokens of 8 heads, d = 128, 1.35 GB: 264 us or 5.1 TB/s) and half by its
// own instructions (issue slots 45 %), by its launch for a decoding step (256 tokens 1.7 us in a graph).
// A thread rounds 16 channels (32 bytes in, 8 out), two neighbours share a scale.  A block
// takes p.tok tokens of K or of V (blockIdx.y), all their heads.  W32: tokens begin on
// 32-byte borders, and a thread's channels are read at once.  AHEAD: the next item is read
// before this one is rounded.
template <int D, bool BF16, bool W32, bool AHEAD>
__global__ void __launch_bounds__(kAppThreads) attn_kv4_append_kernel(const __grid_constant__ Kv4AppendArgs p) {
  griddep_wait();
  constexpr int kParts = D / 16;  // threads to a token and head
  const int kv = blockIdx.y;
  const long long t0 = (long long)blockIdx.x * p.tok;
  const int n_tok = (int)min((long long)p.tok, p.T - t0);
  const int items = n_tok * p.H * kParts;
  const uint8_t* x = static_cast<const uint8_t*>(p.x[kv]);
  const int ps = 1 << p.page_shift;
  auto fetch = [&](int i, uint32_t* w, long long& at) {  // (w on a 16-byte border)
    const int row = i / kParts, part = i % kParts;
    const int tl = (int)__umulhi((uint32_t)row * 2, p.h_magic), h = row - tl * p.H;
    at = -1;
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 0;
    if (i < items) {
      const long long t = t0 + tl, slot = p.slots[t];
      const uint8_t* src = x + (t * p.x_stride[kv] + (long long)h * D + part * 16) * 2;
      if constexpr (W32) {
        ld_global_32(src, w);
      } else {
        *reinterpret_cast<uint4*>(w) = *reinterpret_cast<const uint4*>(src);
        *reinterpret_cast<uint4*>(w + 4) = *reinterpret_cast<const uint4*>(src + 16);
      }
      if (slot >= 0 && slot < p.n_slots)
        at = ((((slot >> p.page_shift) * p.H + h) << p.page_shift) + (slot & (ps - 1))) * kParts + part;
    }
  };
  __align__(16) uint32_t next[8];
  long long next_at = -1;  // (page, head, place) of an item, -1: none
  if constexpr (AHEAD) fetch(threadIdx.x, next, next_at);
  for (int i = threadIdx.x; i - (int)threadIdx.x < items; i += kAppThreads) {
    __align__(16) uint32_t w[8];
    long long at = next_at;
    if constexpr (AHEAD) {
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] = next[j];
      if (i - (int)threadIdx.x + kAppThreads < items) fetch(i + kAppThreads, next, next_at);
    } else {
      fetch(i, w, at);
    }
    // largest magnitude as the 16 bits of it: ordered as numbers, infinity and NaN above all
    uint32_t top = w[0] & 0x7fff7fffu;
#pragma unroll
    for (int j = 1; j < 8; ++j) top = max_u16x2(top, w[j] & 0x7fff7fffu);
    top = max_u16x2(top, __shfl_xor_sync(0xffffffffu, top, 1));
    top = max(top & 0xffffu, top >> 16);
    const float amax = unpack2<BF16>(top).x;
    // s = amax / 6 rounded to bf16.  (The quotient of 11 bits by 6 is exact in 32 bits where
    // it lies half-way between two bf16 values, so rounding it twice is rounding it once.)
    // fminf and fmaxf pass a NaN over, so a NaN is put back.
    const float f = fminf(fmaxf(__fdiv_rn(amax, 6.f), 0x1p-64f), 0x1p60f);
    const uint32_t sb = amax != amax ? 0x7fc0u : (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rn(f));
    const float s = __uint_as_float(sb << 16), inv = 1.f / s;
    float2 y[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float2 n = unpack2<BF16>(w[j] ^ 0x80008000u);  // -x
      if (amax > 0x1p63f) {  // (beyond the largest scale: saturated below; an infinity has no residual)
        n.x = fminf(fmaxf(n.x, -0x1p63f), 0x1p63f);
        n.y = fminf(fmaxf(n.y, -0x1p63f), 0x1p63f);
      }
      // x / s to 32 bits: the product with 1 / s, corrected by its residual.  A quotient of 11 by 8
      // bits that is no border between two codes is at least 2^-12 of its value away from it; one
      // that is comes out exactly.  (From -x, so that a zero keeps its sign.)
      y[j] = mul2(n, make_float2(-inv, -inv));
      const float2 r = fma2(y[j], make_float2(s, s), n);
      y[j] = fma2(r, make_float2(-inv, -inv), y[j]);
    }
    if (at >= 0) {
      *reinterpret_cast<uint2*>(p.cache[kv] + at * 8) =
          make_uint2(pack8_e2m1(y[0], y[1], y[2], y[3]), pack8_e2m1(y[4], y[5], y[6], y[7]));
      if ((i & 1) == 0) p.scale[kv][at >> 1] = (uint16_t)sb;
    }
  }
  if (threadIdx.x == 0) griddep_launch_dependents();
}

// ------------------------------------------------------------------ decode
__host__ __device__ constexpr int up1024(int x) { return (x + 1023) / 1024 * 1024; }

// A row is 128 channels: a token (d = 128) or two (d = 64).  A tile is 128 rows.  WG
// warpgroups of softmax take four query rows each.
template <int D, int WG, int NP>
struct Kv4Layout {
  static constexpr int TPR = 128 / D;                 // tokens to a row
  static constexpr int kTileShift = D == 128 ? 7 : 8; // tokens to a tile
  static constexpr int RP = 4 * WG;                   // query rows
  // warps: softmax, producer, MMA (with query terms and scale maxima)
  static constexpr int kWarpProd = 4 * WG, kWarpMma = 4 * WG + 1, kWarps = 4 * WG + 2, kThreads = kWarps * 32;
  static constexpr int N4 = 4 * NP;                   // operand rows of a warpgroup: its rows times terms
  static constexpr int NG = RP * NP;                  // of all
  // S^T has a set of NG columns for each group of 32 channels.  M = 128 takes columns by 16: eight are
  // written by twos, a set with the next one (the other's rows of the query operand are zeros there).
  static constexpr bool kPair = NG == 8;
  static constexpr int NS = kPair ? 16 : (NG + 15) / 16 * 16;  // MMA columns
  static constexpr int kSet = kPair ? 8 : NS;         // columns from one set to the next
  static constexpr int NO = 4 * NG;                   // O^T: a set for each warpgroup and group of channels
  static constexpr int PW = NO <= 32 ? 32 : (NO <= 64 ? 64 : 128);  // bytes of a P row, and its swizzle
  // CTAs to an SM and stages, by what shared memory, TMEM and registers leave
  static constexpr int kSegCost = kv4_seg_cost(RP, NP == 2);
  static constexpr int kCtas = WG == 4 ? 1 : (PW == 32 ? 3 : 2);
  static constexpr int kStages = WG == 4 ? 5 : (PW == 64 ? 3 : 2);
  static constexpr int kCode = 128 * 128;             // bytes of a tile's codes: 16 to 16 bytes, 8 of them filled
  static constexpr int kScl = 128 * 8;                // bytes of its scales: four bf16 a row
  static constexpr int kQ = 0;
  static constexpr int kP = kQ + up1024(NS * 128);
  // three rings: K codes, V codes, scales (stage s: K's at + s * 2 kScl, V's behind them)
  static constexpr int kK = kP + up1024(128 * PW);
  static constexpr int kV = kK + kStages * kCode;
  static constexpr int kSc = kV + kStages * kCode;
  static constexpr int kNorm = kSc + kStages * 2 * kScl;  // [stages][4] 2^-e, [4] 2^e: powers above the groups' largest V scale
  static constexpr int kXm = kNorm + kStages * 32;    // [2][WG][4 warps][4 rows] fp32 row maxima
  static constexpr int kXl = kXm + 2 * WG * 64;       // [RP][4 warps] fp32 row sums
  static constexpr int kQs = kXl + RP * 16;           // [RP] fp32 row factors
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
  static constexpr int kStart = kTmemSlot + 8;        // start of the CTA's range: long long u0, u1; int b, hr, t
  static constexpr int kScan = kXm;                   // [kWarps] warp sums of the prologue
  static constexpr int kSmem = kStart + 32;
  // TMEM: two buffers of S^T and of O^T where the columns are there, else one
  static constexpr int kMaxCols = kCtas == 3 ? 128 : (kCtas == 2 ? 256 : 512);
  static constexpr int kBufs = 2 * (4 * kSet + NO) <= kMaxCols ? 2 : 1;
  static constexpr int kCols = kBufs * (4 * kSet + NO) <= 128 ? 128 : (kBufs * (4 * kSet + NO) <= 256 ? 256 : 512);
  static constexpr int kColS = 0, kColO = kBufs * 4 * kSet;
  static_assert(kBufs * (4 * kSet + NO) <= kCols && kCols * kCtas <= 512, "TMEM budget");
  static_assert((kSmem + 1024) * kCtas <= 228 * 1024, "shared memory budget");
  static_assert(NO % 16 == 0 && NO <= PW && kWarps * 8 <= 2 * WG * 64, "P rows, scan");
  static_assert(kBar % 8 == 0 && kNorm % 16 == 0 && kXm % 16 == 0 && kInfo % 16 == 0 && kStart % 8 == 0, "alignment");
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

// Four fp32 values to e4m3, from the lowest byte up.
__device__ __forceinline__ uint32_t pack4_e4m3(float2 a, float2 b) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 lo, %2, %1;\n\t"
      "cvt.rn.satfinite.e4m3x2.f32 hi, %4, %3;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r) : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// e4m3 of (h - 16 t) for four values: h fp16 (two pairs), t the e4m3 values of w.
__device__ __forceinline__ uint32_t rest4_e4m3(uint32_t h_lo, uint32_t h_hi, uint32_t w) {
  uint32_t r;
  asm("{\n\t.reg .b16 lo, hi;\n\t.reg .b32 a, b, m;\n\t"
      "mov.b32 {lo, hi}, %3;\n\t"
      "cvt.rn.f16x2.e4m3x2 a, lo;\n\t"
      "cvt.rn.f16x2.e4m3x2 b, hi;\n\t"
      "mov.b32 m, 0xcc00cc00;\n\t"  // -16
      "fma.rn.f16x2 a, a, m, %1;\n\t"
      "fma.rn.f16x2 b, b, m, %2;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 lo, a;\n\t"
      "cvt.rn.satfinite.e4m3x2.f16x2 hi, b;\n\t"
      "mov.b32 %0, {lo, hi};\n\t}"
      : "=r"(r) : "r"(h_lo), "r"(h_hi), "r"(w));
  return r;
}

constexpr float kNone = -3e38f;  // the maximum of scores that are all masked
// A token's values count for the row's reference as this much of the tile's largest scale, if they are smaller: p is at
// most 2^88 then, and its sum over 2^31 tokens below the 2^126 that __fdividef takes.  (A zero value whose token has
// 2^gap times the others' weight lifts the reference by gap - 80: below that the others' P keeps its precision.  With
// 2^-30 it was off by 1 % at a gap of 45 and gone at 55.)
constexpr float kLeast = 0x1p-80f;

// CL: a cluster of p.cluster CTAs takes one segment, whose tiles are dealt to them evenly, and joins
// their parts through shared memory: no merge kernel, and no sums over the lengths to begin with.
template <int D, int WG, int NP, bool CL>
__global__ void __launch_bounds__(Kv4Layout<D, WG, NP>::kThreads, Kv4Layout<D, WG, NP>::kCtas)
    attn_kv4_split_kernel(const __grid_constant__ KvDecArgs p) {
  using L = Kv4Layout<D, WG, NP>;
  constexpr int RP = L::RP, kWarpProd = L::kWarpProd, kWarpMma = L::kWarpMma;
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
      mbar_init(bar(L::kBarCEmpty + s), WG);
    }
    mbar_init(bar(L::kBarSFull), 2);
    mbar_init(bar(L::kBarSFull + 1), 2);
    mbar_init(bar(L::kBarPFull), 4 * WG);
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
  // What comes next may be scheduled as CTAs end: the merge kernel looks at the lengths meanwhile.  The warp that
  // says so has its tensor memory: a kernel that took it first would wait for this one, which could not begin.
  if (threadIdx.x == kWarpMma * 32) griddep_launch_dependents();
  Walk w0;
  Seg mine;  // CL: the segment
  const int rank = CL ? (int)(blockIdx.x % (unsigned)p.cluster) : 0;
  if constexpr (CL) {
    const unsigned seg = blockIdx.x / (unsigned)p.cluster;
    mine.b = (int)(seg / (unsigned)Hr);
    mine.hr = (int)(seg - (unsigned)mine.b * Hr);
    mine.len = kv_len(p, mine.b);
    mine.nt = kv_tiles<TS>(mine.len);
    const int per = (mine.nt + p.cluster - 1) / p.cluster;
    mine.t0 = min(mine.nt, rank * per);
    mine.t1 = min(mine.nt, mine.t0 + per);
    w0.left = mine.t1 - mine.t0;
  } else if (p.B <= kWarpDealB) {
    w0 = deal_warp<TS, L::kSegCost>(p, Hr);
  } else {
    deal_range<TS, L::kSegCost, L::kThreads>(p, Hr, reinterpret_cast<long long*>(sbase + L::kScan),
                                             reinterpret_cast<long long*>(sbase + L::kStart));
    __syncthreads();
    w0 = first_walk(reinterpret_cast<const long long*>(sbase + L::kStart));
    __syncthreads();  // (the scan lies where the row maxima will)
  }
  auto next_segment = [&](Walk& w, Seg& sg) {
    if constexpr (CL) {
      const bool first = w.left > 0;
      w.left = 0;
      sg = mine;
      return first;
    } else {
      return next_seg<TS, L::kSegCost>(p, Hr, w, sg);
    }
  };
  // Barriers and TMEM are there for the warps that wait here; the producer, which made the
  // barriers, goes on.
  uint32_t tmem = 0;
  if (warp == kWarpProd) {
    __syncwarp();
    named_bar_arrive(2 + WG, L::kThreads);
  } else {
    tc_fence_before();
    named_bar_sync(2 + WG, L::kThreads);
    tc_fence_after();
    tmem = *reinterpret_cast<volatile uint32_t*>(sbase + L::kTmemSlot);
  }

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
      while (ok && next_segment(w, sg)) {
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
      // Magnitudes as bits + 0x7f, so that a NaN, negative as 16 signed bits, does not count: its own scale makes
      // its group a NaN, and the others are measured without it.
      uint32_t a = 0x007f007fu, b = a;  // the largest of groups 0 and 1, 2 and 3
      auto with = [](uint32_t top, uint32_t v) { return max_s16x2(top, (v & 0x7fff7fffu) + 0x007f007fu); };
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint4 v = sc[i * 32 + lane];  // rows 2 (32 i + lane) and the next
        const int tok = 2 * (i * 32 + lane) * TPR;
        if (tok < live) a = with(a, v.x);
        if (tok + TPR - 1 < live) b = with(b, v.y);
        if (tok + TPR < live) a = with(a, v.z);
        if (tok + 2 * TPR - 1 < live) b = with(b, v.w);
      }
      if (TPR == 2) a = max_s16x2(a, b);  // one measure for the first and the second tokens of the rows
      uint32_t top[4] = {__reduce_max_sync(0xffffffffu, a & 0xffffu), __reduce_max_sync(0xffffffffu, a >> 16)};
      top[2] = TPR == 2 ? top[0] : __reduce_max_sync(0xffffffffu, b & 0xffffu);
      top[3] = TPR == 2 ? top[1] : __reduce_max_sync(0xffffffffu, b >> 16);
      if (lane < 4) {
        const uint32_t m = (lane == 0 ? top[0] : (lane == 1 ? top[1] : (lane == 2 ? top[2] : top[3]))) - 0x7f;
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
    constexpr int E = D / 8;  // elements per lane; four rows, those of a warpgroup, at a time
    uint4 qv[WG][E / 8];
    auto load_q = [&](const Seg& sg) {
      const int h = sg.hr / p.n_rb, rb = sg.hr % p.n_rb;
#pragma unroll
      for (int ps = 0; ps < WG; ++ps) {
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
      for (int ps = 0; ps < WG; ++ps) {
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
#pragma unroll
          for (int half = 0; half < TPR; ++half) {  // (d = 64: against both tokens of a row)
            const uint32_t byte = half * 64 + c * E;
            // (sets by twos: rows 0-7 hold the even groups, 8-15 the odd ones)
            const uint32_t row = ps * L::N4 + t * 4 + (lane >> 3) + (L::kPair ? ((byte >> 5) & 1) * 8 : 0);
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
    bool more = next_segment(w, sg);
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
      more = next_segment(w, sg);
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
    // All of a segment's barriers are passed by all warps, however a wait ends: the one over
    // all warpgroups at its start and at its end, and within the tiles those of a warpgroup.
    const int wg = warp >> 2, qw = warp & 3;
    const int kl = threadIdx.x & 127;  // row of the tile = TMEM lane of S^T; channel of the row = lane of O^T
    const uint32_t lane_off = (uint32_t)(qw * 32) << 16;
    const uint32_t tS = tmem + lane_off + L::kColS + wg * L::N4;
    const uint32_t tO = tmem + lane_off + L::kColO + (wg * 4 + qw) * L::N4;
    float* xl = reinterpret_cast<float*>(sbase + L::kXl) + wg * 16;
    const float4* qs = reinterpret_cast<const float4*>(sbase + L::kQs) + wg;
    uint8_t* prow = sbase + L::kP;
    // CL: the CTA's part, where K was (all of its copies have been waited for)
    float* part_o = reinterpret_cast<float*>(sbase + L::kK);
    float2* part_ml = reinterpret_cast<float2*>(sbase + L::kK + RP * 512);
    const uint32_t all_bar = 1, wg_bar = WG == 1 ? 1 : 2 + wg;  // hardware barriers
    int g = 0, st = 0;
    for (int seg = 0;; ++seg) {
      bool ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarQFull), seg & 1, wc));
      if (!named_bar_and(all_bar, 128 * WG, ok)) break;
      const int4 info = *reinterpret_cast<const int4*>(sbase + L::kInfo + (seg & 1) * 16);
      const int len = info.x, t0 = info.y, t1 = info.z;
      if (t0 == t1) break;
      const uint8_t* qi = sbase + L::kQi + (seg & 1) * RP + wg * 4;
      float m[4], l[4], acc[4];  // sums of 2^(x - m), m the running maximum less 8: what P carries
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        m[r] = kNone;
        l[r] = 0.f;
        acc[r] = 0.f;
      }
      const int lim0 = p.causal ? len - p.Nq : len - 1;  // tokens <= lim0 are seen by every row
      // O^T of a tile is added a tile later, while the tensor core works on the
      // next one: be is the factor of the tile whose O^T is outstanding (acc is
      // already on that tile's scale), the power of two of its V scales in it.
      float be[4];
      auto add_o = [&](int go) {
        tc_fence_after();
        uint32_t r_[L::N4];
        tmem_ld_n<L::N4>(tO + (go % NB) * L::NO, r_);
        tmem_ld_wait();
        reg_fence<L::N4>(r_);
        tc_fence_before();
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          float o = __uint_as_float(r_[r]), c = __uint_as_float(r_[4 + r]);
          if constexpr (NP == 3) c = fmaf(__uint_as_float(r_[8 + r]), 0.0625f, c);
          o = fmaf(c, 0.0625f, o);
          acc[r] = fmaf(o, be[r], acc[r]);
        }
      };
      for (int t = t0; t < t1; ++t, ++g, st = st + 1 == L::kStages ? 0 : st + 1) {
        const int kv0 = (t << TS) + kl * TPR;  // first token of this row
        const bool later = t > t0;  // the tile before is of this segment, its O^T outstanding
        // S^T, and with the scales' maxima the scales: the MMA warp has waited for them
        ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarSFull + (g & 1)), (g >> 1) & 1, wc));
        float2 x[TPR][2];  // scores in log2 units
        float f[4], lv[TPR], mul = 0.f;
        float4* xm = reinterpret_cast<float4*>(sbase + L::kXm) + ((g & 1) * WG + wg) * 4;
        if (ok) {
          tc_fence_after();
          uint32_t r_[4 * L::N4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            if constexpr (L::kPair) {
              if (k == 0) tmem_ld_n<4 * L::N4>(tS + (g % NB) * 4 * L::kSet, r_);
            } else {
              tmem_ld_n<L::N4>(tS + (g % NB) * 4 * L::kSet + k * L::kSet, r_ + k * L::N4);
            }
          }
          const uint2 kw = *reinterpret_cast<const uint2*>(sbase + L::kSc + st * 2 * L::kScl + kl * 8);
          const uint2 vw = *reinterpret_cast<const uint2*>(sbase + L::kSc + st * 2 * L::kScl + L::kScl + kl * 8);
          const float4 inv = *reinterpret_cast<const float4*>(sbase + L::kNorm + st * 32);
          const float4 q4 = *qs;
          mul = *reinterpret_cast<const float*>(sbase + L::kNorm + st * 32 + 16 + qw * 4);
          const float ks[4] = {bf16_lo(kw.x), bf16_hi(kw.x), bf16_lo(kw.y), bf16_hi(kw.y)};
          f[0] = bf16_lo(vw.x) * inv.x;
          f[1] = bf16_hi(vw.x) * inv.y;
          f[2] = bf16_lo(vw.y) * inv.z;
          f[3] = bf16_hi(vw.y) * inv.w;
          if ((t + 1) << TS > len) {  // (a token behind the end has no weight, whatever its scales hold)
#pragma unroll
            for (int k = 0; k < 4; ++k)
              if (kv0 + k * TPR / 4 >= len) f[k] = 0.f;
          }
          // the largest weight of each token's value, at most 1
          if constexpr (TPR == 1) {
            lv[0] = __log2f(fmaxf(fmaxf(fmaxf(f[0], f[1]), fmaxf(f[2], f[3])), kLeast));
          } else {
            lv[0] = __log2f(fmaxf(fmaxf(f[0], f[1]), kLeast));
            lv[1] = __log2f(fmaxf(fmaxf(f[2], f[3]), kLeast));
          }
          tmem_ld_wait();
          reg_fence<4 * L::N4>(r_);
          tc_fence_before();
          constexpr int per = 4 / TPR;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 k2 = make_float2(ks[k], ks[k]), sixteenth = make_float2(0.0625f, 0.0625f);
#pragma unroll
            for (int r = 0; r < 2; ++r) {
              auto term = [&](int t2) {
                const uint32_t* z = r_ + k * L::N4 + t2 * 4 + r * 2;
                return make_float2(__uint_as_float(z[0]), __uint_as_float(z[1]));
              };
              float2 c = term(1);
              if constexpr (NP == 3) c = fma2(term(2), sixteenth, c);
              const float2 s2 = fma2(c, sixteenth, term(0));
              float2& to = x[k / per][r];
              to = k % per == 0 ? mul2(s2, k2) : fma2(s2, k2, to);
            }
          }
#pragma unroll
          for (int j = 0; j < TPR; ++j) {
            x[j][0] = mul2(x[j][0], make_float2(q4.x, q4.y));
            x[j][1] = mul2(x[j][1], make_float2(q4.z, q4.w));
          }
          if ((t << TS) + (1 << TS) - 1 > lim0) {
            const uint32_t q8 = *reinterpret_cast<const uint32_t*>(qi);
#pragma unroll
            for (int r = 0; r < 4; ++r) {
              const int lim = p.causal ? min(len - 1, len - p.Nq + (int)((q8 >> (8 * r)) & 255)) : len - 1;
#pragma unroll
              for (int j = 0; j < TPR; ++j)
                if (kv0 + j > lim) (r & 1 ? x[j][r / 2].y : x[j][r / 2].x) = -INFINITY;
            }
          }
          float2 y[2];
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            y[r] = add2(x[0][r], make_float2(lv[0], lv[0]));
            if constexpr (TPR == 2) {
              const float2 z = add2(x[1][r], make_float2(lv[1], lv[1]));
              y[r] = make_float2(fmaxf(y[r].x, z.x), fmaxf(y[r].y, z.y));
            }
          }
          const float4 top = make_float4(warp_max(y[0].x), warp_max(y[0].y), warp_max(y[1].x), warp_max(y[1].y));
          if (lane == 0) xm[qw] = top;
        }
        // (the O^T outstanding is complete: its MMA has read P, which is written again below)
        if (ok && later) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarOFull), (g - 1) & 1, wc));
        ok = named_bar_and(wg_bar, 128, ok);
        if (!ok) break;
        if (kl == 0) mbar_arrive(bar(L::kBarCEmpty + st));  // (every warp of the group has its scales)
        if (NB == 1 && later) add_o(g - 1);  // (before P lets the next O^T overwrite it)
        const float4 v0 = xm[0], v1 = xm[1], v2 = xm[2], v3 = xm[3];
        const float mt4[4] = {max3(max3(v0.x, v1.x, v2.x), v3.x, kNone) - 8.f, max3(max3(v0.y, v1.y, v2.y), v3.y, kNone) - 8.f,
                              max3(max3(v0.z, v1.z, v2.z), v3.z, kNone) - 8.f, max3(max3(v0.w, v1.w, v2.w), v3.w, kNone) - 8.f};
        float al_t[4], be_t[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          // running maximum: one of the factors of the old and the new part is 1
          const float d = mt4[r] - m[r], e = ex2(-fabsf(d));
          al_t[r] = d > 0.f ? e : 1.f;
          const float be_r = d < 0.f ? e : 1.f;
          m[r] = fmaxf(m[r], mt4[r]);
          float sum = 0.f;
#pragma unroll
          for (int j = 0; j < TPR; ++j) {
            float& y = r & 1 ? x[j][r / 2].y : x[j][r / 2].x;
            y = ex2(y - mt4[r]);  // p 2^8
            sum += y;
          }
          l[r] = fmaf(sum, be_r, l[r] * al_t[r]);
          be_t[r] = be_r * mul;
        }
        uint32_t code[4][NP];  // terms of p f for the four groups of channels, four rows to a word
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2* pr = x[k * TPR / 4];
          const float2 f2 = make_float2(f[k], f[k]);
          float2 a = mul2(pr[0], f2), b = mul2(pr[1], f2);
          const float2 mul16 = make_float2(16.f, 16.f);
          code[k][0] = pack4_e4m3(a, b);
          if constexpr (NP == 2) {  // what the first term leaves, in fp16: 16 p f to 2^-11 less 16 times the term
            a = mul2(a, mul16);
            b = mul2(b, mul16);
            code[k][1] = rest4_e4m3(pack2<false>(a.x, a.y), pack2<false>(b.x, b.y), code[k][0]);
          } else {
#pragma unroll
            for (int t2 = 1; t2 < NP; ++t2) {
              a = mul2(sub2(a, unpack_e4m3(code[k][t2 - 1] & 0xffffu)), mul16);
              b = mul2(sub2(b, unpack_e4m3(code[k][t2 - 1] >> 16)), mul16);
              code[k][t2] = pack4_e4m3(a, b);
            }
          }
        }
        // row kl of P: column (warpgroup, group, term, row) one byte each
        const uint32_t* cw = &code[0][0];
#pragma unroll
        for (int c = 0; c < NP; ++c)
          *reinterpret_cast<uint4*>(prow + p_off<L::PW>(kl, wg * NP + c)) =
              make_uint4(cw[4 * c], cw[4 * c + 1], cw[4 * c + 2], cw[4 * c + 3]);
        fence_proxy_async_smem();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(L::kBarPFull));
        if (NB == 2 && later) add_o(g - 1);
#pragma unroll
        for (int r = 0; r < 4; ++r) {
          acc[r] *= al_t[r];
          be[r] = be_t[r];
        }
      }
      if (ok) ok = __all_sync(0xffffffffu, mbar_wait(bar(L::kBarOFull), (g - 1) & 1, wc));
      if (ok) add_o(g - 1);
      // ---- end of the segment: row sums over the tile's rows, then O.  A lane keeps half of its rows and
      // sends the others, until it has one, whose sum over the lanes that hold it goes on.
      {
        const bool up = lane & 16, up2 = lane & 8;
        const float s0 = (up ? l[2] : l[0]) + __shfl_xor_sync(0xffffffffu, up ? l[0] : l[2], 16);
        const float s1 = (up ? l[3] : l[1]) + __shfl_xor_sync(0xffffffffu, up ? l[1] : l[3], 16);
        float s = (up2 ? s1 : s0) + __shfl_xor_sync(0xffffffffu, up2 ? s0 : s1, 8);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
        if (lane % 8 == 0) xl[((up ? 2 : 0) + (up2 ? 1 : 0)) * 4 + qw] = s;
      }
      // (d = 64: lanes 64 to 127 hold the second token's part; P's rows are free)
      float* half = reinterpret_cast<float*>(prow) + wg * 256;
      if (TPR == 2 && kl >= 64) {
#pragma unroll
        for (int r = 0; r < 4; ++r) half[r * 64 + kl - 64] = acc[r];
      }
      if (!named_bar_and(all_bar, 128 * WG, ok)) break;
      const bool whole = t1 - t0 == info.w;
      const int2* rows = reinterpret_cast<const int2*>(sbase + L::kRow) + (seg & 1) * RP + wg * 4;
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const int2 at = rows[r];
        const float4 l4 = *reinterpret_cast<const float4*>(xl + r * 4);
        const float lt = (l4.x + l4.y) + (l4.z + l4.w);
        const float sum = TPR == 2 && kl < 64 ? acc[r] + half[r * 64 + kl] : acc[r];
        if (at.x < 0) continue;
        if constexpr (CL) {  // joined below
          part_o[(wg * 4 + r) * 128 + kl] = sum;
          if (kl == 0) part_ml[wg * 4 + r] = make_float2(m[r], lt);
          continue;
        }
        if (whole) {
          const float v = lt != 0.f ? __fdividef(sum, lt) : 0.f;
          if (kl < D) reinterpret_cast<uint16_t*>(p.o)[(size_t)at.x * D + kl] = (uint16_t)pack2<BF16>(v, 0.f);
          if (kl == 0) p.lse[at.y] = lt != 0.f ? (m[r] + __log2f(lt)) * kLn2 : -INFINITY;
        } else {
          const size_t part = ((size_t)blockIdx.x * 2 + (seg > 0 ? 1 : 0)) * RP + wg * 4 + r;
          if (kl < D) p.ws_o[part * D + kl] = sum;
          if (kl == 0) {
            p.ws_ml[part * 2] = m[r];
            p.ws_ml[part * 2 + 1] = lt;
          }
        }
      }
      // (the next segment's P and row sums are written behind the barrier at its start)
    }
  }
  if constexpr (CL) {
    if (mine.nt == 0) {  // a request without tokens
      if (rank == 0 && warp < 4 * WG) {
        const int h = mine.hr / p.n_rb, rb = mine.hr % p.n_rb;
        for (int r = warp; r < RP; r += 4 * WG) {
          const int idx = rb * RP + r, i = idx / p.G, hq = h * p.G + idx % p.G;
          if (idx >= p.Nq * p.G) break;
          const size_t at = ((size_t)mine.b * p.Nq + i) * p.Hq + hq;
          for (int c = lane; c < D; c += 32) reinterpret_cast<uint16_t*>(p.o)[at * D + c] = 0;
          if (lane == 0) p.lse[((size_t)mine.b * p.Hq + hq) * p.Nq + i] = -INFINITY;
        }
      }
    } else {
      // The parts of the CTAs that had tiles; those deal the rows among them, in the order of rows.
      cluster_sync();
      const int per = (mine.nt + p.cluster - 1) / p.cluster, n = (mine.nt + per - 1) / per;
      if (rank < n && warp < 4 * WG) {
        const int c = threadIdx.x & 127;
        const int2* rows = reinterpret_cast<const int2*>(sbase + L::kRow);
        for (int r = rank + n * (warp >> 2); r < RP; r += n * WG) {
          const int2 at = rows[r];
          if (at.x < 0) break;
          float mr[kKv4MaxCluster], lr[kKv4MaxCluster], o[kKv4MaxCluster], M = kNone;
#pragma unroll
          for (int k = 0; k < kKv4MaxCluster; ++k) {
            mr[k] = kNone;
            lr[k] = o[k] = 0.f;
            if (k < n) {
              const float2 ml = ld_cluster_f2(base + L::kK + RP * 512 + r * 8, k);
              mr[k] = ml.x;
              lr[k] = ml.y;
              o[k] = ld_cluster_f(base + L::kK + (r * 128 + c) * 4, k);
            }
          }
#pragma unroll
          for (int k = 0; k < kKv4MaxCluster; ++k) M = fmaxf(M, mr[k]);
          float l = 0.f, sum = 0.f;
#pragma unroll
          for (int k = 0; k < kKv4MaxCluster; ++k) {
            const float w = ex2(mr[k] - M);
            l = fmaf(w, lr[k], l);
            sum = fmaf(w, o[k], sum);
          }
          if (c < D) reinterpret_cast<uint16_t*>(p.o)[(size_t)at.x * D + c] = (uint16_t)pack2<BF16>(l != 0.f ? __fdividef(sum, l) : 0.f, 0.f);
          if (c == 0) p.lse[at.y] = l != 0.f ? (M + __log2f(l)) * kLn2 : -INFINITY;
        }
      }
      cluster_sync();  // (before any of them leaves)
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, L::kCols);
  }
}

// Launches the kernel for `a`, or, with `fit`, asks how many of its clusters the GPU can hold at once.
template <int D, int WG, int NP>
cudaError_t split_t(const KvDecArgs& a, cudaStream_t stream, int* fit) {
  using L = Kv4Layout<D, WG, NP>;
  auto* k = a.cluster ? attn_kv4_split_kernel<D, WG, NP, true> : attn_kv4_split_kernel<D, WG, NP, false>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, L::kSmem);
  if (e == cudaSuccess && a.cluster > 8) e = cudaFuncSetAttribute(k, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.grid);
  cfg.blockDim = dim3(L::kThreads);
  cfg.dynamicSmemBytes = L::kSmem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)a.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cudaLaunchAttribute& pdl = attr[a.cluster ? 1 : 0];
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (fit) return cudaOccupancyMaxActiveClusters(fit, k, &cfg);
  pdl.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  pdl.val.programmaticStreamSerializationAllowed = 1;
  cfg.numAttrs = a.cluster ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, a);
}

template <int D>
cudaError_t split_d(const KvDecArgs& a, cudaStream_t stream, int* fit) {
  if (a.bf16)
    return a.rp == 4 ? split_t<D, 1, 2>(a, stream, fit)
                     : (a.rp == 8 ? split_t<D, 2, 2>(a, stream, fit) : split_t<D, 4, 2>(a, stream, fit));
  return a.rp == 4 ? split_t<D, 1, 3>(a, stream, fit) : split_t<D, 2, 3>(a, stream, fit);
}

}  // namespace

template <int D, bool BF16>
static cudaError_t launch_append_t(const Kv4AppendArgs& a, bool w32, bool ahead, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.T + a.tok - 1) / a.tok), 2);
  cfg.blockDim = dim3(kAppThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  if (ahead)
    return w32 ? cudaLaunchKernelEx(&cfg, attn_kv4_append_kernel<D, BF16, true, true>, a)
               : cudaLaunchKernelEx(&cfg, attn_kv4_append_kernel<D, BF16, false, true>, a);
  return w32 ? cudaLaunchKernelEx(&cfg, attn_kv4_append_kernel<D, BF16, true, false>, a)
             : cudaLaunchKernelEx(&cfg, attn_kv4_append_kernel<D, BF16, false, false>, a);
}

cudaError_t launch_kv4_append(Kv4AppendArgs a, int sms, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  // An item a thread, or all of a token's; where there are many blocks four, the next one read ahead
  // (256k tokens of 8 heads, d = 128: 264 us, 293 with one; 31749 of 4 heads, d = 64: 7.1, 7.5 with four;
  // a step of 256: 1.7 and 3.4).
  const long long per_tok = (long long)a.H * (a.d / 16);
  const bool ahead = a.T * per_tok * 2 / kAppThreads > 64ll * sms;
  kv_rows(&a, (ahead ? 4 : 1) * (long long)kAppThreads / per_tok);
  const bool w32 = !((reinterpret_cast<uintptr_t>(a.x[0]) | reinterpret_cast<uintptr_t>(a.x[1])) & 31u) &&
                   a.x_stride[0] % 16 == 0 && a.x_stride[1] % 16 == 0;
  if (a.d == 128) return a.bf16 ? launch_append_t<128, true>(a, w32, ahead, stream) : launch_append_t<128, false>(a, w32, ahead, stream);
  return a.bf16 ? launch_append_t<64, true>(a, w32, ahead, stream) : launch_append_t<64, false>(a, w32, ahead, stream);
}

cudaError_t launch_kv4_split(const KvDecArgs& a, cudaStream_t stream) {
  return a.d == 128 ? split_d<128>(a, stream, nullptr) : split_d<64>(a, stream, nullptr);
}

bool kv4_clusters_fit(const KvDecArgs& a) {
  int n = 0;
  if ((a.d == 128 ? split_d<128>(a, nullptr, &n) : split_d<64>(a, nullptr, &n)) == cudaSuccess) return n > 0;
  cudaGetLastError();  // (an answer, not a fault of the call)
  return false;
}

}  // namespace attn
