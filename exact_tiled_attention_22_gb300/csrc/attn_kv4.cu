// attn_kv4.cu -- a paged key/value cache held in 4 bits, for sm_103a.
//
// A cached value is s * c: c an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
// negatives), s a bf16 scale shared by 32 consecutive channels of one token
// and head.  4.5 bits a value; a token is rounded by itself, so nothing that is
// in the cache is ever rounded again.
//
// attn_kv4_append_kernel   rounds new keys and values into their slots.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "kv_split.cuh"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

// ------------------------------------------------------------------ append
constexpr int kAppThreads = 256;

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

}  // namespace attn
