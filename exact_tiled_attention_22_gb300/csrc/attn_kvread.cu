// attn_kvread.cu -- cached keys and values back as packed 16-bit rows, for sm_103a:
// what a prompt attends to that goes on after a prefix in the paged cache.
//
// Bound by memory: 94k tokens of 8 heads, d = 128, from 4 bits (386 MB, four fifths of it written) 64 us or
// 6.0 TB/s; 48k from 8 bits (294 MB) 46 us or 6.3 TB/s; 24 prefixes, 7 and 11 MB, 3.5 and 3.9 us.
// What it took: 32 bytes a thread and store instead of 16 (103 -> 75 us), rows of four chunks to a block (-> 64).
//
// Row cu[b] + i of the outputs is token i of request b.  A block takes some rows of K
// or of V: it looks up each row's request and page once, then every thread turns 16 codes
// into 32 bytes at a time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kReadThreads = 256;
constexpr int kReadMaxTok = 128;

// A product in 32 bits, cut off towards zero, with its last bit set where that lost something: rounding it to 16 bits
// rounds the product itself, ties included.  (Infinities and NaN leave no rest that is a number.)  48k tokens with scales
// of 24 bits: 47.6 us, 46.3 with powers of two.
__device__ __forceinline__ float mul_to_odd(float a, float b) {
  const float r = __fmul_rz(a, b);
  return fabsf(fmaf(a, b, -r)) > 0.f ? __uint_as_float(__float_as_uint(r) | 1u) : r;
}

// BITS = 8: e4m3 codes, a scale for each page and head.  BITS = 4: e2m1 codes, a scale
// for 32 channels of a token and head.
template <int D, int BITS, bool BF16, int U>
__global__ void __launch_bounds__(kReadThreads) attn_kv_read_kernel(const __grid_constant__ KvReadArgs p) {
  __shared__ long long src[kReadMaxTok];  // (page, 0, place) of the row; -1: not written, -2: zeros
  griddep_wait();
  constexpr int kParts = D / 16;  // threads to a token and head
  const int kv = blockIdx.y, ps = 1 << p.page_shift;
  const long long t0 = (long long)blockIdx.x * p.tok;
  const int n_tok = (int)min((long long)p.tok, p.T - t0);
  if (threadIdx.x < n_tok) {
    const long long t = t0 + threadIdx.x;
    // the last request whose rows begin at t or before
    int lo = 0, hi = p.B;  // cu[lo] <= t < cu[hi], if at all
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (p.cu[mid] <= t) lo = mid;
      else hi = mid;
    }
    const long long i = t - p.cu[lo];
    const long long len = min((long long)p.lens[lo], (long long)p.width << p.page_shift);
    long long s = -1;
    if (i >= 0 && i < len && t < p.cu[lo + 1]) {
      const int page = p.table[(size_t)lo * p.width + (i >> p.page_shift)];
      s = page >= 0 && page < p.P ? (((long long)page * p.H) << p.page_shift) + (i & (ps - 1)) : -2;
    }
    src[threadIdx.x] = s;
  }
  __syncthreads();
  const int items = n_tok * p.H * kParts;
  const uint8_t* codes = p.cache[kv];
  for (int i0 = threadIdx.x; i0 < items; i0 += kReadThreads * U) {
    uint4 c[U];
    float s[U];
    long long dst[U];  // -1: not written
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kReadThreads;
      const int row = i / kParts, part = i % kParts;
      const int tl = (int)__umulhi((uint32_t)row * 2, p.h_magic), h = row - tl * p.H;
      c[u] = make_uint4(0, 0, 0, 0);
      s[u] = 0.f;
      dst[u] = -1;
      if (i < items) {
        const long long at = src[tl];
        if (at != -1) dst[u] = ((t0 + tl) * p.H + h) * kParts + part;
        if (at >= 0) {
          const long long a = at + ((long long)h << p.page_shift);  // (page, head, place)
          if constexpr (BITS == 8) {
            c[u] = *reinterpret_cast<const uint4*>(codes + (a * kParts + part) * 16);
            s[u] = static_cast<const float*>(p.scale[kv])[a >> p.page_shift];
          } else {
            const uint2 two = *reinterpret_cast<const uint2*>(codes + (a * kParts + part) * 8);
            c[u].x = two.x;
            c[u].y = two.y;
            s[u] = __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.scale[kv])[(a * kParts + part) >> 1] << 16);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (dst[u] < 0) continue;
      uint32_t w[8];
      const uint32_t* cw = &c[u].x;
#pragma unroll
      for (int j = 0; j < 8; j += 4) {  // eight channels
        float2 f[4];
        if constexpr (BITS == 8) {
#pragma unroll
          for (int k = 0; k < 4; ++k) f[k] = unpack_e4m3(cw[j / 2 + k / 2] >> (16 * (k & 1)));
        } else {
          uint32_t hw[4];
          unpack_e2m1(cw[j / 4], hw);
#pragma unroll
          for (int k = 0; k < 4; ++k) f[k] = unpack2<false>(hw[k]);
        }
        // (e2m1 times bf16 has 11 bits, e4m3 times a scale of 20 has 24: exact, as with append's powers of two)
        if (BITS == 8 && (__float_as_uint(s[u]) & 15u)) {
#pragma unroll
          for (int k = 0; k < 4; ++k) w[j + k] = pack2_sat<BF16>(mul_to_odd(f[k].x, s[u]), mul_to_odd(f[k].y, s[u]));
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) w[j + k] = pack2_sat<BF16>(f[k].x * s[u], f[k].y * s[u]);
        }
      }
      st_global_32(static_cast<uint8_t*>(p.out[kv]) + dst[u] * 32, w);
    }
  }
  if (threadIdx.x == 0) griddep_launch_dependents();
}

template <int D, int BITS, int U>
cudaError_t launch_read_d(const KvReadArgs& a, cudaStream_t stream) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)((a.T + a.tok - 1) / a.tok), 2);
  cfg.blockDim = dim3(kReadThreads);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return a.bf16 ? cudaLaunchKernelEx(&cfg, attn_kv_read_kernel<D, BITS, true, U>, a)
                : cudaLaunchKernelEx(&cfg, attn_kv_read_kernel<D, BITS, false, U>, a);
}

}  // namespace

// Two chunks of 16 channels a thread in flight for 8-bit codes, one for 4-bit ones, and R times
// that many a block where there are blocks enough: the rows of a block are looked up once.
// (94k tokens of 8 heads, d = 128, in 4 bits: 75, 68, 65 us with R = 1, 2, 4, 67 with two
// chunks; 48k tokens in 8 bits 47.6, 46.5, 47.5, 48 with one.  24 prefixes, 11k tokens of 4 heads,
// d = 64: 3.5 and 3.8 us with R = 1, 4.2 and 4.6 with 4.)
template <int BITS>
static cudaError_t launch_read_bits(KvReadArgs a, int sms, cudaStream_t stream) {
  constexpr int U = BITS == 8 ? 2 : 1, R = BITS == 8 ? 2 : 4;
  const long long per_tok = (long long)a.H * (a.d / 16), blocks = a.T * per_tok * 2 / (U * kReadThreads);
  const long long runs = blocks / (16ll * sms), tok = (runs < 1 ? 1 : (runs < R ? runs : R)) * U * kReadThreads / per_tok;
  kv_rows(&a, tok < kReadMaxTok ? tok : kReadMaxTok);
  return a.d == 128 ? launch_read_d<128, BITS, U>(a, stream) : launch_read_d<64, BITS, U>(a, stream);
}

cudaError_t launch_kv_read(const KvReadArgs& a, int sms, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  return a.bits == 8 ? launch_read_bits<8>(a, sms, stream) : launch_read_bits<4>(a, sms, stream);
}

}  // namespace attn
