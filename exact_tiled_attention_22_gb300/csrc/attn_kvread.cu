// attn_kvread.cu -- cached keys and values back as packed 16-bit rows, for sm_103a:
// what a prompt attends to that goes on after a prefix in the paged cache.
//
// Row cu[b] + i of the outputs is token i of request b.  A block takes some rows of K
// or of V: it looks up each row's request and page once, then every thread turns 8 codes
// into 16 bytes at a time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "kernels.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kReadThreads = 256;
constexpr int kReadMaxTok = 128;

// BITS = 8: e4m3 codes, a scale for each page and head.  BITS = 4: e2m1 codes, a scale
// for 32 channels of a token and head.
template <int D, int BITS, bool BF16>
__global__ void __launch_bounds__(kReadThreads) attn_kv_read_kernel(const __grid_constant__ KvReadArgs p) {
  __shared__ long long src[kReadMaxTok];  // (page, 0, place) of the row; -1: not written, -2: zeros
  griddep_wait();
  constexpr int kParts = D / 8, U = 4;
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
    uint2 c[U];
    float s[U];
    bool put[U];
    long long dst[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * kReadThreads;
      const int row = i / kParts, part = i % kParts;
      const int tl = (int)__umulhi((uint32_t)row * 2, p.h_magic), h = row - tl * p.H;
      put[u] = false;
      c[u] = make_uint2(0, 0);
      s[u] = 0.f;
      if (i < items) {
        const long long at = src[tl];
        put[u] = at != -1;
        dst[u] = (t0 + tl) * p.H * kParts + (long long)h * kParts + part;
        if (at >= 0) {
          const long long a = at + ((long long)h << p.page_shift);  // (page, head, place)
          if constexpr (BITS == 8) {
            c[u] = *reinterpret_cast<const uint2*>(codes + a * D + part * 8);
            s[u] = static_cast<const float*>(p.scale[kv])[a >> p.page_shift];
          } else {
            c[u].x = *reinterpret_cast<const uint32_t*>(codes + (a * kParts + part) * 4);
            s[u] = __uint_as_float((uint32_t) static_cast<const uint16_t*>(p.scale[kv])[(a * kParts + part) >> 2] << 16);
          }
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!put[u]) continue;
      float2 f[4];
      if constexpr (BITS == 8) {
        f[0] = unpack_e4m3(c[u].x & 0xffffu);
        f[1] = unpack_e4m3(c[u].x >> 16);
        f[2] = unpack_e4m3(c[u].y & 0xffffu);
        f[3] = unpack_e4m3(c[u].y >> 16);
      } else {
        uint32_t hw[4];
        unpack_e2m1(c[u].x, hw);
#pragma unroll
        for (int j = 0; j < 4; ++j) f[j] = unpack2<false>(hw[j]);
      }
      uint32_t w[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = pack2_sat<BF16>(f[j].x * s[u], f[j].y * s[u]);
      static_cast<uint4*>(p.out[kv])[dst[u]] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
  if (threadIdx.x == 0) griddep_launch_dependents();
}

template <int D, int BITS>
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
  return a.bf16 ? cudaLaunchKernelEx(&cfg, attn_kv_read_kernel<D, BITS, true>, a)
                : cudaLaunchKernelEx(&cfg, attn_kv_read_kernel<D, BITS, false>, a);
}

}  // namespace

cudaError_t launch_kv_read(KvReadArgs a, int sms, cudaStream_t stream) {
  if (a.T == 0) return cudaSuccess;
  const long long per_tok = (long long)a.H * (a.d / 8);
  long long tok = 4ll * kReadThreads / per_tok;
  if (tok > kReadMaxTok) tok = kReadMaxTok;
  kv_rows(&a, tok);
  if (a.d == 128) return a.bits == 8 ? launch_read_d<128, 8>(a, stream) : launch_read_d<128, 4>(a, stream);
  return a.bits == 8 ? launch_read_d<64, 8>(a, stream) : launch_read_d<64, 4>(a, stream);
}

}  // namespace attn
