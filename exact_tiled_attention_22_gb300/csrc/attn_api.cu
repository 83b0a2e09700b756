// attn_api.cu -- the C ABI (include/attn.h): argument checks, TMA tensor-map
// encoding, launch geometry, the device status word and per-kernel timing.
// The kernels themselves live in attn_fwd.cu and attn_bwd.cu.
#include <cuda.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <cstdarg>
#include <cstdint>
#include <cstdio>
#include <cstring>
#include <mutex>
#include <string>
#include <vector>

#include "attn.h"
#include "kernels.h"

namespace {

// Per-device status word read by attn_status(); kernels set it when a bounded
// wait runs out.  One copy per device (module globals are per context).
__device__ int g_attn_status;

constexpr int kMaxDevices = 64;
constexpr unsigned long long kDefaultWaitNs = 2000000000ull;  // 2 s

thread_local std::string t_err;

int fail(int code, const char* fmt, ...) __attribute__((format(printf, 2, 3)));
int fail(int code, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  t_err = buf;
  return code;
}

int cuda_fail(cudaError_t e, const char* what) {
  return fail(ATTN_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
}

struct DeviceInfo {
  bool ready = false;
  bool supported = false;
  int sms = 0;
  int* status = nullptr;            // device address of g_attn_status ...
  unsigned long long status_ctx = 0;  // ... in the context with this id
  // In that context, of each form of the 4-bit decode two bits: whether a cluster of 16 was asked for, and fits.
  std::atomic<unsigned> kv4_fit{0};
};

std::mutex g_mu;
DeviceInfo g_dev[kMaxDevices];
unsigned long long g_wait_ns = kDefaultWaitNs;
int g_debug_flags = 0;

using EncodeTiledFn = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*,
                                   const cuuint64_t*, const cuuint64_t*, const cuuint32_t*,
                                   const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                   CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiledFn g_encode = nullptr;

using CtxGetCurrentFn = CUresult (*)(CUcontext*);
using CtxGetIdFn = CUresult (*)(CUcontext, unsigned long long*);
CtxGetCurrentFn g_ctx_current = nullptr;
CtxGetIdFn g_ctx_id = nullptr;
std::once_flag g_ctx_once;

// Looks up the current device: architecture and SM count once per device,
// the status word's address once per context.
int current_device(DeviceInfo** out) {
  int dev = -1;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return cuda_fail(e, "cudaGetDevice");
  if (dev < 0 || dev >= kMaxDevices) return fail(ATTN_ERR_UNSUPPORTED, "device %d out of range", dev);
  // Binds the device's primary context to this thread: the tensor-map
  // encoding is a driver call, and a thread that has made no runtime call
  // yet (e.g. a framework's backward worker) has no current context.
  if ((e = cudaSetDevice(dev)) != cudaSuccess) return cuda_fail(e, "cudaSetDevice");
  std::lock_guard<std::mutex> lk(g_mu);
  DeviceInfo& d = g_dev[dev];
  if (!d.ready) {
    int major = 0, minor = 0, sms = 0;
    if ((e = cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev)) != cudaSuccess ||
        (e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess)
      return cuda_fail(e, "cudaDeviceGetAttribute");
    d.supported = (major == 10 && minor == 3);
    d.sms = sms;
    if (!g_encode) {
      void* fn = nullptr;
      cudaDriverEntryPointQueryResult q;
      e = cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &fn, 12000, cudaEnableDefault, &q);
      if (e != cudaSuccess || q != cudaDriverEntryPointSuccess || !fn)
        return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled entry point not found");
      g_encode = reinterpret_cast<EncodeTiledFn>(fn);
    }
    d.ready = true;
  }
  if (!d.supported)
    return fail(ATTN_ERR_UNSUPPORTED, "device %d is not sm_103 (GB300); no other path exists", dev);
  // The status word's address belongs to the context the module was loaded
  // in: look it up again whenever the thread's current context is another
  // one (a context torn down by cudaDeviceReset and created anew included;
  // context ids are never reused within a process).
  unsigned long long ctx = 0;
  if (attn::current_context_id(&ctx) != cudaSuccess)
    return fail(ATTN_ERR_CUDA, "cannot identify the current CUDA context");
  if (!d.status || d.status_ctx != ctx) {
    void* ptr = nullptr;
    if ((e = cudaGetSymbolAddress(&ptr, g_attn_status)) != cudaSuccess)
      return cuda_fail(e, "cudaGetSymbolAddress(status)");
    d.status = static_cast<int*>(ptr);
    d.status_ctx = ctx;
    d.kv4_fit = 0;
  }
  *out = &d;
  return ATTN_OK;
}

// A [B, N, H, d] 16-bit tensor as a 4-D TMA map (d, H, N, B), 128-byte
// swizzle, boxes of 64 columns x `rows` sequence rows of one (b, h).
int encode_bnhd(CUtensorMap* m, const void* ptr, int B, int N, int H, int d, int rows, bool bf16) {
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)N, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)H * d * 2, (cuuint64_t)N * H * d * 2};
  const cuuint32_t box[4] = {64, 1, (cuuint32_t)rows, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = g_encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                        const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return ATTN_OK;
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

struct Range {
  uintptr_t lo, hi;
};
bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
Range rng(const void* p, size_t bytes) {
  uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return {a, a + bytes};
}

// Bytes of a block mask [H][nb][nb], nb = ceil(N / 128).
size_t mask_bytes(int H, int N) {
  const size_t nb = ((size_t)N + 127) / 128;
  return (size_t)H * nb * nb;
}

// The block-sparse variants keep one 128-row block list per CTA in shared
// memory: N / 128 is bounded.
int check_block_mask(int N) {
  if ((N + 127) / 128 > attn::kMaxSparseTiles)
    return fail(ATTN_ERR_INVALID, "block_mask supports N <= %d, got %d", attn::kMaxSparseTiles * 128, N);
  return ATTN_OK;
}

// Dropout probability -> keep threshold and the kernels' constants (t = 256:
// no dropout).  p must lie in [0, 1) and keep a threshold of at least 1.
int make_dropout(float dropout_p, uint64_t seed, uint32_t offset, attn::DropoutArgs* out) {
  const double p = (double)dropout_p;
  if (!(p >= 0.0 && p < 1.0))
    return fail(ATTN_ERR_INVALID, "dropout_p must be in [0, 1), got %g", p);
  const int t = (int)std::floor(256.0 * (1.0 - p) + 0.5);
  if (t < 1) return fail(ATTN_ERR_INVALID, "dropout_p %g keeps no score (256 (1 - p) < 1/2)", p);
  out->k0 = (uint32_t)(seed & 0xFFFFFFFFull);
  out->k1 = (uint32_t)(seed >> 32);
  out->offset = offset;
  out->t = t;
  out->cmp = (uint32_t)(256 - t) * 0x00010001u;
  out->scale = 256.0f / (float)t;
  for (int r = 0; r < 10; ++r) {
    out->rk[2 * r] = out->k0 + (uint32_t)r * attn::kPhiloxW0;
    out->rk[2 * r + 1] = out->k1 + (uint32_t)r * attn::kPhiloxW1;
  }
  return ATTN_OK;
}

int check_common(int B, int H, int N, int d, float scale, attn_dtype_t dtype) {
  if (B < 1 || H < 1 || N < 1) return fail(ATTN_ERR_INVALID, "B, H, N must be >= 1 (got %d, %d, %d)", B, H, N);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim d=%d not supported (64 or 128)", d);
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return fail(ATTN_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  // Kernels index tensors with 64-bit offsets; what must fit in 31 bits is
  // B*H and the grids (at most ceil(N/128) blocks per head, 64 per head
  // when decoding).
  const long long bh = (long long)B * H;
  if (bh * (((long long)N + 127) / 128) >= (1ll << 31) || bh * 64 >= (1ll << 31))
    return fail(ATTN_ERR_INVALID, "B*H*ceil(N/128) = %lld blocks too many (< 2^31, and B*H < 2^25)",
                bh * (((long long)N + 127) / 128));
  const long long elems = bh * N * d;
  if (elems >= (1ll << 40)) return fail(ATTN_ERR_INVALID, "B*H*N*d = %lld too large (< 2^40)", elems);
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(ATTN_ERR_INVALID, "scale must be finite and > 0");
  return ATTN_OK;
}

// ---------------------------------------------------------------- profiling
struct ProfState {
  bool on = false;
  std::vector<cudaEvent_t> pool;
  size_t used = 0;
  std::vector<int> kind;  // one per event pair
};
ProfState g_prof;
std::mutex g_prof_mu;
constexpr size_t kProfPairs = 8192;

// Runs `launch` bracketed by events when profiling is on.
template <typename F>
cudaError_t timed(int kind, cudaStream_t stream, F&& launch) {
  cudaEvent_t e0 = nullptr, e1 = nullptr;
  {
    std::lock_guard<std::mutex> lk(g_prof_mu);
    if (g_prof.on && g_prof.used + 2 <= g_prof.pool.size()) {
      e0 = g_prof.pool[g_prof.used];
      e1 = g_prof.pool[g_prof.used + 1];
      g_prof.used += 2;
      g_prof.kind.push_back(kind);
    }
  }
  if (e0) cudaEventRecord(e0, stream);
  cudaError_t e = launch();
  if (e1) cudaEventRecord(e1, stream);
  return e;
}

}  // namespace

namespace attn {
cudaError_t current_context_id(unsigned long long* id) {
  std::call_once(g_ctx_once, [] {
    void* fn = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &fn, 12000, cudaEnableDefault, &q) ==
            cudaSuccess && q == cudaDriverEntryPointSuccess)
      g_ctx_current = reinterpret_cast<CtxGetCurrentFn>(fn);
    fn = nullptr;
    if (cudaGetDriverEntryPointByVersion("cuCtxGetId", &fn, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      g_ctx_id = reinterpret_cast<CtxGetIdFn>(fn);
  });
  if (!g_ctx_current || !g_ctx_id) return cudaErrorNotSupported;
  CUcontext c = nullptr;
  if (g_ctx_current(&c) != CUDA_SUCCESS || !c) return cudaErrorDeviceUninitialized;
  return g_ctx_id(c, id) == CUDA_SUCCESS ? cudaSuccess : cudaErrorDeviceUninitialized;
}

void set_last_error(const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof buf, fmt, ap);
  va_end(ap);
  t_err = buf;
}
}  // namespace attn

extern "C" {

const char* attn_last_error_string(void) { return t_err.c_str(); }

int attn_set_wait_limit(unsigned long long limit_ns, int debug_flags) {
  std::lock_guard<std::mutex> lk(g_mu);
  g_wait_ns = limit_ns ? limit_ns : kDefaultWaitNs;
  g_debug_flags = debug_flags;
  return ATTN_OK;
}

int attn_fwd_ex(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N,
                int d, float scale, int causal, const float* alibi_slopes, const uint8_t* block_mask,
                float dropout_p, uint64_t seed, uint32_t offset, attn_dtype_t dtype, void* stream) {
  t_err.clear();
  if (!q || !k || !v || !o || !lse) return fail(ATTN_ERR_INVALID, "null pointer argument");
  if (alibi_slopes && !aligned4(alibi_slopes)) return fail(ATTN_ERR_ALIGN, "alibi_slopes must be 4-byte aligned");
  int rc = check_common(B, H, N, d, scale, dtype);
  if (rc) return rc;
  if (block_mask && (rc = check_block_mask(N))) return rc;
  attn::DropoutArgs drop;
  if ((rc = make_dropout(dropout_p, seed, offset, &drop))) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(ATTN_ERR_ALIGN, "all pointers must be 16-byte aligned");
  const size_t tb = (size_t)B * N * H * d * 2, lb = (size_t)B * H * N * 4;
  const Range outs[2] = {rng(o, tb), rng(lse, lb)};
  const Range ins[5] = {rng(q, tb), rng(k, tb), rng(v, tb), rng(alibi_slopes, alibi_slopes ? (size_t)H * 4 : 0),
                        rng(block_mask, block_mask ? mask_bytes(H, N) : 0)};
  if (overlap(outs[0], outs[1])) return fail(ATTN_ERR_INVALID, "o and lse overlap");
  for (const Range& a : outs)
    for (const Range& b : ins)
      if (overlap(a, b)) return fail(ATTN_ERR_INVALID, "an output overlaps an input");

  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  attn::FwdArgs a;
  std::memset(&a, 0, sizeof a);
  const bool bf16 = dtype == ATTN_BF16;
  if ((rc = encode_bnhd(&a.tm_q, q, B, N, H, d, 128, bf16)) ||
      (rc = encode_bnhd(&a.tm_k, k, B, N, H, d, 128, bf16)) ||
      (rc = encode_bnhd(&a.tm_v, v, B, N, H, d, 128, bf16)) ||
      (rc = encode_bnhd(&a.tm_o, o, B, N, H, d, 128, bf16)))
    return rc;
  a.o = o;
  a.lse = lse;
  a.alibi = alibi_slopes;
  a.bmask = block_mask;
  a.drop = drop;
  a.B = B; a.H = H; a.N = N; a.d = d;
  a.causal = causal ? 1 : 0;
  a.scale = scale;
  a.bf16 = bf16;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    a.debug_flags = g_debug_flags;
    a.wait.limit_ns = g_wait_ns;
  }
  a.wait.status = dev->status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed(attn::kKFwd, s, [&] { return attn::launch_fwd(a, s); });
  if (e != cudaSuccess) return cuda_fail(e, "attn_fwd launch");
  return ATTN_OK;
}

int attn_fwd_sparse(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N,
                    int d, float scale, int causal, const float* alibi_slopes, const uint8_t* block_mask,
                    attn_dtype_t dtype, void* stream) {
  return attn_fwd_ex(q, k, v, o, lse, B, H, N, d, scale, causal, alibi_slopes, block_mask, 0.f, 0, 0, dtype,
                     stream);
}

int attn_fwd_alibi(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N,
                   int d, float scale, int causal, const float* alibi_slopes, attn_dtype_t dtype,
                   void* stream) {
  return attn_fwd_ex(q, k, v, o, lse, B, H, N, d, scale, causal, alibi_slopes, nullptr, 0.f, 0, 0, dtype,
                     stream);
}

int attn_fwd(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int N, int d,
             float scale, int causal, attn_dtype_t dtype, void* stream) {
  return attn_fwd_ex(q, k, v, o, lse, B, H, N, d, scale, causal, nullptr, nullptr, 0.f, 0, 0, dtype, stream);
}

size_t attn_decode_workspace_size(int B, int H, int Nq, int Nk, int d) {
  if (B < 1 || H < 1 || Nq < 1 || Nk < 1 || (d != 64 && d != 128)) return 0;
  const size_t parts = (size_t)B * H * attn::decode_n_split(B, H, Nk) * Nq;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  return up(parts * d * 4) + up(parts * 2 * 4);
}

int attn_decode_alibi(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H,
                      int Nq, int Nk, int d, float scale, int causal, const float* alibi_slopes,
                      attn_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  t_err.clear();
  if (!q || !k || !v || !o || !lse) return fail(ATTN_ERR_INVALID, "null pointer argument");
  if (alibi_slopes && !aligned4(alibi_slopes)) return fail(ATTN_ERR_ALIGN, "alibi_slopes must be 4-byte aligned");
  if (Nq < 1 || Nk < 1) return fail(ATTN_ERR_INVALID, "Nq, Nk must be >= 1 (got %d, %d)", Nq, Nk);
  if (Nq > 128) return fail(ATTN_ERR_UNSUPPORTED, "decode takes at most 128 query rows (got %d)", Nq);
  if (causal && Nq > Nk) return fail(ATTN_ERR_INVALID, "causal decode needs Nq <= Nk (got %d > %d)", Nq, Nk);
  int rc = check_common(B, H, Nk, d, scale, dtype);
  if (rc) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(ATTN_ERR_ALIGN, "all pointers must be 16-byte aligned");
  const size_t need = attn_decode_workspace_size(B, H, Nq, Nk, d);
  if (!workspace || workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(ATTN_ERR_ALIGN, "workspace must be 256-byte aligned");
  const size_t qb = (size_t)B * Nq * H * d * 2, kb = (size_t)B * Nk * H * d * 2, lb = (size_t)B * H * Nq * 4;
  const Range outs[3] = {rng(o, qb), rng(lse, lb), rng(workspace, need)};
  const Range ins[4] = {rng(q, qb), rng(k, kb), rng(v, kb), rng(alibi_slopes, alibi_slopes ? (size_t)H * 4 : 0)};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (overlap(outs[i], outs[j])) return fail(ATTN_ERR_INVALID, "outputs or workspace overlap");
  for (const Range& a : outs)
    for (const Range& b : ins)
      if (overlap(a, b)) return fail(ATTN_ERR_INVALID, "an output overlaps an input");

  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  attn::DecArgs a;
  std::memset(&a, 0, sizeof a);
  const bool bf16 = dtype == ATTN_BF16;
  if ((rc = encode_bnhd(&a.tm_q, q, B, Nq, H, d, 128, bf16)) ||
      (rc = encode_bnhd(&a.tm_k, k, B, Nk, H, d, 128, bf16)) ||
      (rc = encode_bnhd(&a.tm_v, v, B, Nk, H, d, 128, bf16)))
    return rc;
  a.o = o;
  a.lse = lse;
  a.alibi = alibi_slopes;
  a.B = B; a.H = H; a.Nq = Nq; a.Nk = Nk; a.d = d;
  a.n_split = attn::decode_n_split(B, H, Nk);
  a.keys_per_split = attn::decode_keys_per_split(Nk, a.n_split);
  const size_t parts = (size_t)B * H * a.n_split * Nq;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.ws_o = reinterpret_cast<float*>(ws);
  a.ws_ml = reinterpret_cast<float*>(ws + (parts * d * 4 + 255) / 256 * 256);
  a.causal = causal ? 1 : 0;
  a.scale = scale;
  a.bf16 = bf16;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    a.debug_flags = g_debug_flags;
    a.wait.limit_ns = g_wait_ns;
  }
  a.wait.status = dev->status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed(attn::kKDecSplit, s, [&] { return attn::launch_decode_split(a, s); });
  if (e != cudaSuccess) return cuda_fail(e, "attn_decode chunk launch");
  e = timed(attn::kKDecMerge, s, [&] { return attn::launch_decode_merge(a, s); });
  if (e != cudaSuccess) return cuda_fail(e, "attn_decode merge launch");
  return ATTN_OK;
}

int attn_decode(const void* q, const void* k, const void* v, void* o, float* lse, int B, int H, int Nq,
                int Nk, int d, float scale, int causal, attn_dtype_t dtype, void* workspace,
                size_t workspace_bytes, void* stream) {
  return attn_decode_alibi(q, k, v, o, lse, B, H, Nq, Nk, d, scale, causal, nullptr, dtype, workspace,
                           workspace_bytes, stream);
}

size_t attn_bwd_workspace_size(int B, int H, int N, int d) {
  if (B < 1 || H < 1 || N < 1 || (d != 64 && d != 128)) return 0;
  const size_t npad = ((size_t)N + 127) / 128 * 128;
  const size_t rows = (size_t)B * H * npad;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  return up(rows * 4) * 2 + up(rows * d * 4) + 256;
}

int attn_bwd_ex(const void* q, const void* k, const void* v, const void* o, const float* lse,
                const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale,
                int causal, const float* alibi_slopes, const uint8_t* block_mask, float dropout_p,
                uint64_t seed, uint32_t offset, attn_dtype_t dtype, void* workspace,
                size_t workspace_bytes, void* stream) {
  t_err.clear();
  if (!q || !k || !v || !o || !lse || !dO || !dq || !dk || !dv)
    return fail(ATTN_ERR_INVALID, "null pointer argument");
  if (alibi_slopes && !aligned4(alibi_slopes)) return fail(ATTN_ERR_ALIGN, "alibi_slopes must be 4-byte aligned");
  int rc = check_common(B, H, N, d, scale, dtype);
  if (rc) return rc;
  if (block_mask && (rc = check_block_mask(N))) return rc;
  attn::DropoutArgs drop;
  if ((rc = make_dropout(dropout_p, seed, offset, &drop))) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) ||
      !aligned16(dO) || !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return fail(ATTN_ERR_ALIGN, "all pointers must be 16-byte aligned");
  const size_t need = attn_bwd_workspace_size(B, H, N, d);
  if (!workspace || workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(ATTN_ERR_ALIGN, "workspace must be 256-byte aligned");
  const size_t tb = (size_t)B * N * H * d * 2, lb = (size_t)B * H * N * 4;
  const Range outs[4] = {rng(dq, tb), rng(dk, tb), rng(dv, tb), rng(workspace, need)};
  const Range ins[8] = {rng(q, tb), rng(k, tb), rng(v, tb), rng(o, tb), rng(lse, lb), rng(dO, tb),
                        rng(alibi_slopes, alibi_slopes ? (size_t)H * 4 : 0),
                        rng(block_mask, block_mask ? mask_bytes(H, N) : 0)};
  for (int i = 0; i < 4; ++i) {
    for (int j = i + 1; j < 4; ++j)
      if (overlap(outs[i], outs[j])) return fail(ATTN_ERR_INVALID, "output buffers overlap");
    for (const Range& b : ins)
      if (overlap(outs[i], b)) return fail(ATTN_ERR_INVALID, "an output or the workspace overlaps an input");
  }

  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  attn::BwdArgs a;
  std::memset(&a, 0, sizeof a);
  const bool bf16 = dtype == ATTN_BF16;
  const int qrows = attn::bwd_q_rows(d);
  if ((rc = encode_bnhd(&a.tm_q, q, B, N, H, d, qrows, bf16)) ||
      (rc = encode_bnhd(&a.tm_k, k, B, N, H, d, 128, bf16)) ||
      (rc = encode_bnhd(&a.tm_v, v, B, N, H, d, 128, bf16)) ||
      (rc = encode_bnhd(&a.tm_do, dO, B, N, H, d, qrows, bf16)) ||
      (rc = encode_bnhd(&a.tm_dk, dk, B, N, H, d, 128, bf16)) ||
      (rc = encode_bnhd(&a.tm_dv, dv, B, N, H, d, 128, bf16)))
    return rc;
  const int npad = (N + 127) / 128 * 128;
  const size_t rows = (size_t)B * H * npad;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.o = o;
  a.dO = dO;
  a.lse = lse;
  a.alibi = alibi_slopes;
  a.bmask = block_mask;
  a.drop = drop;
  a.lse2 = reinterpret_cast<float*>(ws);
  a.dvec = reinterpret_cast<float*>(ws + up(rows * 4));
  a.dqacc = reinterpret_cast<float*>(ws + 2 * up(rows * 4));
  a.sched = reinterpret_cast<unsigned*>(ws + 2 * up(rows * 4) + up(rows * (size_t)d * 4));
  a.dq = dq; a.dk = dk; a.dv = dv;
  a.B = B; a.H = H; a.N = N; a.Npad = npad; a.d = d;
  a.sms = dev->sms;
  a.causal = causal ? 1 : 0;
  a.scale = scale;
  a.bf16 = bf16;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    a.debug_flags = g_debug_flags;
    a.wait.limit_ns = g_wait_ns;
  }
  a.wait.status = dev->status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed(attn::kKBwdPre, s, [&] { return attn::launch_bwd_pre(a, s); });
  if (e != cudaSuccess) return cuda_fail(e, "attn_bwd preprocess launch");
  e = timed(attn::kKBwdMain, s, [&] { return attn::launch_bwd_main(a, s); });
  if (e != cudaSuccess) return cuda_fail(e, "attn_bwd main launch");
  e = timed(attn::kKDqPost, s, [&] { return attn::launch_dq_post(a, s); });
  if (e != cudaSuccess) return cuda_fail(e, "attn_bwd dQ conversion launch");
  return ATTN_OK;
}

int attn_bwd_sparse(const void* q, const void* k, const void* v, const void* o, const float* lse,
                    const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale,
                    int causal, const float* alibi_slopes, const uint8_t* block_mask, attn_dtype_t dtype,
                    void* workspace, size_t workspace_bytes, void* stream) {
  return attn_bwd_ex(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, alibi_slopes, block_mask, 0.f,
                     0, 0, dtype, workspace, workspace_bytes, stream);
}

int attn_bwd_alibi(const void* q, const void* k, const void* v, const void* o, const float* lse,
                   const void* dO, void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale,
                   int causal, const float* alibi_slopes, attn_dtype_t dtype, void* workspace,
                   size_t workspace_bytes, void* stream) {
  return attn_bwd_ex(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, alibi_slopes, nullptr, 0.f,
                     0, 0, dtype, workspace, workspace_bytes, stream);
}

int attn_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
             void* dq, void* dk, void* dv, int B, int H, int N, int d, float scale, int causal,
             attn_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  return attn_bwd_ex(q, k, v, o, lse, dO, dq, dk, dv, B, H, N, d, scale, causal, nullptr, nullptr, 0.f, 0, 0,
                     dtype, workspace, workspace_bytes, stream);
}

int attn_fwd_acc(const void* q, const void* k, const void* v, float* o_acc, float* lse, void* o, int B, int H,
                 int N, int d, float scale, int causal, int flags, attn_dtype_t dtype, void* stream) {
  t_err.clear();
  if (flags < 0 || flags > (ATTN_ACC_FIRST | ATTN_ACC_LAST))
    return fail(ATTN_ERR_INVALID, "flags must be a combination of ATTN_ACC_FIRST and ATTN_ACC_LAST");
  const bool first = (flags & ATTN_ACC_FIRST) != 0, last = (flags & ATTN_ACC_LAST) != 0;
  if (!q || !k || !v || !lse) return fail(ATTN_ERR_INVALID, "null pointer argument");
  if (!(first && last) && !o_acc) return fail(ATTN_ERR_INVALID, "o_acc is needed unless flags has FIRST and LAST");
  if (last && !o) return fail(ATTN_ERR_INVALID, "o is needed with ATTN_ACC_LAST");
  int rc = check_common(B, H, N, d, scale, dtype);
  if (rc) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(lse) || !aligned16(o_acc) || !aligned16(o))
    return fail(ATTN_ERR_ALIGN, "all pointers must be 16-byte aligned");
  const size_t tb = (size_t)B * N * H * d * 2, lb = (size_t)B * H * N * 4;
  const Range outs[3] = {rng(o_acc, (first && last) ? 0 : 2 * tb), rng(lse, lb), rng(o, last ? tb : 0)};
  const Range ins[3] = {rng(q, tb), rng(k, tb), rng(v, tb)};
  for (int i = 0; i < 3; ++i) {
    for (int j = i + 1; j < 3; ++j)
      if (overlap(outs[i], outs[j])) return fail(ATTN_ERR_INVALID, "output buffers overlap");
    for (const Range& b : ins)
      if (overlap(outs[i], b)) return fail(ATTN_ERR_INVALID, "an output overlaps an input");
  }
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  attn::FwdArgs a;
  std::memset(&a, 0, sizeof a);
  const bool bf16 = dtype == ATTN_BF16;
  if ((rc = encode_bnhd(&a.tm_q, q, B, N, H, d, 128, bf16)) ||
      (rc = encode_bnhd(&a.tm_k, k, B, N, H, d, 128, bf16)) ||
      (rc = encode_bnhd(&a.tm_v, v, B, N, H, d, 128, bf16)))
    return rc;
  a.o = o;
  a.lse = lse;
  a.o_acc = o_acc;
  a.acc_flags = flags;
  if ((rc = make_dropout(0.f, 0, 0, &a.drop))) return rc;
  a.B = B; a.H = H; a.N = N; a.d = d;
  a.causal = causal ? 1 : 0;
  a.scale = scale;
  a.bf16 = bf16;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    a.debug_flags = g_debug_flags;
    a.wait.limit_ns = g_wait_ns;
  }
  a.wait.status = dev->status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed(attn::kKFwd, s, [&] { return attn::launch_fwd_acc(a, s); });
  if (e != cudaSuccess) return cuda_fail(e, "attn_fwd_acc launch");
  return ATTN_OK;
}

int attn_bwd_acc(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                 void* dq, float* dk_acc, float* dv_acc, int B, int H, int N, int d, float scale, int causal,
                 int dq_flags, int kv_flags, attn_dtype_t dtype, void* workspace, size_t workspace_bytes,
                 void* stream) {
  t_err.clear();
  const int all = ATTN_ACC_FIRST | ATTN_ACC_LAST;
  if (dq_flags < 0 || dq_flags > all || kv_flags < 0 || kv_flags > ATTN_ACC_FIRST)
    return fail(ATTN_ERR_INVALID, "dq_flags: FIRST and/or LAST; kv_flags: 0 or ATTN_ACC_FIRST");
  const bool dq_last = (dq_flags & ATTN_ACC_LAST) != 0;
  if (!q || !k || !v || !o || !lse || !dO || !dk_acc || !dv_acc || (dq_last && !dq))
    return fail(ATTN_ERR_INVALID, "null pointer argument");
  int rc = check_common(B, H, N, d, scale, dtype);
  if (rc) return rc;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) || !aligned16(dO) ||
      !aligned16(dq) || !aligned16(dk_acc) || !aligned16(dv_acc))
    return fail(ATTN_ERR_ALIGN, "all pointers must be 16-byte aligned");
  const size_t need = attn_bwd_workspace_size(B, H, N, d);
  if (!workspace || workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(ATTN_ERR_ALIGN, "workspace must be 256-byte aligned");
  const size_t tb = (size_t)B * N * H * d * 2, lb = (size_t)B * H * N * 4;
  const Range outs[4] = {rng(dq, dq_last ? tb : 0), rng(dk_acc, 2 * tb), rng(dv_acc, 2 * tb), rng(workspace, need)};
  const Range ins[6] = {rng(q, tb), rng(k, tb), rng(v, tb), rng(o, tb), rng(lse, lb), rng(dO, tb)};
  for (int i = 0; i < 4; ++i) {
    for (int j = i + 1; j < 4; ++j)
      if (overlap(outs[i], outs[j])) return fail(ATTN_ERR_INVALID, "output buffers overlap");
    for (const Range& b : ins)
      if (overlap(outs[i], b)) return fail(ATTN_ERR_INVALID, "an output or the workspace overlaps an input");
  }
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  attn::BwdArgs a;
  std::memset(&a, 0, sizeof a);
  const bool bf16 = dtype == ATTN_BF16;
  const int qrows = attn::bwd_q_rows(d);
  if ((rc = encode_bnhd(&a.tm_q, q, B, N, H, d, qrows, bf16)) ||
      (rc = encode_bnhd(&a.tm_k, k, B, N, H, d, 128, bf16)) ||
      (rc = encode_bnhd(&a.tm_v, v, B, N, H, d, 128, bf16)) ||
      (rc = encode_bnhd(&a.tm_do, dO, B, N, H, d, qrows, bf16)))
    return rc;
  const int npad = (N + 127) / 128 * 128;
  const size_t rows = (size_t)B * H * npad;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.o = o;
  a.dO = dO;
  a.lse = lse;
  if ((rc = make_dropout(0.f, 0, 0, &a.drop))) return rc;
  a.lse2 = reinterpret_cast<float*>(ws);
  a.dvec = reinterpret_cast<float*>(ws + up(rows * 4));
  a.dqacc = reinterpret_cast<float*>(ws + 2 * up(rows * 4));
  a.sched = reinterpret_cast<unsigned*>(ws + 2 * up(rows * 4) + up(rows * (size_t)d * 4));
  a.dq = dq;
  a.dk_acc = dk_acc;
  a.dv_acc = dv_acc;
  a.kv_flags = kv_flags;
  a.B = B; a.H = H; a.N = N; a.Npad = npad; a.d = d;
  a.sms = dev->sms;
  a.causal = causal ? 1 : 0;
  a.scale = scale;
  a.bf16 = bf16;
  {
    std::lock_guard<std::mutex> lk(g_mu);
    a.debug_flags = g_debug_flags;
    a.wait.limit_ns = g_wait_ns;
  }
  a.wait.status = dev->status;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (dq_flags & ATTN_ACC_FIRST) {
    e = timed(attn::kKBwdPre, s, [&] { return attn::launch_bwd_pre(a, s); });
    if (e != cudaSuccess) return cuda_fail(e, "attn_bwd_acc preprocess launch");
  }
  e = timed(attn::kKBwdMain, s, [&] { return attn::launch_bwd_main_acc(a, s); });
  if (e != cudaSuccess) return cuda_fail(e, "attn_bwd_acc main launch");
  if (dq_last) {
    e = timed(attn::kKDqPost, s, [&] { return attn::launch_dq_post(a, s); });
    if (e != cudaSuccess) return cuda_fail(e, "attn_bwd_acc dQ conversion launch");
  }
  return ATTN_OK;
}

int attn_cast_acc(const float* acc, void* out, size_t n, float mul, attn_dtype_t dtype, void* stream) {
  t_err.clear();
  if (!acc || !out) return fail(ATTN_ERR_INVALID, "null pointer argument");
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return fail(ATTN_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (n == 0 || n % 8 != 0 || n >= (1ull << 40))
    return fail(ATTN_ERR_INVALID, "n must be a positive multiple of 8 below 2^40 (got %zu)", n);
  if (!std::isfinite(mul)) return fail(ATTN_ERR_INVALID, "mul must be finite");
  if (!aligned16(acc) || !aligned16(out)) return fail(ATTN_ERR_ALIGN, "all pointers must be 16-byte aligned");
  if (overlap(rng(acc, n * 4), rng(out, n * 2))) return fail(ATTN_ERR_INVALID, "out overlaps acc");
  DeviceInfo* dev = nullptr;
  int rc = current_device(&dev);
  if (rc) return rc;
  cudaError_t e = attn::launch_cast_acc(acc, out, (long long)n, mul, dtype == ATTN_BF16, dev->sms,
                                        static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "attn_cast_acc launch");
  return ATTN_OK;
}

// ------------------------------------------------------------ paged 8-bit cache
namespace {

int page_shift_of(int page) {
  for (int s = 4; s <= 7; ++s)
    if (page == 1 << s) return s;
  return -1;
}

// One page of one head of a code tensor [P, H, page, d] per box.
int encode_pages(CUtensorMap* m, const void* ptr, long long PH, int page, int d) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)page, (cuuint64_t)PH};
  const cuuint64_t strides[2] = {(cuuint64_t)d, (cuuint64_t)page * d};
  const cuuint32_t box[3] = {(cuuint32_t)d, (cuuint32_t)page, 1};
  const cuuint32_t estr[3] = {1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, d == 128 ? CU_TENSOR_MAP_SWIZZLE_128B : CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return ATTN_OK;
}

// Outputs must not overlap one another or any input; allowed[i] (an input
// index or -1) names the input that output i may be.
int check_overlaps(const Range* outs, int n_out, const Range* ins, int n_in, const int* allowed = nullptr) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = i + 1; j < n_out; ++j)
      if (overlap(outs[i], outs[j])) return fail(ATTN_ERR_INVALID, "output buffers overlap");
    for (int j = 0; j < n_in; ++j) {
      if (allowed && allowed[i] == j && outs[i].lo == ins[j].lo) continue;
      if (overlap(outs[i], ins[j])) return fail(ATTN_ERR_INVALID, "an output or the workspace overlaps an input");
    }
  }
  return ATTN_OK;
}

int check_pages(const void* const* ptrs, int n, int B, int width, int free_cap, int page) {
  for (int i = 0; i < n; ++i) {
    if (!ptrs[i]) return fail(ATTN_ERR_INVALID, "null pointer argument");
    if (!aligned4(ptrs[i])) return fail(ATTN_ERR_ALIGN, "pointers must be 4-byte aligned");
  }
  if (B < 1 || width < 1 || free_cap < 1)
    return fail(ATTN_ERR_INVALID, "B, width, free_cap must be >= 1 (got %d, %d, %d)", B, width, free_cap);
  if (B > attn::kPagesMaxB) return fail(ATTN_ERR_UNSUPPORTED, "at most %d requests (got %d)", attn::kPagesMaxB, B);
  if (page_shift_of(page) < 0) return fail(ATTN_ERR_UNSUPPORTED, "page must be 16, 32, 64 or 128 (got %d)", page);
  if ((long long)width * page >= (1ll << 31)) return fail(ATTN_ERR_INVALID, "width * page must be < 2^31");
  return ATTN_OK;
}

void wait_ctl(DeviceInfo* dev, attn::WaitCtlHost* w, int* debug_flags) {
  std::lock_guard<std::mutex> lk(g_mu);
  *debug_flags = g_debug_flags;
  w->limit_ns = g_wait_ns;
  w->status = dev->status;
}

}  // namespace

int attn_pages_extend(const int32_t* lens, const int32_t* add, int B, int32_t* block_table, int width,
                      const int32_t* free_pages, const int32_t* free_count, int free_cap, int page, long long T,
                      int32_t* new_lens, int32_t* granted, int32_t* cu_new, int64_t* slots, int32_t* free_left,
                      void* stream) {
  t_err.clear();
  const void* ptrs[9] = {lens, add, block_table, free_pages, free_count, new_lens, granted, cu_new, free_left};
  int rc = check_pages(ptrs, 9, B, width, free_cap, page);
  if (rc) return rc;
  if (T < 0 || T >= (1ll << 31)) return fail(ATTN_ERR_INVALID, "T must be in [0, 2^31) (got %lld)", T);
  if (T > 0 && !slots) return fail(ATTN_ERR_INVALID, "null pointer argument");
  if (reinterpret_cast<uintptr_t>(slots) & 7u) return fail(ATTN_ERR_ALIGN, "slots must be 8-byte aligned");
  const size_t bb = (size_t)B * 4;
  const Range outs[6] = {rng(new_lens, bb), rng(free_left, 4), rng(block_table, bb * width), rng(granted, bb),
                         rng(cu_new, bb + 4), rng(slots, (size_t)T * 8)};
  const Range ins[4] = {rng(lens, bb), rng(free_count, 4), rng(add, bb), rng(free_pages, (size_t)free_cap * 4)};
  const int allowed[6] = {0, 1, -1, -1, -1, -1};
  if ((rc = check_overlaps(outs, 6, ins, 4, allowed))) return rc;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  attn::PagesArgs a = {};
  a.lens = lens; a.add = add; a.table = block_table; a.free_pages = free_pages; a.free_count = free_count;
  a.new_lens = new_lens; a.granted = granted; a.cu_new = cu_new;
  a.slots = reinterpret_cast<long long*>(slots);
  a.left = free_left;
  a.B = B; a.width = width; a.free_cap = free_cap; a.page_shift = page_shift_of(page); a.T = T;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed(attn::kKPagesExtend, s, [&] { return attn::launch_pages_extend(a, s); });
  return e != cudaSuccess ? cuda_fail(e, "attn_pages_extend launch") : ATTN_OK;
}

int attn_pages_release(const int32_t* lens, const int32_t* finished, int B, const int32_t* block_table, int width,
                       int32_t* free_pages, const int32_t* free_count, int free_cap, int page, int32_t* new_lens,
                       int32_t* free_left, void* stream) {
  t_err.clear();
  const void* ptrs[7] = {lens, finished, block_table, free_pages, free_count, new_lens, free_left};
  int rc = check_pages(ptrs, 7, B, width, free_cap, page);
  if (rc) return rc;
  const size_t bb = (size_t)B * 4;
  const Range outs[3] = {rng(new_lens, bb), rng(free_left, 4), rng(free_pages, (size_t)free_cap * 4)};
  const Range ins[4] = {rng(lens, bb), rng(free_count, 4), rng(finished, bb), rng(block_table, bb * width)};
  const int allowed[3] = {0, 1, -1};
  if ((rc = check_overlaps(outs, 3, ins, 4, allowed))) return rc;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  attn::PagesArgs a = {};
  a.lens = lens; a.add = finished; a.table = const_cast<int32_t*>(block_table); a.free_out = free_pages;
  a.free_count = free_count; a.new_lens = new_lens; a.left = free_left;
  a.B = B; a.width = width; a.free_cap = free_cap; a.page_shift = page_shift_of(page);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed(attn::kKPagesRelease, s, [&] { return attn::launch_pages_release(a, s); });
  return e != cudaSuccess ? cuda_fail(e, "attn_pages_release launch") : ATTN_OK;
}

// What the calls on a cache in `bits` bits ask of it.  (In 4 bits its rows are copied by TMA,
// which unpacks them: 32-byte aligned.)
static int check_cache(const uint8_t* k_cache, const uint8_t* v_cache, const void* k_scale, const void* v_scale, int H,
                       int d, int P, int page, attn_dtype_t dtype, int bits) {
  if (!k_cache || !v_cache || !k_scale || !v_scale) return fail(ATTN_ERR_INVALID, "null pointer argument");
  if (H < 1 || P < 1) return fail(ATTN_ERR_INVALID, "H >= 1, P >= 1 needed (got %d, %d)", H, P);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim d=%d not supported (64 or 128)", d);
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return fail(ATTN_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (page_shift_of(page) < 0) return fail(ATTN_ERR_UNSUPPORTED, "page must be 16, 32, 64 or 128 (got %d)", page);
  if ((long long)P * H >= (1ll << 31) || (long long)H * d >= (1ll << 32))
    return fail(ATTN_ERR_INVALID, "P * H must be < 2^31, H * d < 2^32");
  const uintptr_t c = reinterpret_cast<uintptr_t>(k_cache) | reinterpret_cast<uintptr_t>(v_cache);
  const uintptr_t s = reinterpret_cast<uintptr_t>(k_scale) | reinterpret_cast<uintptr_t>(v_scale);
  if (c & (bits == 4 ? 31u : 15u)) return fail(ATTN_ERR_ALIGN, "the caches must be %d-byte aligned", bits == 4 ? 32 : 16);
  if (s & (bits == 4 ? 15u : 3u)) return fail(ATTN_ERR_ALIGN, "scales must be %d-byte aligned", bits == 4 ? 16 : 4);
  return ATTN_OK;
}
static size_t code_bytes(int P, int H, int page, int d, int bits) { return (size_t)P * H * page * (d * bits / 8); }
static size_t scale_bytes(int P, int H, int page, int d, int bits) {
  return (size_t)P * H * (bits == 4 ? (size_t)page * (d / 32) * 2 : 4);
}

int attn_kv4_append(const void* k, const void* v, long long k_stride, long long v_stride, const int64_t* slots,
                    long long T, int H, int d, uint8_t* k_cache, uint8_t* v_cache, uint16_t* k_scale,
                    uint16_t* v_scale, int P, int page, attn_dtype_t dtype, void* stream) {
  t_err.clear();
  if (T == 0) return ATTN_OK;
  if (!k || !v || !slots) return fail(ATTN_ERR_INVALID, "null pointer argument");
  int rc = check_cache(k_cache, v_cache, k_scale, v_scale, H, d, P, page, dtype, 4);
  if (rc) return rc;
  if (T < 0 || T >= (1ll << 31) || T * H >= (1ll << 30)) return fail(ATTN_ERR_INVALID, "T * H must be in [0, 2^30)");
  const long long hd = (long long)H * d;
  if (k_stride < hd || v_stride < hd || k_stride % 8 || v_stride % 8 || k_stride >= (1ll << 32) || v_stride >= (1ll << 32))
    return fail(ATTN_ERR_INVALID, "token strides must be multiples of 8, at least H * d, below 2^32");
  if (!aligned16(k) || !aligned16(v)) return fail(ATTN_ERR_ALIGN, "k and v must be 16-byte aligned");
  if (reinterpret_cast<uintptr_t>(slots) & 7u) return fail(ATTN_ERR_ALIGN, "slots must be 8-byte aligned");
  const size_t cb = code_bytes(P, H, page, d, 4), sb = scale_bytes(P, H, page, d, 4);
  const Range outs[4] = {rng(k_cache, cb), rng(v_cache, cb), rng(k_scale, sb), rng(v_scale, sb)};
  const Range ins[3] = {rng(k, ((size_t)(T - 1) * k_stride + hd) * 2), rng(v, ((size_t)(T - 1) * v_stride + hd) * 2),
                        rng(slots, (size_t)T * 8)};
  if ((rc = check_overlaps(outs, 4, ins, 3))) return rc;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  attn::Kv4AppendArgs a = {};
  a.x[0] = k; a.x[1] = v;
  a.cache[0] = k_cache; a.cache[1] = v_cache;
  a.scale[0] = k_scale; a.scale[1] = v_scale;
  a.slots = reinterpret_cast<const long long*>(slots);
  a.x_stride[0] = k_stride; a.x_stride[1] = v_stride;
  a.T = T;
  a.n_slots = (long long)P * page;
  a.H = H; a.d = d; a.page_shift = page_shift_of(page); a.bf16 = dtype == ATTN_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed(attn::kKKv4Append, s, [&] { return attn::launch_kv4_append(a, dev->sms, s); });
  return e != cudaSuccess ? cuda_fail(e, "attn_kv4_append launch") : ATTN_OK;
}

size_t attn_kv4_decode_workspace_size(int Nq, int Hq, int H, int d) {
  if (Nq < 1 || Nq > 128 || H < 1 || Hq < H || Hq % H || Hq / H > (1 << 23) || (d != 64 && d != 128)) return 0;
  const size_t rows = (size_t)attn::kKvMaxCtas * 2 * attn::kv4_rows(Nq * (Hq / H), true);
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  return up(rows * d * 4) + up(rows * 2 * 4);
}

// A page of one head a box, rows of 128 channels, unpacked by the copy.
static int encode_pages4(CUtensorMap* m, const void* ptr, long long PH, int page, int d) {
  const cuuint32_t rows = (cuuint32_t)(page * d / 128);
  const cuuint64_t dims[3] = {128, rows, (cuuint64_t)PH}, strides[2] = {64, (cuuint64_t)rows * 64};
  const cuuint32_t box[3] = {128, rows, 1}, estr[3] = {1, 1, 1};
  CUresult r = g_encode(m, CU_TENSOR_MAP_DATA_TYPE_16U4_ALIGN16B, 3, const_cast<void*>(ptr), dims, strides, box, estr,
                        CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return ATTN_OK;
}

// Whether the GPU has the SMs together for a cluster of the call's: beyond 8 not every GPU, or part of one, does.  Asked
// once for each form of the kernel (0.7 us).
static bool kv4_fits(DeviceInfo* dev, const attn::KvDecArgs& a) {
  const int bit = 2 * ((a.d == 128 ? 0 : 6) + (a.bf16 ? 0 : 3) + (a.rp == 4 ? 0 : (a.rp == 8 ? 1 : 2)));
  unsigned got = dev->kv4_fit >> bit & 3u;
  if (!got) {
    got = attn::kv4_clusters_fit(a) ? 3u : 1u;
    dev->kv4_fit |= got << bit;
  }
  return got == 3u;
}

int attn_kv4_decode(const void* q, const uint8_t* k_cache, const uint8_t* v_cache, const uint16_t* k_scale,
                    const uint16_t* v_scale, const int32_t* block_table, const int32_t* lens, void* o, float* lse, int B,
                    int Nq, int Hq, int H, int d, int P, int page, int width, float scale, int causal,
                    attn_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  t_err.clear();
  if (!q || !block_table || !lens || !o || !lse) return fail(ATTN_ERR_INVALID, "null pointer argument");
  int rc = check_cache(k_cache, v_cache, k_scale, v_scale, H, d, P, page, dtype, 4);
  if (rc) return rc;
  if (B < 1 || Nq < 1 || Hq < 1 || width < 1) return fail(ATTN_ERR_INVALID, "B, Nq, Hq, width must be >= 1");
  if (Hq % H) return fail(ATTN_ERR_INVALID, "Hq = %d is no multiple of H = %d", Hq, H);
  if (Nq > 128) return fail(ATTN_ERR_UNSUPPORTED, "decode takes at most 128 query rows (got %d)", Nq);
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(ATTN_ERR_INVALID, "scale must be finite and > 0");
  // (the kernels round a length up to whole tiles of 256 tokens in 32 bits)
  if ((long long)width * page > (1ll << 31) - 256 || (long long)B * Nq * Hq >= (1ll << 31) || Hq / H > (1 << 23))
    return fail(ATTN_ERR_INVALID, "B * Nq * Hq must be < 2^31, Hq / H at most 2^23, width * page at most 2^31 - 256");
  if (!aligned16(q) || !aligned16(o) || !aligned16(lse)) return fail(ATTN_ERR_ALIGN, "q, o and lse must be 16-byte aligned");
  if (!aligned4(block_table) || !aligned4(lens)) return fail(ATTN_ERR_ALIGN, "block_table and lens must be 4-byte aligned");
  const size_t need = attn_kv4_decode_workspace_size(Nq, Hq, H, d);
  if (!workspace || workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(ATTN_ERR_ALIGN, "workspace must be 256-byte aligned");
  const size_t qb = (size_t)B * Nq * Hq * d * 2, cb = code_bytes(P, H, page, d, 4), sb = scale_bytes(P, H, page, d, 4);
  const Range outs[3] = {rng(o, qb), rng(lse, (size_t)B * Nq * Hq * 4), rng(workspace, need)};
  const Range ins[7] = {rng(q, qb), rng(k_cache, cb), rng(v_cache, cb), rng(k_scale, sb), rng(v_scale, sb),
                        rng(block_table, (size_t)B * width * 4), rng(lens, (size_t)B * 4)};
  if ((rc = check_overlaps(outs, 3, ins, 7))) return rc;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  attn::KvDecArgs a;
  std::memset(&a, 0, sizeof a);
  if ((rc = encode_pages4(&a.tm_k, k_cache, (long long)P * H, page, d)) ||
      (rc = encode_pages4(&a.tm_v, v_cache, (long long)P * H, page, d)))
    return rc;
  a.q = q; a.o = o; a.lse = lse;
  a.k_scale16 = k_scale; a.v_scale16 = v_scale; a.table = block_table; a.lens = lens;
  a.B = B; a.Nq = Nq; a.Hq = Hq; a.H = H; a.G = Hq / H; a.d = d;
  a.width = width; a.page_shift = page_shift_of(page); a.P = P;
  const int R = Nq * a.G;
  a.bf16 = dtype == ATTN_BF16;
  a.rp = attn::kv4_rows(R, a.bf16);
  a.n_rb = (R + a.rp - 1) / a.rp;
  a.causal = causal ? 1 : 0;
  a.scale = scale;
  const long long tile = 128 * (128 / d), tiles = ((long long)width * page + tile - 1) / tile;
  const long long segs = (long long)B * H * a.n_rb;
  auto deal = [&](int most) {
    a.cluster = attn::kv4_cluster(a.rp, a.bf16, dev->sms, B, segs, tiles, most);
    a.grid = a.cluster ? (int)(segs * a.cluster) : attn::kv4_grid(a.rp, a.bf16, dev->sms, tiles * segs);
  };
  deal(attn::kKv4MaxCluster);
  if (a.cluster > 8 && !kv4_fits(dev, a)) deal(8);
  a.full = attn::kv4_full(a.rp, a.bf16, dev->sms, a.grid);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.ws_o = reinterpret_cast<float*>(ws);
  a.ws_ml = reinterpret_cast<float*>(ws + ((size_t)attn::kKvMaxCtas * 2 * a.rp * d * 4 + 255) / 256 * 256);
  wait_ctl(dev, &a.wait, &a.debug_flags);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed(attn::kKKv4Split, s, [&] { return attn::launch_kv4_split(a, s); });
  if (e != cudaSuccess) return cuda_fail(e, "attn_kv4_decode launch");
  if (a.cluster) return ATTN_OK;
  e = timed(attn::kKKv4Merge, s, [&] { return attn::launch_kv_merge(a, s); });
  return e != cudaSuccess ? cuda_fail(e, "attn_kv4_decode merge launch") : ATTN_OK;
}

int attn_kv_read(const uint8_t* k_cache, const uint8_t* v_cache, const void* k_scale, const void* v_scale,
                 const int32_t* block_table, const int32_t* lens, const int32_t* cu, void* k, void* v, int B,
                 long long T, int H, int d, int P, int page, int width, int bits, attn_dtype_t dtype, void* stream) {
  t_err.clear();
  if (bits != 8 && bits != 4) return fail(ATTN_ERR_UNSUPPORTED, "caches hold 8 or 4 bits (got %d)", bits);
  int rc = check_cache(k_cache, v_cache, k_scale, v_scale, H, d, P, page, dtype, bits);
  if (rc) return rc;
  if (!block_table || !lens || !cu || (T > 0 && (!k || !v))) return fail(ATTN_ERR_INVALID, "null pointer argument");
  if (B < 1 || width < 1) return fail(ATTN_ERR_INVALID, "B >= 1, width >= 1 needed (got %d, %d)", B, width);
  if (T < 0 || T >= (1ll << 31) || T * H >= (1ll << 33)) return fail(ATTN_ERR_INVALID, "T must be in [0, 2^31), T * H below 2^33");
  if ((long long)width * page >= (1ll << 31)) return fail(ATTN_ERR_INVALID, "width * page must be < 2^31");
  if ((reinterpret_cast<uintptr_t>(k) | reinterpret_cast<uintptr_t>(v)) & 31u)
    return fail(ATTN_ERR_ALIGN, "k and v must be 32-byte aligned");
  if (!aligned4(block_table) || !aligned4(lens) || !aligned4(cu))
    return fail(ATTN_ERR_ALIGN, "block_table, lens and cu must be 4-byte aligned");
  if (T == 0) return ATTN_OK;
  const size_t cb = code_bytes(P, H, page, d, bits), sb = scale_bytes(P, H, page, d, bits), ob = (size_t)T * H * d * 2;
  const Range outs[2] = {rng(k, ob), rng(v, ob)};
  const Range ins[7] = {rng(k_cache, cb), rng(v_cache, cb), rng(k_scale, sb), rng(v_scale, sb),
                        rng(block_table, (size_t)B * width * 4), rng(lens, (size_t)B * 4), rng(cu, (size_t)B * 4 + 4)};
  if ((rc = check_overlaps(outs, 2, ins, 7))) return rc;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  attn::KvReadArgs a = {};
  a.cache[0] = k_cache; a.cache[1] = v_cache;
  a.scale[0] = k_scale; a.scale[1] = v_scale;
  a.out[0] = k; a.out[1] = v;
  a.table = block_table; a.lens = lens; a.cu = cu;
  a.T = T;
  a.B = B; a.H = H; a.d = d; a.P = P; a.page_shift = page_shift_of(page); a.width = width;
  a.bf16 = dtype == ATTN_BF16; a.bits = bits;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed(attn::kKKvRead, s, [&] { return attn::launch_kv_read(a, dev->sms, s); });
  return e != cudaSuccess ? cuda_fail(e, "attn_kv_read launch") : ATTN_OK;
}

int attn_kv8_append(const void* k, const void* v, long long k_stride, long long v_stride, const int64_t* slots,
                    long long T, int H, int d, uint8_t* k_cache, uint8_t* v_cache, float* k_scale, float* v_scale,
                    int P, int page, attn_dtype_t dtype, void* stream) {
  t_err.clear();
  if (T == 0) return ATTN_OK;
  if (!k || !v || !slots || !k_cache || !v_cache || !k_scale || !v_scale)
    return fail(ATTN_ERR_INVALID, "null pointer argument");
  if (T < 0 || H < 1 || P < 1) return fail(ATTN_ERR_INVALID, "T >= 0, H >= 1, P >= 1 needed (got %lld, %d, %d)", T, H, P);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim d=%d not supported (64 or 128)", d);
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return fail(ATTN_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (page_shift_of(page) < 0) return fail(ATTN_ERR_UNSUPPORTED, "page must be 16, 32, 64 or 128 (got %d)", page);
  if (T * H >= (1ll << 30) || T >= (1ll << 31)) return fail(ATTN_ERR_INVALID, "T * H must be < 2^30");
  if ((long long)P * H >= (1ll << 31)) return fail(ATTN_ERR_INVALID, "P * H must be < 2^31");
  const long long hd = (long long)H * d;
  if (k_stride < hd || v_stride < hd || k_stride % 8 || v_stride % 8 || k_stride >= (1ll << 32) || v_stride >= (1ll << 32))
    return fail(ATTN_ERR_INVALID, "token strides must be multiples of 8, at least H * d");
  if (!aligned16(k) || !aligned16(v) || !aligned16(k_cache) || !aligned16(v_cache))
    return fail(ATTN_ERR_ALIGN, "k, v and the caches must be 16-byte aligned");
  if (!aligned4(k_scale) || !aligned4(v_scale) || (reinterpret_cast<uintptr_t>(slots) & 7u))
    return fail(ATTN_ERR_ALIGN, "scales must be 4-byte, slots 8-byte aligned");
  const size_t cb = (size_t)P * H * page * d, sb = (size_t)P * H * 4;
  const Range outs[4] = {rng(k_cache, cb), rng(v_cache, cb), rng(k_scale, sb), rng(v_scale, sb)};
  const Range ins[3] = {rng(k, ((size_t)(T - 1) * k_stride + hd) * 2), rng(v, ((size_t)(T - 1) * v_stride + hd) * 2),
                        rng(slots, (size_t)T * 8)};
  int rc = check_overlaps(outs, 4, ins, 3);
  if (rc) return rc;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  attn::Kv8AppendArgs a = {};
  a.x[0] = k; a.x[1] = v;
  a.cache[0] = k_cache; a.cache[1] = v_cache;
  a.scale[0] = k_scale; a.scale[1] = v_scale;
  a.slots = reinterpret_cast<const long long*>(slots);
  a.x_stride[0] = k_stride; a.x_stride[1] = v_stride;
  a.T = T;
  a.n_slots = (long long)P * page;
  a.H = H; a.d = d; a.page_shift = page_shift_of(page); a.bf16 = dtype == ATTN_BF16;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed(attn::kKKv8Append, s, [&] { return attn::launch_kv8_append(a, dev->sms, s); });
  return e != cudaSuccess ? cuda_fail(e, "attn_kv8_append launch") : ATTN_OK;
}

size_t attn_kv8_decode_workspace_size(int Nq, int Hq, int H, int d) {
  if (Nq < 1 || H < 1 || Hq < H || Hq % H || (d != 64 && d != 128)) return 0;
  const size_t rows = (size_t)attn::kKvMaxCtas * 2 * attn::kv8_rows(Nq * (Hq / H));
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  return up(rows * d * 4) + up(rows * 2 * 4);
}

int attn_kv8_decode(const void* q, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                    const float* v_scale, const int32_t* block_table, const int32_t* lens, void* o, float* lse, int B,
                    int Nq, int Hq, int H, int d, int P, int page, int width, float scale, int causal,
                    attn_dtype_t dtype, void* workspace, size_t workspace_bytes, void* stream) {
  t_err.clear();
  if (!q || !k_cache || !v_cache || !k_scale || !v_scale || !block_table || !lens || !o || !lse)
    return fail(ATTN_ERR_INVALID, "null pointer argument");
  if (B < 1 || Nq < 1 || H < 1 || Hq < 1 || P < 1 || width < 1)
    return fail(ATTN_ERR_INVALID, "B, Nq, Hq, H, P, width must be >= 1");
  if (Hq % H) return fail(ATTN_ERR_INVALID, "Hq = %d is no multiple of H = %d", Hq, H);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim d=%d not supported (64 or 128)", d);
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return fail(ATTN_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (Nq > 128) return fail(ATTN_ERR_UNSUPPORTED, "decode takes at most 128 query rows (got %d)", Nq);
  const int shift = page_shift_of(page);
  if (shift < 0) return fail(ATTN_ERR_UNSUPPORTED, "page must be 16, 32, 64 or 128 (got %d)", page);
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(ATTN_ERR_INVALID, "scale must be finite and > 0");
  // (the kernels round a length up to whole tiles of 128 keys in 32 bits)
  if ((long long)P * H >= (1ll << 31) || (long long)width * page > (1ll << 31) - 128 || (long long)B * Nq * Hq >= (1ll << 31))
    return fail(ATTN_ERR_INVALID, "P * H and B * Nq * Hq must be < 2^31, width * page at most 2^31 - 128");
  if (!aligned16(q) || !aligned16(k_cache) || !aligned16(v_cache) || !aligned16(o) || !aligned16(lse))
    return fail(ATTN_ERR_ALIGN, "q, o, lse and the caches must be 16-byte aligned");
  if (!aligned4(k_scale) || !aligned4(v_scale) || !aligned4(block_table) || !aligned4(lens))
    return fail(ATTN_ERR_ALIGN, "scales, block_table and lens must be 4-byte aligned");
  const size_t need = attn_kv8_decode_workspace_size(Nq, Hq, H, d);
  if (!workspace || workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(ATTN_ERR_ALIGN, "workspace must be 256-byte aligned");
  const size_t qb = (size_t)B * Nq * Hq * d * 2, cb = (size_t)P * H * page * d, sb = (size_t)P * H * 4;
  const Range outs[3] = {rng(o, qb), rng(lse, (size_t)B * Nq * Hq * 4), rng(workspace, need)};
  const Range ins[7] = {rng(q, qb), rng(k_cache, cb), rng(v_cache, cb), rng(k_scale, sb), rng(v_scale, sb),
                        rng(block_table, (size_t)B * width * 4), rng(lens, (size_t)B * 4)};
  int rc = check_overlaps(outs, 3, ins, 7);
  if (rc) return rc;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  attn::KvDecArgs a;
  std::memset(&a, 0, sizeof a);
  if ((rc = encode_pages(&a.tm_k, k_cache, (long long)P * H, page, d)) ||
      (rc = encode_pages(&a.tm_v, v_cache, (long long)P * H, page, d)))
    return rc;
  a.q = q; a.o = o; a.lse = lse;
  a.k_scale = k_scale; a.v_scale = v_scale; a.table = block_table; a.lens = lens;
  a.B = B; a.Nq = Nq; a.Hq = Hq; a.H = H; a.G = Hq / H; a.d = d;
  a.width = width; a.page_shift = shift; a.P = P;
  const int R = Nq * a.G;
  a.rp = attn::kv8_rows(R);
  a.n_rb = (R + a.rp - 1) / a.rp;
  a.causal = causal ? 1 : 0;
  a.bf16 = dtype == ATTN_BF16;
  a.scale = scale;
  const long long tiles = ((long long)width * page + 127) / 128;
  a.grid = attn::kv8_grid(a.rp, dev->sms, tiles * B * H * a.n_rb);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.ws_o = reinterpret_cast<float*>(ws);
  a.ws_ml = reinterpret_cast<float*>(ws + ((size_t)attn::kKvMaxCtas * 2 * a.rp * d * 4 + 255) / 256 * 256);
  wait_ctl(dev, &a.wait, &a.debug_flags);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed(attn::kKKv8Split, s, [&] { return attn::launch_kv8_split(a, s); });
  if (e != cudaSuccess) return cuda_fail(e, "attn_kv8_decode launch");
  e = timed(attn::kKKv8Merge, s, [&] { return attn::launch_kv_merge(a, s); });
  return e != cudaSuccess ? cuda_fail(e, "attn_kv8_decode merge launch") : ATTN_OK;
}

// ------------------------------------------------------------ packed batches
namespace {

// A packed [T, H, d] 16-bit tensor, `stride` elements from token to token, as
// (d, head, row window, place): the last two dimensions both step by a token,
// so that a box of `heads` heads and `rows` tokens may begin up to `rows` tokens
// before its place and reads zeros there (see attn_fwd.cu).
int encode_packed(CUtensorMap* m, const void* ptr, long long T, int H, int d, long long stride, int heads, int rows,
                  bool bf16) {
  const cuuint64_t dims[4] = {(cuuint64_t)d, (cuuint64_t)H, 128, (cuuint64_t)T};
  const cuuint64_t strides[3] = {(cuuint64_t)d * 2, (cuuint64_t)stride * 2, (cuuint64_t)stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)heads, (cuuint32_t)rows, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  CUresult r = g_encode(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
                        const_cast<void*>(ptr), dims, strides, box, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                        CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
  if (r != CUDA_SUCCESS) return fail(ATTN_ERR_CUDA, "cuTensorMapEncodeTiled failed (%d)", (int)r);
  return ATTN_OK;
}

int check_packed(const int32_t* cu_q, const int32_t* cu_k, int B, long long Tq, long long Tk, int Hq, int Hkv, int d,
                 long long q_stride, long long k_stride, long long v_stride, float scale, attn_dtype_t dtype) {
  if (!cu_q || !cu_k) return fail(ATTN_ERR_INVALID, "null pointer argument");
  if (!aligned4(cu_q) || !aligned4(cu_k)) return fail(ATTN_ERR_ALIGN, "cu_q, cu_k must be 4-byte aligned");
  if (B < 1 || Hq < 1 || Hkv < 1) return fail(ATTN_ERR_INVALID, "B, Hq, Hkv must be >= 1 (got %d, %d, %d)", B, Hq, Hkv);
  if (B > attn::kVarMaxB) return fail(ATTN_ERR_UNSUPPORTED, "at most %d sequences (got %d)", attn::kVarMaxB, B);
  if (Hq % Hkv || Hq / Hkv > 1024)
    return fail(ATTN_ERR_INVALID, "Hq = %d must be a multiple of Hkv = %d, at most 1024 times it", Hq, Hkv);
  if (Tq < 0 || Tk < 0 || Tq >= (1ll << 26) || Tk >= (1ll << 26))
    return fail(ATTN_ERR_INVALID, "Tq, Tk must be in [0, 2^26) (got %lld, %lld)", Tq, Tk);
  if (d != 64 && d != 128) return fail(ATTN_ERR_UNSUPPORTED, "head dim d=%d not supported (64 or 128)", d);
  if (dtype != ATTN_F16 && dtype != ATTN_BF16) return fail(ATTN_ERR_UNSUPPORTED, "unknown dtype %d", (int)dtype);
  if (!std::isfinite(scale) || !(scale > 0.f)) return fail(ATTN_ERR_INVALID, "scale must be finite and > 0");
  const long long hq = (long long)Hq * d, hk = (long long)Hkv * d;
  if (q_stride < hq || k_stride < hk || v_stride < hk || q_stride % d || k_stride % d || v_stride % d ||
      q_stride >= (1ll << 30) || k_stride >= (1ll << 30) || v_stride >= (1ll << 30))
    return fail(ATTN_ERR_INVALID, "token strides must be multiples of d, at least heads * d");
  if ((Tq / 128 + B) * Hq >= (1ll << 31) || (Tk / 128 + B) * Hkv >= (1ll << 31) || Tq * hq >= (1ll << 40) ||
      Tk * hk >= (1ll << 40))
    return fail(ATTN_ERR_INVALID, "too many tiles or elements");
  return ATTN_OK;
}

long long varlen_padded(int B, long long Tq) { return (Tq / 64 + B) * 64; }

size_t packed_bytes(long long T, long long stride, long long row) {
  return T > 0 ? ((size_t)(T - 1) * stride + row) * 2 : 0;
}

}  // namespace

// CTAs that share a pair of query tiles, and the CTAs in all.
static int varlen_fwd_split(int B, long long Tq, long long Tk, int Hq, int Hkv, long long* ctas) {
  int Gp, R;
  attn::fwd_varlen_shape(Hq / Hkv, Tq, B, &Gp, &R);
  const long long n = attn::fwd_varlen_grid(Tq, B, Hq, Gp, R);
  const int nsplit = attn::fwd_varlen_nsplit(n, Tk);
  *ctas = n * nsplit;
  return nsplit;
}

size_t attn_varlen_fwd_workspace_size(int B, long long Tq, long long Tk, int Hq, int Hkv, int d) {
  if (B < 1 || B > attn::kVarMaxB || Tq < 1 || Tk < 0 || Tq >= (1ll << 26) || Tk >= (1ll << 26) || Hkv < 1 ||
      Hq < Hkv || Hq % Hkv || (d != 64 && d != 128))
    return 0;
  long long ctas = 0;
  if (varlen_fwd_split(B, Tq, Tk, Hq, Hkv, &ctas) == 1) return 0;
  return (size_t)ctas * 2 * 128 * (d + 2) * 4;
}

int attn_varlen_fwd(const void* q, const void* k, const void* v, void* o, float* lse, const int32_t* cu_q,
                    const int32_t* cu_k, int B, long long Tq, long long Tk, int Hq, int Hkv, int d, long long q_stride,
                    long long k_stride, long long v_stride, float scale, int causal, attn_dtype_t dtype,
                    void* workspace, size_t workspace_bytes, void* stream) {
  t_err.clear();
  int rc = check_packed(cu_q, cu_k, B, Tq, Tk, Hq, Hkv, d, q_stride, k_stride, v_stride, scale, dtype);
  if (rc) return rc;
  if (Tq == 0) return ATTN_OK;
  if (!q || !o || !lse || (Tk > 0 && (!k || !v))) return fail(ATTN_ERR_INVALID, "null pointer argument");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse))
    return fail(ATTN_ERR_ALIGN, "q, k, v, o and lse must be 16-byte aligned");
  const size_t need = attn_varlen_fwd_workspace_size(B, Tq, Tk, Hq, Hkv, d);
  if (need && (!workspace || workspace_bytes < need))
    return fail(ATTN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  if (need && (reinterpret_cast<uintptr_t>(workspace) & 255u))
    return fail(ATTN_ERR_ALIGN, "workspace must be 256-byte aligned");
  const long long hq = (long long)Hq * d, hk = (long long)Hkv * d;
  const size_t cb = ((size_t)B + 1) * 4;
  const Range outs[3] = {rng(o, packed_bytes(Tq, hq, hq)), rng(lse, (size_t)Tq * Hq * 4), rng(workspace, need)};
  const Range ins[5] = {rng(q, packed_bytes(Tq, q_stride, hq)), rng(k, packed_bytes(Tk, k_stride, hk)),
                        rng(v, packed_bytes(Tk, v_stride, hk)), rng(cu_q, cb), rng(cu_k, cb)};
  if ((rc = check_overlaps(outs, 3, ins, 5))) return rc;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  attn::FwdArgs a;
  std::memset(&a, 0, sizeof a);
  const bool bf16 = dtype == ATTN_BF16;
  a.G = Hq / Hkv;
  attn::fwd_varlen_shape(a.G, Tq, B, &a.Gp, &a.R);
  // (without keys no K or V tile is loaded; their maps still need an address)
  if ((rc = encode_packed(&a.tm_q, q, Tq, Hq, d, q_stride, a.Gp, a.R, bf16)) ||
      (rc = encode_packed(&a.tm_k, Tk ? k : q, Tk ? Tk : 1, Hkv, d, Tk ? k_stride : hk, 1, 128, bf16)) ||
      (rc = encode_packed(&a.tm_v, Tk ? v : q, Tk ? Tk : 1, Hkv, d, Tk ? v_stride : hk, 1, 128, bf16)) ||
      (rc = encode_packed(&a.tm_o, o, Tq, Hq, d, hq, a.Gp, a.R, bf16)))
    return rc;
  a.o = o;
  a.lse = lse;
  if ((rc = make_dropout(0.f, 0, 0, &a.drop))) return rc;
  a.B = B; a.H = Hq; a.N = (int)Tq; a.d = d;
  a.cu_q = cu_q; a.cu_k = cu_k;
  a.Nk = (int)Tk;
  long long ctas = 0;
  a.nsplit = varlen_fwd_split(B, Tq, Tk, Hq, Hkv, &ctas);
  if (need) {
    a.ws_o = static_cast<float*>(workspace);
    a.ws_ml = a.ws_o + (size_t)ctas * 2 * 128 * d;
  }
  a.causal = causal ? 1 : 0;
  a.scale = scale;
  a.bf16 = bf16;
  wait_ctl(dev, &a.wait, &a.debug_flags);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed(attn::kKFwd, s, [&] { return attn::launch_fwd_varlen(a, s); });
  if (e != cudaSuccess) return cuda_fail(e, "attn_varlen_fwd launch");
  if (a.nsplit == 1) return ATTN_OK;
  e = timed(attn::kKVarMerge, s, [&] { return attn::launch_var_merge(a, s); });
  return e != cudaSuccess ? cuda_fail(e, "attn_varlen_fwd merge launch") : ATTN_OK;
}

// Bytes of the partial dK, dV tiles.
static size_t varlen_parts_bytes(long long Tq, int Hq, int Hkv, int d) {
  return attn::var_may_split(Tq, Hq / Hkv) ? (size_t)attn::kVarMaxParts * 2 * 128 * d * 4 : 0;
}

// Integers of the item counts and the order of the sequences.
static size_t varlen_items(int B) { return (size_t)attn::kVarClasses * B + 1 + B; }

size_t attn_varlen_bwd_workspace_size(int B, long long Tq, int Hq, int Hkv, int d) {
  if (B < 1 || B > attn::kVarMaxB || Tq < 0 || Tq >= (1ll << 26) || Hkv < 1 || Hq < Hkv || Hq % Hkv ||
      (d != 64 && d != 128))
    return 0;
  const size_t rows = (size_t)varlen_padded(B, Tq) * Hq;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  return up(rows * 4) * 2 + up(rows * d * 4) + 256 + up((size_t)B * sizeof(attn::VarBwdSeq)) +
         up(varlen_items(B) * 4) + varlen_parts_bytes(Tq, Hq, Hkv, d);
}

int attn_varlen_bwd(const void* q, const void* k, const void* v, const void* o, const float* lse, const void* dO,
                    void* dq, void* dk, void* dv, const int32_t* cu_q, const int32_t* cu_k, int B, long long Tq,
                    long long Tk, int Hq, int Hkv, int d, long long q_stride, long long k_stride, long long v_stride,
                    float scale, int causal, attn_dtype_t dtype, void* workspace, size_t workspace_bytes,
                    void* stream) {
  t_err.clear();
  int rc = check_packed(cu_q, cu_k, B, Tq, Tk, Hq, Hkv, d, q_stride, k_stride, v_stride, scale, dtype);
  if (rc) return rc;
  if (Tq == 0 && Tk == 0) return ATTN_OK;
  if ((Tq > 0 && (!q || !o || !lse || !dO || !dq)) || (Tk > 0 && (!k || !v || !dk || !dv)))
    return fail(ATTN_ERR_INVALID, "null pointer argument");
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || !aligned16(lse) || !aligned16(dO) ||
      !aligned16(dq) || !aligned16(dk) || !aligned16(dv))
    return fail(ATTN_ERR_ALIGN, "all pointers must be 16-byte aligned");
  const size_t need = attn_varlen_bwd_workspace_size(B, Tq, Hq, Hkv, d);
  if (!workspace || workspace_bytes < need)
    return fail(ATTN_ERR_WORKSPACE, "workspace of %zu bytes needed, %zu given", need, workspace_bytes);
  if (reinterpret_cast<uintptr_t>(workspace) & 255u)
    return fail(ATTN_ERR_ALIGN, "workspace must be 256-byte aligned");
  const long long hq = (long long)Hq * d, hk = (long long)Hkv * d;
  const size_t cb = ((size_t)B + 1) * 4, qb = packed_bytes(Tq, hq, hq), kb = packed_bytes(Tk, hk, hk);
  const Range outs[4] = {rng(dq, qb), rng(dk, kb), rng(dv, kb), rng(workspace, need)};
  const Range ins[8] = {rng(q, packed_bytes(Tq, q_stride, hq)), rng(k, packed_bytes(Tk, k_stride, hk)),
                        rng(v, packed_bytes(Tk, v_stride, hk)), rng(o, qb), rng(lse, (size_t)Tq * Hq * 4),
                        rng(dO, qb), rng(cu_q, cb), rng(cu_k, cb)};
  if ((rc = check_overlaps(outs, 4, ins, 8))) return rc;
  DeviceInfo* dev = nullptr;
  if ((rc = current_device(&dev))) return rc;
  attn::BwdArgs a;
  std::memset(&a, 0, sizeof a);
  const bool bf16 = dtype == ATTN_BF16;
  const long long npad = varlen_padded(B, Tq);
  const size_t rows = (size_t)npad * Hq;
  auto up = [](size_t x) { return (x + 255) / 256 * 256; };
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  a.o = o;
  a.dO = dO;
  a.lse = lse;
  if ((rc = make_dropout(0.f, 0, 0, &a.drop))) return rc;
  a.lse2 = reinterpret_cast<float*>(ws);
  a.dvec = reinterpret_cast<float*>(ws + up(rows * 4));
  a.dqacc = reinterpret_cast<float*>(ws + 2 * up(rows * 4));
  ws += 2 * up(rows * 4) + up(rows * (size_t)d * 4);
  a.sched = reinterpret_cast<unsigned*>(ws);
  a.var_seq = reinterpret_cast<attn::VarBwdSeq*>(ws + 256);
  a.var_items = reinterpret_cast<int*>(ws + 256 + up((size_t)B * sizeof(attn::VarBwdSeq)));
  a.var_order = a.var_items + varlen_items(B) - B;
  a.var_parts = reinterpret_cast<float*>(ws + 256 + up((size_t)B * sizeof(attn::VarBwdSeq)) + up(varlen_items(B) * 4));
  a.dq = dq; a.dk = dk; a.dv = dv;
  a.B = B; a.H = Hq; a.N = (int)Tq; a.Npad = (int)npad; a.d = d;
  a.cu_q = cu_q; a.cu_k = cu_k;
  a.Nk = (int)Tk; a.G = Hq / Hkv; a.Hkv = Hkv;
  a.sms = dev->sms;
  a.causal = causal ? 1 : 0;
  a.scale = scale;
  a.bf16 = bf16;
  wait_ctl(dev, &a.wait, &a.debug_flags);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  cudaError_t e = timed(attn::kKBwdPre, s, [&] { return attn::launch_var_pre(a, s); });
  if (e != cudaSuccess) return cuda_fail(e, "attn_varlen_bwd preprocess launch");
  if (Tq > 0 && Tk > 0) {
    const int qrows = attn::bwd_q_rows(d);
    if ((rc = encode_packed(&a.tm_q, q, Tq, Hq, d, q_stride, 1, qrows, bf16)) ||
        (rc = encode_packed(&a.tm_k, k, Tk, Hkv, d, k_stride, 1, 128, bf16)) ||
        (rc = encode_packed(&a.tm_v, v, Tk, Hkv, d, v_stride, 1, 128, bf16)) ||
        (rc = encode_packed(&a.tm_do, dO, Tq, Hq, d, hq, 1, qrows, bf16)) ||
        (rc = encode_packed(&a.tm_dk, dk, Tk, Hkv, d, hk, 1, 128, bf16)) ||
        (rc = encode_packed(&a.tm_dv, dv, Tk, Hkv, d, hk, 1, 128, bf16)))
      return rc;
    e = timed(attn::kKBwdMain, s, [&] { return attn::launch_bwd_main_varlen(a, s); });
    if (e != cudaSuccess) return cuda_fail(e, "attn_varlen_bwd main launch");
  }
  if (Tq > 0) {
    e = timed(attn::kKDqPost, s, [&] { return attn::launch_var_post(a, s); });
    if (e != cudaSuccess) return cuda_fail(e, "attn_varlen_bwd dQ conversion launch");
  }
  return ATTN_OK;
}

int attn_status(void* stream) {
  t_err.clear();
  DeviceInfo* dev = nullptr;
  int rc = current_device(&dev);
  if (rc) return rc;
  cudaError_t e = cudaStreamSynchronize(static_cast<cudaStream_t>(stream));
  if (e != cudaSuccess) return cuda_fail(e, "cudaStreamSynchronize");
  int h = 0;
  if ((e = cudaMemcpyFromSymbol(&h, g_attn_status, sizeof h)) != cudaSuccess)
    return cuda_fail(e, "read status word");
  if (h != 0) {
    const int zero = 0;
    if ((e = cudaMemcpyToSymbol(g_attn_status, &zero, sizeof zero)) != cudaSuccess)
      return cuda_fail(e, "clear status word");
    return fail(ATTN_ERR_TIMEOUT, "a device-side wait ran out of time (status %d)", h);
  }
  return ATTN_OK;
}

int attn_profile_begin(void) {
  std::lock_guard<std::mutex> lk(g_prof_mu);
  if (g_prof.pool.empty()) {
    g_prof.pool.resize(2 * kProfPairs);
    for (auto& ev : g_prof.pool) {
      cudaError_t e = cudaEventCreate(&ev);
      if (e != cudaSuccess) {
        g_prof.pool.clear();
        return cuda_fail(e, "cudaEventCreate");
      }
    }
  }
  g_prof.used = 0;
  g_prof.kind.clear();
  g_prof.on = true;
  return ATTN_OK;
}

int attn_profile_end(int* launches, double* total_ms, int n) {
  std::lock_guard<std::mutex> lk(g_prof_mu);
  g_prof.on = false;
  const int m = n < attn::kKNum ? n : attn::kKNum;
  for (int i = 0; i < m; ++i) {
    if (launches) launches[i] = 0;
    if (total_ms) total_ms[i] = 0.0;
  }
  for (size_t i = 0; i < g_prof.kind.size(); ++i) {
    cudaEvent_t e0 = g_prof.pool[2 * i], e1 = g_prof.pool[2 * i + 1];
    cudaError_t e = cudaEventSynchronize(e1);
    if (e != cudaSuccess) return cuda_fail(e, "cudaEventSynchronize");
    float ms = 0.f;
    if ((e = cudaEventElapsedTime(&ms, e0, e1)) != cudaSuccess) return cuda_fail(e, "cudaEventElapsedTime");
    const int k = g_prof.kind[i];
    if (k < m) {
      if (launches) launches[k] += 1;
      if (total_ms) total_ms[k] += ms;
    }
  }
  g_prof.kind.clear();
  g_prof.used = 0;
  return m;
}

}  // extern "C"
