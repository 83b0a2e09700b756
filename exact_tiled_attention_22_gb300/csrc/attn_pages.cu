// attn_pages.cu -- block tables and slot maps of a paged key/value cache,
// built on the GPU from request lengths.
//
// A request b holds len_b tokens in ceil(len_b / ps) pages of ps tokens, whose
// ids stand in row b of the block table.  The free pages are a stack.  With
// add_b new tokens the request needs
//   need_b = ceil((len_b + add_b) / ps) - ceil(len_b / ps)
// pages; with N_b = sum_{a <= b} need_a (inclusive) it is served iff
// need_b = 0 or N_b <= free, its k-th new page being the stack's entry
// free - 1 - (N_b - need_b + k), so every new entry and every slot
//   slot(t) = page(pos / ps) * ps + pos % ps,   pos = len_b + t - cu_b
// is a function of two prefix sums over the requests and needs no allocator
// loop.  The call moves a few kilobytes: its time is launch and the chain
// lengths -> prefix sums -> page id -> slot.  One cluster of up to eight
// CTAs: each CTA computes the prefix sums for itself (B values, from L2), then
// they share the tokens and table rows; the cluster barrier between the reads
// of the lengths and their update lets new_lens be lens and left be
// free_count.  Measured (graph replay): one token for each of 256 requests
// 4.8 us (four CTAs of 256 threads), 28005 tokens of 48 prompts 6.8 us (eight of
// 1024).  The release is one CTA: 5.8 us for 256 requests of up to 64 pages, an eighth of
// them finished, 15 for 1024, 97 for 8192 of up to 16.
#include <climits>

#include "kernels.h"
#include "sm103_ptx.cuh"

namespace attn {
namespace {

constexpr int kPgThreads = 1024;

// Exclusive prefix sums of x and y over the block's threads, added to the
// carries, which become the totals.  wx, wy: shared, NW warps.
template <int NW>
__device__ __forceinline__ void block_scan2(long long& x, long long& y, long long& cx, long long& cy, long long* wx,
                                            long long* wy) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long ix = x, iy = y;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long ax = __shfl_up_sync(0xffffffffu, ix, o), ay = __shfl_up_sync(0xffffffffu, iy, o);
    if (lane >= o) {
      ix += ax;
      iy += ay;
    }
  }
  if (lane == 31) {
    wx[warp] = ix;
    wy[warp] = iy;
  }
  __syncthreads();
  long long bx = 0, by = 0, tx = 0, ty = 0;
  {
    const long long vx = lane < NW ? wx[lane] : 0, vy = lane < NW ? wy[lane] : 0;
    long long sx = vx, sy = vy;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const long long ax = __shfl_up_sync(0xffffffffu, sx, o), ay = __shfl_up_sync(0xffffffffu, sy, o);
      if (lane >= o) {
        sx += ax;
        sy += ay;
      }
    }
    tx = __shfl_sync(0xffffffffu, sx, 31);
    ty = __shfl_sync(0xffffffffu, sy, 31);
    bx = __shfl_sync(0xffffffffu, sx - vx, warp);
    by = __shfl_sync(0xffffffffu, sy - vy, warp);
  }
  x = cx + bx + ix - x;
  y = cy + by + iy - y;
  cx += tx;
  cy += ty;
  __syncthreads();
}

__device__ __forceinline__ void cluster_sync_all() {
  asm volatile("barrier.cluster.arrive.aligned;\n\tbarrier.cluster.wait.aligned;" ::: "memory");
}

// Per request, in shared memory: cu (exclusive sum of the new tokens), the
// stack offset of its first new page (-1: not served) and its old length.
struct PageReq {
  int cu, off, len;
};

template <int NT>
__global__ void __launch_bounds__(NT, 1) attn_pages_extend_kernel(const __grid_constant__ PagesArgs p) {
  constexpr int NW = NT / 32;
  extern __shared__ __align__(16) uint8_t pg_smem[];
  PageReq* req = reinterpret_cast<PageReq*>(pg_smem);
  __shared__ long long wx[NW], wy[NW];
  griddep_wait();
  const int ps = 1 << p.page_shift;
  const int n_cta = gridDim.x, cta = blockIdx.x;
  const int count = min(max(*p.free_count, 0), p.free_cap);
  long long c_need = 0, c_add = 0;
  for (int b0 = 0; b0 < p.B; b0 += NT) {
    const int b = b0 + threadIdx.x;
    int len = 0, add = 0;
    if (b < p.B) {
      len = p.lens[b];
      add = p.add[b];
    }
    const long long end = (long long)len + add;
    const bool valid = len >= 0 && add >= 0 && end <= (long long)p.width << p.page_shift;
    const int p_old = valid ? (int)(((long long)len + ps - 1) >> p.page_shift) : 0;
    const long long need = valid ? ((end + ps - 1) >> p.page_shift) - p_old : 0;
    long long sn = need, sa = add > 0 ? add : 0;
    block_scan2<NW>(sn, sa, c_need, c_add, wx, wy);
    const bool served = valid && b < p.B && (need == 0 || sn + need <= count);
    if (b < p.B) {
      const int cu = (int)min(sa, (long long)INT_MAX);
      req[b] = PageReq{cu, served ? (need == 0 ? 0 : (int)sn) : -1, len};
    }
  }
  const int total = (int)min(c_add, (long long)INT_MAX);
  __syncthreads();

  // Block table rows: a warp per request.
  const int lane = threadIdx.x & 31;
  const int gw = (cta * NT + (int)threadIdx.x) >> 5, n_gw = n_cta * NW;
  for (int b = gw; b < p.B; b += n_gw) {
    const PageReq r = req[b];
    if (r.off < 0) continue;
    const int add = p.add[b];
    const int j0 = (int)(((long long)r.len + ps - 1) >> p.page_shift);
    const int j1 = (int)(((long long)r.len + add + ps - 1) >> p.page_shift);
    int* row = p.table + (size_t)b * p.width;
    for (int j = j0 + lane; j < j1; j += 32) row[j] = p.free_pages[count - 1 - (r.off + (j - j0))];
  }
  // Slots: a thread per new token; its request by bisection of cu.
  for (long long t = (long long)cta * NT + threadIdx.x; t < p.T; t += (long long)n_cta * NT) {
    long long slot = -1;
    if (t < total) {
      int lo = 0, hi = p.B - 1;  // last request with cu <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (req[mid].cu <= t) lo = mid; else hi = mid - 1;
      }
      const PageReq r = req[lo];
      if (r.off >= 0) {
        const long long pos = (long long)r.len + (t - r.cu);
        const int j = (int)(pos >> p.page_shift), j0 = (int)(((long long)r.len + ps - 1) >> p.page_shift);
        const int page = j < j0 ? p.table[(size_t)lo * p.width + j] : p.free_pages[count - 1 - (r.off + (j - j0))];
        if (page >= 0) slot = ((long long)page << p.page_shift) + (pos & (ps - 1));
      }
    }
    p.slots[t] = slot;
  }
  // Lengths: every CTA has read them by the cluster barrier, so they may be
  // updated in place.
  cluster_sync_all();
  if (cta == 0) {
    long long taken = 0;
    for (int b = threadIdx.x; b < p.B; b += NT) {
      const PageReq r = req[b];
      const int add = p.add[b];
      const int g = r.off >= 0 ? add : 0;
      p.granted[b] = g;
      p.new_lens[b] = r.len + g;
      p.cu_new[b] = r.cu;
      if (r.off >= 0) {
        const long long need = (((long long)r.len + add + ps - 1) >> p.page_shift) - (((long long)r.len + ps - 1) >> p.page_shift);
        if (need > 0) taken = max(taken, r.off + need);
      }
    }
    // Pages taken: the served needs are a prefix of all of them (a refused
    // request's inclusive sum is above the count, and so is every later one
    // that needs a page), so it is the largest served inclusive sum.
    __shared__ long long most[NW];
    for (int o = 16; o > 0; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
    if (lane == 0) most[threadIdx.x >> 5] = taken;
    __syncthreads();
    if (threadIdx.x < 32) {
      long long v = threadIdx.x < NW ? most[threadIdx.x] : 0;
      for (int o = 16; o > 0; o >>= 1) v = max(v, __shfl_xor_sync(0xffffffffu, v, o));
      if (threadIdx.x == 0) {
        p.cu_new[p.B] = total;
        *p.left = count - (int)v;
      }
    }
  }
  griddep_launch_dependents();
}

// Pages of the finished requests go back on the stack, in the order of the
// requests and of their pages; their lengths become 0.  One CTA.
__global__ void __launch_bounds__(kPgThreads, 1) attn_pages_release_kernel(const __grid_constant__ PagesArgs p) {
  constexpr int NW = kPgThreads / 32;
  extern __shared__ __align__(16) uint8_t pg_smem[];
  int* off = reinterpret_cast<int*>(pg_smem);  // [B] stack offset of the request's first page, -1: kept
  __shared__ long long wx[NW], wy[NW];
  griddep_wait();
  const int ps = 1 << p.page_shift, lane = threadIdx.x & 31;
  const int count = min(max(*p.free_count, 0), p.free_cap);
  long long c_n = 0, c_z = 0;
  for (int b0 = 0; b0 < p.B; b0 += kPgThreads) {
    const int b = b0 + threadIdx.x;
    long long n = 0, z = 0;
    bool gone = false;
    if (b < p.B) {
      const int len = p.lens[b];
      gone = p.add[b] != 0;
      if (gone && len > 0) n = min(((long long)len + ps - 1) >> p.page_shift, (long long)p.width);
    }
    const long long own = n;
    block_scan2<NW>(n, z, c_n, c_z, wx, wy);
    if (b < p.B) off[b] = gone && own > 0 ? (int)min(n, (long long)INT_MAX) : -1;
  }
  __syncthreads();
  for (int b = threadIdx.x >> 5; b < p.B; b += NW) {
    if (off[b] < 0) continue;
    const int n = (int)min(((long long)p.lens[b] + ps - 1) >> p.page_shift, (long long)p.width);
    const int* row = p.table + (size_t)b * p.width;
    for (int j = lane; j < n; j += 32) {
      const long long at = (long long)count + off[b] + j;
      if (at < p.free_cap) p.free_out[at] = row[j];
    }
  }
  __syncthreads();
  for (int b = threadIdx.x; b < p.B; b += kPgThreads) p.new_lens[b] = p.add[b] != 0 ? 0 : p.lens[b];
  if (threadIdx.x == 0) *p.left = (int)min((long long)count + c_n, (long long)p.free_cap);
  griddep_launch_dependents();
}

}  // namespace

template <int NT>
static cudaError_t launch_extend_t(const PagesArgs& a, cudaStream_t stream) {
  auto* k = attn_pages_extend_kernel<NT>;
  const size_t smem = sizeof(PageReq) * (size_t)a.B;
  if (smem > 40 * 1024) {  // (48 KB, the static part included, need no attribute)
    const cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(PageReq) * kPagesMaxB);
    if (e != cudaSuccess) return e;
  }
  // a thread to a token and four to a request: one CTA up to 64 requests' decoding step,
  // four for 256 requests', up to eight (a portable cluster) for prompts
  const long long want = ((a.T > 4ll * a.B ? (long long)a.T : 4ll * a.B) + NT - 1) / NT;
  const unsigned n = (unsigned)(want >= 8 ? 8 : (want >= 4 ? 4 : (want >= 2 ? 2 : 1)));
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(n);
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = n;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, k, a);
}

// Blocks of 256 threads while they take one look at the requests and four at the
// tokens (a token for each of 256 requests: 4.8 us, 5.7 with 1024 threads, whose
// scans and barriers are longer), of 1024 above (28005 tokens of 48 prompts: 6.8 us, 9.7
// with 256).
cudaError_t launch_pages_extend(const PagesArgs& a, cudaStream_t stream) {
  return a.B <= 256 && a.T <= 1024 ? launch_extend_t<256>(a, stream) : launch_extend_t<kPgThreads>(a, stream);
}

cudaError_t launch_pages_release(const PagesArgs& a, cudaStream_t stream) {
  auto* k = attn_pages_release_kernel;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, sizeof(PageReq) * kPagesMaxB);
  if (e != cudaSuccess) return e;
  return launch_pdl(k, 1, kPgThreads, 4 * (size_t)a.B, stream, a);
}

}  // namespace attn
