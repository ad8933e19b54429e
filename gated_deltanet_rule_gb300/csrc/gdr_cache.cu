// Pages of a key/value cache shared by rows: fork, reserve, free and the move of an accepted path.
//
// The page table and the reference counts are the whole state: a page is free when its count is 0,
// and pages are handed out lowest first to rows in order, so every call's result is a function of
// its inputs alone (counts change by integer atomics, whose order does not matter).
//
// A fork, reserve or free call runs up to three small kernels: release (one block a row: checks the
// row, returns its pages, says how many it needs), alloc (one block: the rows' needs as running sums,
// then the free pages in ascending order), and take (fork: shares the source's full pages and copies
// the partly filled one; reserve: enters the new pages). Copies are bound by HBM or, for few rows,
// by the three launches.
#include <cuda_runtime.h>

#include "gdr_serve.h"
#include "ptx.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr int kAllocThreads = 1024;

// Workspace: per listed row its need (-1: refused) and its place in the list of new pages, then the
// number of new pages found, then the list.
__device__ __forceinline__ int32_t* ws_need(const CacheArgs& a) { return a.ws; }
__device__ __forceinline__ int32_t* ws_first(const CacheArgs& a) { return a.ws + a.F; }
__device__ __forceinline__ int32_t* ws_found(const CacheArgs& a) { return a.ws + 2 * (size_t)a.F; }
__device__ __forceinline__ int32_t* ws_list(const CacheArgs& a) { return a.ws + 2 * (size_t)a.F + 4; }

enum Mode { kFork = 0, kReserve = 1, kFree = 2 };

// One block per listed row. A row is refused (untouched, kErrDeviceIndex) when its index or its
// source's is out of range, when an earlier entry lists it too, when a fork's source is itself a
// forked row, or when the context (the source's in a fork; not looked at by free), a page that it needs
// or a page that the row holds is out of range.
template <int kMode>
__global__ void __launch_bounds__(kThreads) release_kernel(const CacheArgs a) {
  __shared__ int s_have;
  const int f = blockIdx.x, tid = threadIdx.x;
  const int dst = __ldg(a.dst + f), src = kMode == kFork ? __ldg(a.src + f) : dst;
  bool bad = dst < 0 || dst >= a.rows || src < 0 || src >= a.rows;
  int n = 0, pages = 0, need = 0;
  // (a row that another entry lists may be released under these reads: it is refused whatever they see)
  if (!bad) {
    for (int g = tid; g < a.F; g += kThreads) {
      const int other = __ldg(a.dst + g);
      bad |= (g < f && other == dst) || (kMode == kFork && other == src);
    }
    const int32_t* held = a.table + (size_t)dst * a.M;
    if (kMode != kReserve)   // a page that is none cannot be given back
      for (int m = tid; m < a.M; m += kThreads) bad |= held[m] >= a.P;
    if (kMode != kFree) {
      n = a.ctx[src];
      const long long end = (long long)n + (kMode == kReserve ? a.extra : 0);
      if (n < 0 || end > (long long)a.M * a.page) {
        bad = true;
      } else if (kMode == kFork) {
        const int32_t* from = a.table + (size_t)src * a.M;
        pages = (int)((end + a.page - 1) / a.page);
        for (int m = tid; m < pages; m += kThreads) bad |= from[m] < 0 || from[m] >= a.P;
      } else {
        // pages held: the leading entries. The entry before the first empty one says how many; a page right
        // behind an empty entry, wherever it lies, says that they do not lie together (the row is refused)
        pages = (int)((end + a.page - 1) / a.page);
        for (int m = tid; m < a.M; m += kThreads) {
          const int e = held[m], after = m + 1 < a.M ? held[m + 1] : -1;
          bad |= e >= a.P || (e < 0 && after >= 0);
          if (e >= 0 && after < 0) s_have = m + 1;
          if (e < 0 && m == 0) s_have = 0;
        }
      }
    }
  }
  bad = __syncthreads_or(bad);
  if (!bad && kMode == kFork) need = n % a.page ? 1 : 0;
  if (!bad && kMode == kReserve) {
    const int have = s_have;
    need = pages > have ? pages - have : 0;
    bad = (long long)have * a.page < n;   // pages of the context that never were there
  }
  if (bad) {
    if (tid == 0) {
      atomicCAS(a.err, 0, kErrDeviceIndex);
      if (kMode != kFree) ws_need(a)[f] = -1;
    }
    return;
  }
  if (kMode != kReserve) {   // give back what the row holds
    int32_t* row = a.table + (size_t)dst * a.M;
    for (int m = tid; m < a.M; m += kThreads) {
      const int e = row[m];
      if (e >= 0) atomicSub(a.refs + e, 1);
      row[m] = -1;
    }
    if (tid == 0) a.ctx[dst] = 0;
  }
  if (tid == 0 && kMode != kFree) ws_need(a)[f] = need;
}

// Running sum over a block of kAllocThreads: returns the sum before this thread's value, and the total.
__device__ __forceinline__ int block_scan(int v, int* warp_sums, int& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int incl = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const int up = __shfl_up_sync(0xffffffffu, incl, m);
    if (lane >= m) incl += up;
  }
  if (lane == 31) warp_sums[warp] = incl;
  __syncthreads();
  if (warp == 0) {
    int w = warp_sums[lane];
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
      const int up = __shfl_up_sync(0xffffffffu, w, m);
      if (lane >= m) w += up;
    }
    warp_sums[lane] = w;
  }
  __syncthreads();
  total = warp_sums[31];
  const int before = (warp ? warp_sums[warp - 1] : 0) + incl - v;
  __syncthreads();   // warp_sums may be written again
  return before;
}

__global__ void __launch_bounds__(kAllocThreads) alloc_kernel(const CacheArgs a) {
  __shared__ int sums[32];
  ptx::wait_prerequisite();
  int wanted = 0;
  for (int f0 = 0; f0 < a.F; f0 += kAllocThreads) {
    const int f = f0 + (int)threadIdx.x;
    const int need = f < a.F ? ws_need(a)[f] : 0;
    int total;
    const int before = block_scan(need > 0 ? need : 0, sums, total);
    if (f < a.F) ws_first(a)[f] = wanted + before;
    wanted += total;
  }
  int found = 0;
  for (long long p0 = 0; p0 < a.P && found < wanted; p0 += kAllocThreads * 4) {   // (P may be up to 2^31 - 1)
    const long long p = p0 + (int)threadIdx.x * 4;
    int free4 = 0, count = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (p + e < a.P && a.refs[p + e] == 0) {
        free4 |= 1 << e;
        ++count;
      }
    int total;
    int at = found + block_scan(count, sums, total);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (free4 >> e & 1) {
        if (at < wanted) ws_list(a)[at] = (int)p + e;
        ++at;
      }
    found += total;
  }
  if (threadIdx.x == 0) *ws_found(a) = found < wanted ? found : wanted;
}

// Grid (row, share of the copy). A row whose pages were not all found is left empty with an error.
__global__ void __launch_bounds__(kThreads) fork_take_kernel(const CacheArgs a, int shares) {
  ptx::wait_prerequisite();
  const int f = blockIdx.x, tid = threadIdx.x;
  const int need = ws_need(a)[f];
  if (need < 0) return;
  const int first = ws_first(a)[f];
  if (need > 0 && first + need > *ws_found(a)) {
    if (tid == 0) atomicCAS(a.err, 0, kErrNoPages);
    return;
  }
  const int src = a.src[f], dst = a.dst[f], n = a.ctx[src];
  const int full = n >> a.page_shift, part = n & (a.page - 1);
  const int32_t* from = a.table + (size_t)src * a.M;
  const int fresh = need ? ws_list(a)[first] : -1;
  if (blockIdx.y == 0 && blockIdx.z == 0) {
    int32_t* to = a.table + (size_t)dst * a.M;
    for (int m = tid; m < full; m += kThreads) {
      const int e = from[m];
      to[m] = e;
      atomicAdd(a.refs + e, 1);
    }
    if (tid == 0) {
      if (need) {
        to[full] = fresh;
        atomicAdd(a.refs + fresh, 1);
      }
      a.ctx[dst] = n;
    }
  }
  if (!need) return;
  // the partly filled page: part positions of one layer's keys or values, contiguous
  const int layer = blockIdx.y >> 1;
  uint8_t* cache = (blockIdx.y & 1) ? a.v_cache : a.k_cache;
  const size_t page_bytes = (size_t)a.page * a.row_bytes;
  uint8_t* base = cache + (size_t)layer * a.P * page_bytes;
  const uint4* s = reinterpret_cast<const uint4*>(base + (size_t)from[full] * page_bytes);
  uint4* d = reinterpret_cast<uint4*>(base + (size_t)fresh * page_bytes);
  const long long vecs = (long long)part * a.row_bytes / 16, step = (long long)shares * kThreads;
  constexpr int kFlight = 8;
  for (long long i = (long long)blockIdx.z * kThreads + tid; i < vecs; i += kFlight * step) {
    uint4 x[kFlight];
#pragma unroll
    for (int e = 0; e < kFlight; ++e)
      if (i + e * step < vecs) x[e] = s[i + e * step];
#pragma unroll
    for (int e = 0; e < kFlight; ++e)
      if (i + e * step < vecs) d[i + e * step] = x[e];
  }
}

__global__ void __launch_bounds__(kThreads) reserve_take_kernel(const CacheArgs a) {
  ptx::wait_prerequisite();
  const int f = blockIdx.x, tid = threadIdx.x;
  const int need = ws_need(a)[f];
  if (need <= 0) return;
  const int first = ws_first(a)[f];
  if (first + need > *ws_found(a)) {
    if (tid == 0) atomicCAS(a.err, 0, kErrNoPages);
    return;
  }
  const int dst = a.dst[f];
  const int pages = (int)(((long long)a.ctx[dst] + a.extra + a.page - 1) / a.page);
  int32_t* to = a.table + (size_t)dst * a.M + (pages - need);
  for (int m = tid; m < need; m += kThreads) {
    const int e = ws_list(a)[first + m];
    to[m] = e;
    atomicAdd(a.refs + e, 1);
  }
}

// Moves the entries of an accepted path to the front: position ctx + path[i] to ctx + i, in every
// layer's keys and values. path rises and path[i] >= i, so a thread that walks i upwards over its own
// 16 bytes of every entry reads each position before it is written, in place and without a barrier.
__global__ void __launch_bounds__(kThreads) compact_kernel(const CompactArgs a) {
  extern __shared__ long long slots[];   // from [W], to [W]
  __shared__ int first_move;
  const int b = blockIdx.x, tid = threadIdx.x;
  const int n = __ldg(a.n_path + b), ctx = __ldg(a.ctx + b), shift = __ffs(a.page) - 1;
  const int32_t* path = a.path + (size_t)b * a.W;
  const int32_t* table = a.table + (size_t)b * a.M;
  // (few moves are bound by the latency of dependent reads: the path's do not wait for its length)
  const int node0 = tid < a.W ? __ldg(path + tid) : 0, before0 = tid > 0 && tid <= a.W ? __ldg(path + tid - 1) : -1;
  bool bad = n < 0 || n > a.W || ctx < 0;
  if (tid == 0) first_move = a.W;
  __syncthreads();
  if (!bad) {
    for (int i = tid; i < n; i += kThreads) {
      const int node = i == tid ? node0 : __ldg(path + i), before = i == tid ? before0 : __ldg(path + i - 1);
      const long long from = (long long)ctx + node, to = (long long)ctx + i;
      // to's page too has to be there: from's are checked below to rise through it
      bool off = node <= before || node < i || from >= (long long)a.M * a.page;
      if (!off) {
        const int pf = __ldg(table + (from >> shift)), pt = __ldg(table + (to >> shift));
        off = pf < 0 || pf >= a.P || pt < 0 || pt >= a.P;
        slots[i] = (long long)pf * a.page + (from & (a.page - 1));
        slots[a.W + i] = (long long)pt * a.page + (to & (a.page - 1));
      }
      bad |= off;
      if (node != i) atomicMin(&first_move, i);
    }
  }
  bad = __syncthreads_or(bad);
  if (tid == 0 && blockIdx.y == 0) {
    a.new_ctx[b] = bad ? ctx : ctx + n;
    if (bad) atomicCAS(a.err, 0, kErrDeviceIndex);
  }
  if (bad) return;
  const int vecs = (int)(a.row_bytes / 16);
  const long long cols = (long long)a.layers * 2 * vecs;
  const size_t page_vecs = (size_t)a.page * vecs;
  for (long long col = (long long)blockIdx.y * kThreads + tid; col < cols; col += (long long)gridDim.y * kThreads) {
    const int part = (int)(col / vecs), v = (int)(col - (long long)part * vecs);   // layer and side, vector
    uint4* base = reinterpret_cast<uint4*>((part & 1) ? a.v_cache : a.k_cache) + (size_t)(part >> 1) * a.P * page_vecs + v;
    for (int i = first_move; i < n; i += 8) {
      uint4 x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i + e < n) x[e] = base[(size_t)slots[i + e] * vecs];
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (i + e < n) base[(size_t)slots[a.W + i + e] * vecs] = x[e];
    }
  }
}

// Launch as a programmatic dependent of the kernel before it on the stream: its blocks may be placed
// before that kernel has ended and wait for it on the device.
template <typename... KArgs, typename... Args>
cudaError_t launch_after(void (*kernel)(KArgs...), dim3 grid, int threads, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(threads);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

size_t cache_workspace_bytes(int F, int M) {
  // need and first of each row, the count, and at most M new pages a row
  return ((size_t)F * 2 + 4 + (size_t)F * M) * sizeof(int32_t);
}

cudaError_t launch_cache_fork(const CacheArgs& a, cudaStream_t s) {
  int slot = stage_timer_begin(s, kKernCacheAlloc);
  release_kernel<kFork><<<a.F, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_after(alloc_kernel, dim3(1), kAllocThreads, s, a);
  stage_timer_end(slot, s);
  if (e != cudaSuccess) return e;
  // blocks of a copy: one, or as many as bring the launch to eight blocks a SM (32 KiB a pass and block:
  // a block's start costs as much as copying a few KiB)
  const long long vecs = (long long)a.page * a.row_bytes / 16, copies = 2ll * a.layers * a.F;
  long long shares = (kNumSMs * 8 + copies - 1) / copies;
  const long long most = (vecs + kThreads - 1) / kThreads;
  if (shares > most) shares = most;
  if (shares > 64) shares = 64;
  slot = stage_timer_begin(s, kKernCacheCopy);
  e = launch_after(fork_take_kernel, dim3(a.F, 2 * a.layers, (unsigned)shares), kThreads, s, a, (int)shares);
  stage_timer_end(slot, s);
  return e;
}

cudaError_t launch_cache_reserve(const CacheArgs& a, cudaStream_t s) {
  const int slot = stage_timer_begin(s, kKernCacheAlloc);
  release_kernel<kReserve><<<a.F, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) e = launch_after(alloc_kernel, dim3(1), kAllocThreads, s, a);
  if (e == cudaSuccess) e = launch_after(reserve_take_kernel, dim3(a.F), kThreads, s, a);
  stage_timer_end(slot, s);
  return e;
}

cudaError_t launch_cache_free(const CacheArgs& a, cudaStream_t s) {
  const int slot = stage_timer_begin(s, kKernCacheAlloc);
  release_kernel<kFree><<<a.F, kThreads, 0, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  stage_timer_end(slot, s);
  return e;
}

cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t s) {
  const long long cols = (long long)a.layers * 2 * (a.row_bytes / 16);
  long long y = (cols + kThreads - 1) / kThreads;
  const long long most = (kNumSMs * 32 + a.B - 1) / a.B;   // a few waves in all
  if (y > most) y = most;
  const int slot = stage_timer_begin(s, kKernCacheCopy);
  compact_kernel<<<dim3(a.B, (unsigned)y), kThreads, (size_t)a.W * 2 * sizeof(long long), s>>>(a);
  const cudaError_t e = cudaGetLastError();
  stage_timer_end(slot, s);
  return e;
}

}  // namespace gdr
