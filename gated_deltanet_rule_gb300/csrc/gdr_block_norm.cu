// What stands between two blocks of a layer, in one pass over a row (token) of C channels:
//   z = post_w y / sqrt(mean(y^2) + eps)  (or z = y),   x = h + scale sigmoid(gate) z,
//   h_out = x,   n_out = pre_w x / sqrt(mean(x^2) + eps)
// and its gradient. With g = sigmoid(gate), r = 1 / sqrt(mean(y^2) + eps), s = 1 / sqrt(mean(x^2) + eps):
//   dx = dh_out + s (pre_w dn - x s^2 mean(pre_w dn x)),     dpre_w = sum over rows of dn x s,
//   dh = dx,   dscale = sum dx g z,   dgate = dx scale z g (1 - g),   dz = dx scale g,
//   dpost_w = sum dz y r,   dy = r (post_w dz - y r^2 mean(post_w dz y))  (or dz).
//
// Both are bound by HBM. A block takes a row at a time, a thread 8 neighbouring channels of it (16 bytes of
// bfloat16), so that a row stays in registers from its one reading to its writing; the weights of a
// thread's channels are read once and kept. The next row is on its way while this one is reduced.
//
// The gradient's three sums of a row follow one another (mean(y^2) gives x, x gives dx, dx gives dz), but the
// last is linear in dx: with p = post_w scale g it is
//   sum(p dx y) = sum(p y dh_out) + s sum(p y pre_w dn) - s^3 mean(pre_w dn x) sum(p y x),
// so all but mean(y^2) are taken at once, and a row costs two exchanges instead of three. Sums of the
// weights' gradients stay with the thread that owns the channel (in registers, for more than kWideC
// channels in shared memory), leave as one partial row a block and are summed in order by a second kernel: no
// atomics, the same bits every time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdr_serve.h"
#include "ptx.cuh"

namespace gdr {
namespace {

using bf16 = __nv_bfloat16;
constexpr int kMaxThreads = 512;   // of a block; 8 channels a thread
constexpr int kWideC = 8 * kMaxThreads;
constexpr unsigned kAll = 0xffffffffu;

// 8 channels as they lie in memory
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];
};
__device__ __forceinline__ uint4 stream16(const void* p) {   // read once: nothing for L1 to keep
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
template <typename T>
__device__ __forceinline__ Raw<T> load(const T* p) {
  Raw<T> r;
#pragma unroll
  for (int k = 0; k < (int)(sizeof(T) / 2); ++k) r.v[k] = stream16(reinterpret_cast<const uint4*>(p) + k);
  return r;
}
__device__ __forceinline__ void widen(const Raw<bf16>& r, float* x) {
  const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    x[2 * e] = __uint_as_float(u[e] << 16);
    x[2 * e + 1] = __uint_as_float(u[e] & 0xFFFF0000u);
  }
}
__device__ __forceinline__ void widen(const Raw<float>& r, float* x) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    x[4 * k] = __uint_as_float(r.v[k].x);
    x[4 * k + 1] = __uint_as_float(r.v[k].y);
    x[4 * k + 2] = __uint_as_float(r.v[k].z);
    x[4 * k + 3] = __uint_as_float(r.v[k].w);
  }
}
__device__ __forceinline__ void store(bf16* p, const float* x) {
  *reinterpret_cast<uint4*>(p) = make_uint4(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]),
                                            ptx::pack_bf16x2(x[4], x[5]), ptx::pack_bf16x2(x[6], x[7]));
}
__device__ __forceinline__ void store(float* p, const float* x) {
  reinterpret_cast<float4*>(p)[0] = make_float4(x[0], x[1], x[2], x[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(x[4], x[5], x[6], x[7]);
}
__device__ __forceinline__ void weight8(const float* w, int c, float* x) {   // NULL: ones
  if (!w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) x[e] = 1.f;
    return;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(w + c) + k);
    x[4 * k] = v.x; x[4 * k + 1] = v.y; x[4 * k + 2] = v.z; x[4 * k + 3] = v.w;
  }
}
__device__ __forceinline__ float sigmoid(float x) { return __fdividef(1.f, 1.f + __expf(-x)); }   // (2 ulp; 0 where e^-x is infinite)

// A thread's 16-byte units of the rows to come, in shared memory: a ring of `stages` rows of `parts` units each, every
// unit copied (asynchronously) and read by the same thread, so that rows on their way cost neither registers nor
// barriers. Without stages (rows too wide for two of them) a row is read when it is needed.
struct Ring {
  uint4* mine;      // unit u of stage s at (s parts + u) blockDim.x
  int stages, parts, slot;
  __device__ __forceinline__ uint4* at(int u) const { return mine + (slot * parts + u) * blockDim.x; }
  __device__ __forceinline__ void wait() const {   // for the oldest row
    if (stages >= 4) ptx::cp_async_wait<3>();
    else if (stages == 3) ptx::cp_async_wait<2>();
    else if (stages == 2) ptx::cp_async_wait<1>();
  }
  __device__ __forceinline__ void next() { slot = slot + 1 == stages ? 0 : slot + 1; }
};
template <typename T>
__device__ __forceinline__ void copy(const Ring& g, int u, const T* p) {
#pragma unroll
  for (int j = 0; j < (int)(sizeof(T) / 2); ++j) ptx::cp_async16_zfill(g.at(u + j), reinterpret_cast<const uint4*>(p) + j, 16);
}
template <typename T>
__device__ __forceinline__ Raw<T> take(const Ring& g, int u, const T* p) {
  if (g.stages == 0) return load(p);
  Raw<T> r;
#pragma unroll
  for (int j = 0; j < (int)(sizeof(T) / 2); ++j) r.v[j] = *g.at(u + j);
  return r;
}

// Sums of n values over the block, the same in every thread. red holds 0 where there is no warp; a place of it is
// written again only after another barrier.
template <int n>
__device__ __forceinline__ void block_sum(float (&v)[n], float (*red)[16]) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) v[i] += __shfl_xor_sync(kAll, v[i], m);
  if (blockDim.x == 32) return;
  if ((threadIdx.x & 31) == 0)
#pragma unroll
    for (int i = 0; i < n; ++i) red[i][threadIdx.x >> 5] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < n; ++i) {
    float4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = reinterpret_cast<const float4*>(red[i])[j];
    v[i] = ((x[0].x + x[0].y) + (x[0].z + x[0].w)) + ((x[1].x + x[1].y) + (x[1].z + x[1].w)) +
           (((x[2].x + x[2].y) + (x[2].z + x[2].w)) + ((x[3].x + x[3].y) + (x[3].z + x[3].w)));
  }
}

// One row's vectors of a thread: k-th at channel 8 (threadIdx.x + k blockDim.x).
template <typename T, int K>
__global__ void __launch_bounds__(kMaxThreads, K == 1 ? 2 : 1) block_norm_kernel(const BlockNormArgs a) {
  constexpr int kPart = sizeof(T) / 2;   // units of 8 channels
  extern __shared__ __align__(16) uint4 dyn[];
  __shared__ __align__(16) float red[2][1][16];
  if (threadIdx.x < 32) red[threadIdx.x >> 4][0][threadIdx.x & 15] = 0.f;
  __syncthreads();
  const int C = a.C;
  const float inv_c = 1.f / (float)C;
  int at[K];
#pragma unroll
  for (int k = 0; k < K; ++k) at[k] = 8 * (threadIdx.x + k * blockDim.x);
  const T *h = static_cast<const T*>(a.h), *y = static_cast<const T*>(a.y), *gate = static_cast<const T*>(a.gate);
  Ring ring{dyn + threadIdx.x, a.stages, 3 * K * kPart, 0};
  auto fetch = [&](long long row) {   // into the ring's present slot
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C || row >= a.rows) continue;
      copy(ring, (3 * k) * kPart, y + row * a.y_row + at[k]);
      if (gate) copy(ring, (3 * k + 1) * kPart, gate + row * a.gate_row + at[k]);
      copy(ring, (3 * k + 2) * kPart, h + row * C + at[k]);
    }
    ptx::cp_async_commit();
    ring.next();
  };
  for (int i = 0; i < a.stages; ++i) fetch(blockIdx.x + (long long)i * gridDim.x);
  float w_pre[8], w_post[8], w_scale[8];   // (one vector a thread: kept)
  if (K == 1 && at[0] < C) {
    weight8(a.pre_w, at[0], w_pre);
    weight8(a.post_w, at[0], w_post);
    weight8(a.scale, at[0], w_scale);
  }
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    float x[K][8], z[K][8], g[K][8];
    ring.wait();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      widen(take(ring, (3 * k + 2) * kPart, h + row * C + at[k]), x[k]);
      widen(take(ring, (3 * k) * kPart, y + row * a.y_row + at[k]), z[k]);
      if (gate) widen(take(ring, (3 * k + 1) * kPart, gate + row * a.gate_row + at[k]), g[k]);
    }
    if (ring.stages) fetch(row + (long long)ring.stages * gridDim.x);
    float r = 1.f;
    if (a.post_w) {
      float s[1] = {0.f};
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (at[k] < C)
#pragma unroll
          for (int e = 0; e < 8; ++e) s[0] = fmaf(z[k][e], z[k][e], s[0]);
      block_sum(s, red[0]);
      r = rsqrtf(fmaf(s[0], inv_c, a.eps));
    }
    float s[1] = {0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      if (K > 1) {
        weight8(a.post_w, at[k], w_post);
        weight8(a.scale, at[k], w_scale);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float f = w_scale[e] * (z[k][e] * r * w_post[e]);
        if (gate) f *= sigmoid(g[k][e]);
        x[k][e] += f;
        s[0] = fmaf(x[k][e], x[k][e], s[0]);
      }
      store(static_cast<T*>(a.h_out) + row * C + at[k], x[k]);
    }
    block_sum(s, red[1]);
    r = rsqrtf(fmaf(s[0], inv_c, a.eps));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      if (K > 1) weight8(a.pre_w, at[k], w_pre);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[k][e] *= r * w_pre[e];
      store(static_cast<T*>(a.n_out) + row * C + at[k], x[k]);
    }
    if (!a.post_w) __syncthreads();   // red[1] is written again before another barrier
  }
}

// Sums of the weights' gradients of a thread's channels: in registers, or (more than one vector a thread) in
// shared memory at the thread's own places.
template <typename T, int K>
__global__ void __launch_bounds__(kMaxThreads, 1) block_norm_backward_kernel(const BlockNormArgs a) {
  constexpr int kPart = sizeof(T) / 2;
  extern __shared__ __align__(16) uint4 dyn[];
  __shared__ __align__(16) float red[2][5][16];
  if (threadIdx.x < 32)
#pragma unroll
    for (int i = 0; i < 5; ++i) red[threadIdx.x >> 4][i][threadIdx.x & 15] = 0.f;
  __syncthreads();
  const int C = a.C;
  const float inv_c = 1.f / (float)C;
  int at[K];
#pragma unroll
  for (int k = 0; k < K; ++k) at[k] = 8 * (threadIdx.x + k * blockDim.x);
  const T *h = static_cast<const T*>(a.h), *y = static_cast<const T*>(a.y), *gate = static_cast<const T*>(a.gate);
  const T* dn = static_cast<const T*>(a.dn);
  constexpr int kVec = 4 * kPart + 2;   // units of a thread's vector: y, gate, h, dn, dh_out
  Ring ring{dyn + threadIdx.x, a.stages, K * kVec, 0};
  float* acc_sm = reinterpret_cast<float*>(dyn + (size_t)a.stages * K * kVec * blockDim.x);   // (K > 1) [3][C]
  auto fetch = [&](long long row) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C || row >= a.rows) continue;
      copy(ring, k * kVec, y + row * a.y_row + at[k]);
      if (gate) copy(ring, k * kVec + kPart, gate + row * a.gate_row + at[k]);
      copy(ring, k * kVec + 2 * kPart, h + row * C + at[k]);
      copy(ring, k * kVec + 3 * kPart, dn + row * C + at[k]);
      if (a.dh_out) copy(ring, k * kVec + 4 * kPart, a.dh_out + row * C + at[k]);
    }
    ptx::cp_async_commit();
    ring.next();
  };
  for (int i = 0; i < a.stages; ++i) fetch(blockIdx.x + (long long)i * gridDim.x);
  float w_pre[8], w_post[8], w_scale[8], acc[3][8];
  if (K == 1 && at[0] < C) {
    weight8(a.pre_w, at[0], w_pre);
    weight8(a.post_w, at[0], w_post);
    weight8(a.scale, at[0], w_scale);
  }
#pragma unroll
  for (int i = 0; i < 3; ++i) {
#pragma unroll
    for (int e = 0; e < 8; ++e) acc[i][e] = 0.f;
    if (K > 1)
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (at[k] < C) store(acc_sm + i * C + at[k], acc[i]);
  }
  auto add = [&](int i, int k, const float* d) {
    if (K == 1) {
#pragma unroll
      for (int e = 0; e < 8; ++e) acc[i][e] += d[e];
    } else {
      float4* p = reinterpret_cast<float4*>(acc_sm + i * C + at[k]);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float4 v = p[j];
        v.x += d[4 * j]; v.y += d[4 * j + 1]; v.z += d[4 * j + 2]; v.w += d[4 * j + 3];
        p[j] = v;
      }
    }
  };
  for (long long row = blockIdx.x; row < a.rows; row += gridDim.x) {
    Raw<T> cy[K], cn[K];   // y and dn stay as they are, and are widened where they are used
    float x[K][8], g[K][8], dx[K][8];
    ring.wait();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      cy[k] = take(ring, k * kVec, y + row * a.y_row + at[k]);
      cn[k] = take(ring, k * kVec + 3 * kPart, dn + row * C + at[k]);
      widen(take(ring, k * kVec + 2 * kPart, h + row * C + at[k]), x[k]);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        g[k][e] = 1.f;
        dx[k][e] = 0.f;
      }
      if (gate) widen(take(ring, k * kVec + kPart, gate + row * a.gate_row + at[k]), g[k]);
      if (a.dh_out) widen(take(ring, k * kVec + 4 * kPart, a.dh_out + row * C + at[k]), dx[k]);
    }
    if (ring.stages) fetch(row + (long long)ring.stages * gridDim.x);
    float r = 1.f;
    if (a.post_w) {
      float s[1] = {0.f};
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (at[k] >= C) continue;
        float yv[8];
        widen(cy[k], yv);
#pragma unroll
        for (int e = 0; e < 8; ++e) s[0] = fmaf(yv[e], yv[e], s[0]);
      }
      block_sum(s, red[0]);
      r = rsqrtf(fmaf(s[0], inv_c, a.eps));
    }
    // sums of x^2, pre_w dn x, p y dh_out, p y pre_w dn, p y x
    float s[5] = {0.f, 0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      if (K > 1) {
        weight8(a.post_w, at[k], w_post);
        weight8(a.scale, at[k], w_scale);
        weight8(a.pre_w, at[k], w_pre);
      }
      float yv[8], dn8[8];
      widen(cy[k], yv);
      widen(cn[k], dn8);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (gate) g[k][e] = sigmoid(g[k][e]);
        const float py = w_scale[e] * g[k][e] * w_post[e] * yv[e], wdn = w_pre[e] * dn8[e];
        x[k][e] = fmaf(py, r, x[k][e]);
        s[0] = fmaf(x[k][e], x[k][e], s[0]);
        s[1] = fmaf(wdn, x[k][e], s[1]);
        s[2] = fmaf(py, dx[k][e], s[2]);
        s[3] = fmaf(py, wdn, s[3]);
        s[4] = fmaf(py, x[k][e], s[4]);
      }
    }
    block_sum(s, red[1]);
    const float q = rsqrtf(fmaf(s[0], inv_c, a.eps)), mx = s[1] * inv_c * q * q * q;
    const float my = a.post_w ? (s[2] + q * s[3] - mx * s[4]) * inv_c * r * r * r : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      if (K > 1) {
        weight8(a.post_w, at[k], w_post);
        weight8(a.scale, at[k], w_scale);
        weight8(a.pre_w, at[k], w_pre);
      }
      float yv[8], t[8];
      widen(cn[k], t);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float d = t[e];
        dx[k][e] += w_pre[e] * d * q - x[k][e] * mx;
        t[e] = d * x[k][e] * q;
      }
      store(a.dh + row * C + at[k], dx[k]);
      add(0, k, t);
      widen(cy[k], yv);
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = dx[k][e] * w_scale[e] * g[k][e] * yv[e] * r;   // dz y r
      if (a.post_w) add(1, k, t);
      if (gate) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] *= w_post[e] * (1.f - g[k][e]);
        store(static_cast<T*>(a.dgate) + row * C + at[k], t);
      }
      if (a.scale) {
#pragma unroll
        for (int e = 0; e < 8; ++e) t[e] = dx[k][e] * g[k][e] * yv[e] * r * w_post[e];
        add(2, k, t);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = dx[k][e] * w_scale[e] * g[k][e] * w_post[e] * r - yv[e] * my;
      store(static_cast<T*>(a.dy) + row * C + at[k], t);
    }
    if (!a.post_w) __syncthreads();   // red[1] is written again before another barrier
  }
  // the block's partial sums
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (at[k] >= C) continue;
    for (int i = 0; i < 3; ++i) {
      float t[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) t[e] = K == 1 ? acc[i][e] : acc_sm[i * C + at[k] + e];
      store(a.partial + ((size_t)blockIdx.x * 3 + i) * C + at[k], t);
    }
  }
}

// Sums of the blocks' partial rows, in order: a block 32 channels of one of the three, its 8 warps every 8th
// partial each.
constexpr int kSumWarps = 8;
__global__ void __launch_bounds__(32 * kSumWarps) block_norm_sum_kernel(const BlockNormArgs a, int blocks) {
  __shared__ float part[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.y, c = blockIdx.x * 32 + lane;
  float* out = i == 0 ? a.dpre_w : i == 1 ? a.dpost_w : a.dscale;
  ptx::wait_prerequisite();
  if (!out) return;
  float s = 0.f;
  if (c < a.C)
#pragma unroll 4
    for (int b = warp; b < blocks; b += kSumWarps) s += a.partial[((size_t)b * 3 + i) * a.C + c];
  part[warp][lane] = s;
  __syncthreads();
  if (warp > 0 || c >= a.C) return;
  s = 0.f;
#pragma unroll
  for (int w = 0; w < kSumWarps; ++w) s += part[w][lane];
  out[c] = s;
}

int threads_of(int C) { return std::min(kMaxThreads, (C / 8 + 31) / 32 * 32); }
int vectors_of(int C) { return (C / 8 + kMaxThreads - 1) / kMaxThreads; }
// Blocks of the gradient that a GPU holds: 512 threads an SM.
int backward_blocks(int C) { return kNumSMs * std::min(16, kMaxThreads / threads_of(C)); }
// Rows on their way to a block, of `per` on an SM: at most four, none where not even two fit.
constexpr int kSmemSM = 220 << 10;
int stages_of(int per, int bytes, int more) {
  const int n = std::min(4, (std::min(kSmemSM / per, 224 << 10) - 2048 - more) / bytes);
  return n < 2 ? 0 : n;
}

template <typename T, int K>
cudaError_t forward(BlockNormArgs a, cudaStream_t s) {
  const int t = threads_of(a.C), per = std::min(32, (K == 1 ? 2 : 1) * kMaxThreads / t);
  const int bytes = 3 * K * (int)(sizeof(T) / 2) * t * 16;
  a.stages = stages_of(per, bytes, 0);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(block_norm_kernel<T, K>), 224 << 10, done);
  if (e != cudaSuccess) return e;
  const int slot = stage_timer_begin(s, kKernBlockNorm);
  block_norm_kernel<T, K><<<(unsigned)std::min<long long>(a.rows, kNumSMs * per), t, a.stages * bytes, s>>>(a);
  stage_timer_end(slot, s);
  return cudaGetLastError();
}
template <typename T, int K>
cudaError_t backward(BlockNormArgs a, cudaStream_t s) {
  const int t = threads_of(a.C), blocks = (int)std::min<long long>(a.rows, backward_blocks(a.C));
  const int bytes = K * (4 * (int)(sizeof(T) / 2) + 2) * t * 16, more = K == 1 ? 0 : 3 * a.C * 4;
  a.stages = stages_of(std::min(16, kMaxThreads / t), bytes, more);
  const int smem = a.stages * bytes + more;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(block_norm_backward_kernel<T, K>), 224 << 10, done);
  if (e != cudaSuccess) return e;
  int slot = stage_timer_begin(s, kKernBlockNormBwd);
  block_norm_backward_kernel<T, K><<<blocks, t, smem, s>>>(a);
  stage_timer_end(slot, s);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  slot = stage_timer_begin(s, kKernBlockNormBwd);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((a.C + 31) / 32, 3);
  cfg.blockDim = dim3(32 * kSumWarps);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, block_norm_sum_kernel, a, blocks);
  stage_timer_end(slot, s);
  return e;
}

}  // namespace

size_t block_norm_backward_workspace_bytes(int C) { return (size_t)backward_blocks(C) * 3 * C * sizeof(float); }

cudaError_t launch_block_norm(const BlockNormArgs& a, cudaStream_t s) {
  const int K = vectors_of(a.C);
  if (a.bf16) return K == 1 ? forward<bf16, 1>(a, s) : K == 2 ? forward<bf16, 2>(a, s) : forward<bf16, 4>(a, s);
  return K == 1 ? forward<float, 1>(a, s) : K == 2 ? forward<float, 2>(a, s) : forward<float, 4>(a, s);
}
cudaError_t launch_block_norm_backward(const BlockNormArgs& a, cudaStream_t s) {
  const int K = vectors_of(a.C);
  if (a.bf16) return K == 1 ? backward<bf16, 1>(a, s) : K == 2 ? backward<bf16, 2>(a, s) : backward<bf16, 4>(a, s);
  return K == 1 ? backward<float, 1>(a, s) : K == 2 ? backward<float, 2>(a, s) : backward<float, 4>(a, s);
}

}  // namespace gdr
