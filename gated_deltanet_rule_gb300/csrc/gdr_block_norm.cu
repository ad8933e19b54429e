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
// thread's channels are read once and kept. Up to four rows are on their way to a block's shared memory.
//
// The gradient's three sums of a row follow one another (mean(y^2) gives x, x gives dx, dx gives dz), but the
// last is linear in dx: with p = post_w scale g it is
//   sum(p dx y) = sum(p y dh_out) + s sum(p y pre_w dn) - s^3 mean(pre_w dn x) sum(p y x),
// so all but mean(y^2) are taken at once, and a row costs two exchanges instead of three. The weights' gradients
// need two sums over the rows a channel, A = sum dn x s and B = sum dx g y r: dpre_w = A, dpost_w = scale B,
// dscale = post_w B. They stay with the thread that owns the channel (in registers, for more than kWideC
// channels in shared memory), leave as one partial row a block and are summed in order by a second kernel: no
// atomics, the same bits every time.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>

#include "gdr_serve.h"
#include "pairs.cuh"
#include "ptx.cuh"

namespace gdr {
namespace {

using namespace pairs;
using bf16 = __nv_bfloat16;
constexpr int kMaxThreads = 512;   // of a block; 8 channels a thread
constexpr int kWideC = 8 * kMaxThreads;
constexpr unsigned kAll = 0xffffffffu;

// 8 channels as they lie in memory
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];
};
template <typename T>
__device__ __forceinline__ Raw<T> load(const T* p) {   // read once: nothing for L1 to keep
  Raw<T> r;
#pragma unroll
  for (int k = 0; k < (int)(sizeof(T) / 2); ++k)
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.v[k].x), "=r"(r.v[k].y), "=r"(r.v[k].z), "=r"(r.v[k].w) : "l"(reinterpret_cast<const uint4*>(p) + k));
  return r;
}
// 8 channels to compute with
struct Vec {
  F2 p[4];
};
__device__ __forceinline__ Vec widen(const Raw<bf16>& r) {
  const uint32_t u[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
  Vec x;
#pragma unroll
  for (int e = 0; e < 4; ++e) x.p[e] = pack(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xFFFF0000u));
  return x;
}
__device__ __forceinline__ Vec widen(const Raw<float>& r) {
  Vec x;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    x.p[2 * k] = pack(__uint_as_float(r.v[k].x), __uint_as_float(r.v[k].y));
    x.p[2 * k + 1] = pack(__uint_as_float(r.v[k].z), __uint_as_float(r.v[k].w));
  }
  return x;
}
__device__ __forceinline__ void store(bf16* p, const Vec& x) {
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a, b;
    unpack(x.p[e], a, b);
    u[e] = ptx::pack_bf16x2(a, b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
__device__ __forceinline__ void store(float* p, const Vec& x) {
  float f[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) unpack(x.p[e], f[2 * e], f[2 * e + 1]);
  reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
}
__device__ __forceinline__ Vec filled(float x) { return {both(x), both(x), both(x), both(x)}; }
__device__ __forceinline__ Vec weight8(const float* w, int c) {   // NULL: ones
  if (!w) return filled(1.f);
  Vec x;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float4 v = __ldg(reinterpret_cast<const float4*>(w + c) + k);
    x.p[2 * k] = pack(v.x, v.y);
    x.p[2 * k + 1] = pack(v.z, v.w);
  }
  return x;
}
__device__ __forceinline__ Vec times(const Vec& a, const Vec& b) { return {mul(a.p[0], b.p[0]), mul(a.p[1], b.p[1]), mul(a.p[2], b.p[2]), mul(a.p[3], b.p[3])}; }
// 1 / (1 + e^-x): the exponential's and the reciprocal's approximations are good to 2 and 1 units of the last place;
// an infinite exponential gives 0.
__device__ __forceinline__ F2 sigmoid(F2 x) {
  float a, b;
  unpack(mul(x, both(-1.4426950408889634f)), a, b);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
  unpack(add(pack(a, b), both(1.f)), a, b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  return pack(a, b);
}

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

// Sums over the block, the same in every thread. red holds 0 where there is no warp; a place of it is written again
// only after another barrier.
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(kAll, v, m);
  if (blockDim.x == 32) return v;
  const int lane = threadIdx.x & 31;
  if (lane == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  const float4 x = reinterpret_cast<const float4*>(red)[lane & 3];
  v = (x.x + x.y) + (x.z + x.w);
  v += __shfl_xor_sync(kAll, v, 1);
  return v + __shfl_xor_sync(kAll, v, 2);
}
// Of five values: in each step a lane gives away half of what it holds, so that 9 exchanges do for all (lanes with the
// same upper three bits end with one value), and the warps' sums are read four to a lane.
__device__ __forceinline__ void block_sum5(float (&v)[5], float (*red)[16]) {
  const int lane = threadIdx.x & 31;
  float a[4], b[2], c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // lanes without bit 4 keep values 0 .. 3, those with it 4 .. 7 (of which 4 alone is there)
    const float up = i == 0 ? v[4] : 0.f, got = __shfl_xor_sync(kAll, lane & 16 ? v[i] : up, 16);
    a[i] = (lane & 16 ? up : v[i]) + got;
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) b[i] = (lane & 8 ? a[i + 2] : a[i]) + __shfl_xor_sync(kAll, lane & 8 ? a[i] : a[i + 2], 8);
  c = (lane & 4 ? b[1] : b[0]) + __shfl_xor_sync(kAll, lane & 4 ? b[0] : b[1], 4);
  c += __shfl_xor_sync(kAll, c, 2);
  c += __shfl_xor_sync(kAll, c, 1);
  if (blockDim.x > 32) {
    if ((lane & 3) == 0) red[lane >> 2][threadIdx.x >> 5] = c;
    __syncthreads();
    const float4 x = reinterpret_cast<const float4*>(red[lane >> 2])[lane & 3];
    c = (x.x + x.y) + (x.z + x.w);
    c += __shfl_xor_sync(kAll, c, 1);
    c += __shfl_xor_sync(kAll, c, 2);
  }
#pragma unroll
  for (int i = 0; i < 5; ++i) v[i] = __shfl_sync(kAll, c, 4 * i);
}

// One row's vectors of a thread: k-th at channel 8 (threadIdx.x + k blockDim.x).
template <typename T, int K>
__global__ void __launch_bounds__(kMaxThreads, K == 1 ? 2 : 1) block_norm_kernel(const __grid_constant__ BlockNormArgs a) {
  constexpr int kPart = sizeof(T) / 2;   // units of 8 channels
  extern __shared__ __align__(16) uint4 dyn[];
  __shared__ __align__(16) float red[2][16];
  if (threadIdx.x < 32) red[threadIdx.x >> 4][threadIdx.x & 15] = 0.f;
  __syncthreads();
  const int C = a.C;
  const float inv_c = 1.f / (float)C;
  int at[K];
#pragma unroll
  for (int k = 0; k < K; ++k) at[k] = 8 * (threadIdx.x + k * blockDim.x);
  // the next row to fetch, and the present one
  const T *y = static_cast<const T*>(a.y) + blockIdx.x * a.y_row, *gate = static_cast<const T*>(a.gate), *h = static_cast<const T*>(a.h) + (size_t)blockIdx.x * C;
  if (gate) gate += blockIdx.x * a.gate_row;
  const size_t y_step = (size_t)gridDim.x * a.y_row, gate_step = (size_t)gridDim.x * a.gate_row, step = (size_t)gridDim.x * C;
  T *h_out = static_cast<T*>(a.h_out) + (size_t)blockIdx.x * C, *n_out = static_cast<T*>(a.n_out) + (size_t)blockIdx.x * C;
  long long left = (a.rows - blockIdx.x + gridDim.x - 1) / gridDim.x, to_fetch = left;
  Ring ring{dyn + threadIdx.x, a.stages, 3 * K * kPart, 0};
  auto ahead = [&] {
    y += y_step;
    if (gate) gate += gate_step;
    h += step;
  };
  auto fetch = [&] {   // into the ring's present slot
    if (to_fetch > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (at[k] >= C) continue;
        copy(ring, (3 * k) * kPart, y + at[k]);
        if (gate) copy(ring, (3 * k + 1) * kPart, gate + at[k]);
        copy(ring, (3 * k + 2) * kPart, h + at[k]);
      }
      ahead();
      --to_fetch;
    }
    ptx::cp_async_commit();
    ring.next();
  };
  for (int i = 0; i < a.stages; ++i) fetch();
  Vec w_pre, w_z;   // (one vector a thread: kept)
  if (K == 1 && at[0] < C) {
    w_pre = weight8(a.pre_w, at[0]);
    w_z = times(weight8(a.post_w, at[0]), weight8(a.scale, at[0]));
  }
  for (; left > 0; --left) {
    Vec x[K], z[K], g[K];
    ring.wait();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      x[k] = widen(take(ring, (3 * k + 2) * kPart, h + at[k]));
      z[k] = widen(take(ring, (3 * k) * kPart, y + at[k]));
      if (gate) g[k] = widen(take(ring, (3 * k + 1) * kPart, gate + at[k]));
    }
    if (ring.stages) fetch();
    else ahead();
    float r = 1.f;
    if (a.post_w) {
      F2 s = both(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (at[k] < C)
#pragma unroll
          for (int e = 0; e < 4; ++e) s = fma(z[k].p[e], z[k].p[e], s);
      r = rsqrtf(fmaf(block_sum(sum(s), red[0]), inv_c, a.eps));
    }
    F2 s = both(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      if (K > 1) w_z = times(weight8(a.post_w, at[k]), weight8(a.scale, at[k]));
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const F2 f = mul(mul(z[k].p[e], both(r)), w_z.p[e]);
        x[k].p[e] = gate ? fma(f, sigmoid(g[k].p[e]), x[k].p[e]) : add(x[k].p[e], f);
        s = fma(x[k].p[e], x[k].p[e], s);
      }
      store(h_out + at[k], x[k]);
    }
    r = rsqrtf(fmaf(block_sum(sum(s), red[1]), inv_c, a.eps));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      if (K > 1) w_pre = weight8(a.pre_w, at[k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[k].p[e] = mul(mul(x[k].p[e], both(r)), w_pre.p[e]);
      store(n_out + at[k], x[k]);
    }
    h_out += step;
    n_out += step;
    if (!a.post_w) __syncthreads();   // red[1] is written again before another barrier
  }
}

// The two sums over the rows of a thread's channels: in registers, or (more than one vector a thread) in shared
// memory at the thread's own places.
template <typename T, int K>
__global__ void __launch_bounds__(kMaxThreads, 1) block_norm_backward_kernel(const __grid_constant__ BlockNormArgs a) {
  constexpr int kPart = sizeof(T) / 2;
  extern __shared__ __align__(16) uint4 dyn[];
  __shared__ __align__(16) float red[2][8][16];
  for (int i = threadIdx.x; i < 2 * 8 * 16; i += blockDim.x) (&red[0][0][0])[i] = 0.f;
  __syncthreads();
  const int C = a.C;
  const float inv_c = 1.f / (float)C;
  int at[K];
#pragma unroll
  for (int k = 0; k < K; ++k) at[k] = 8 * (threadIdx.x + k * blockDim.x);
  const T *y = static_cast<const T*>(a.y) + blockIdx.x * a.y_row, *gate = static_cast<const T*>(a.gate);
  const T *h = static_cast<const T*>(a.h) + (size_t)blockIdx.x * C, *dn = static_cast<const T*>(a.dn) + (size_t)blockIdx.x * C;
  const float* dh_out = a.dh_out;
  if (gate) gate += blockIdx.x * a.gate_row;
  if (dh_out) dh_out += (size_t)blockIdx.x * C;
  const size_t y_step = (size_t)gridDim.x * a.y_row, gate_step = (size_t)gridDim.x * a.gate_row, step = (size_t)gridDim.x * C;
  size_t out = (size_t)blockIdx.x * C;   // where the present row's outputs go
  long long left = (a.rows - blockIdx.x + gridDim.x - 1) / gridDim.x, to_fetch = left;
  constexpr int kVec = 4 * kPart + 2;    // units of a thread's vector: y, gate, h, dn, dh_out
  Ring ring{dyn + threadIdx.x, a.stages, K * kVec, 0};
  float* acc_sm = reinterpret_cast<float*>(dyn + (size_t)a.stages * K * kVec * blockDim.x);   // (K > 1) [2][C]
  auto ahead = [&] {
    y += y_step;
    if (gate) gate += gate_step;
    h += step;
    dn += step;
    if (dh_out) dh_out += step;
  };
  auto fetch = [&] {
    if (to_fetch > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (at[k] >= C) continue;
        copy(ring, k * kVec, y + at[k]);
        if (gate) copy(ring, k * kVec + kPart, gate + at[k]);
        copy(ring, k * kVec + 2 * kPart, h + at[k]);
        copy(ring, k * kVec + 3 * kPart, dn + at[k]);
        if (dh_out) copy(ring, k * kVec + 4 * kPart, dh_out + at[k]);
      }
      ahead();
      --to_fetch;
    }
    ptx::cp_async_commit();
    ring.next();
  };
  for (int i = 0; i < a.stages; ++i) fetch();
  Vec w_pre, w_z, acc[2];
  if (K == 1 && at[0] < C) {
    w_pre = weight8(a.pre_w, at[0]);
    w_z = times(weight8(a.post_w, at[0]), weight8(a.scale, at[0]));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    acc[i] = filled(0.f);
    if (K > 1)
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (at[k] < C) store(acc_sm + i * C + at[k], acc[i]);
  }
  for (; left > 0; --left) {
    Raw<T> cy[K], cn[K];   // y and dn stay as they are, and are widened where they are used
    Vec x[K], g[K], dx[K];
    ring.wait();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      cy[k] = take(ring, k * kVec, y + at[k]);
      cn[k] = take(ring, k * kVec + 3 * kPart, dn + at[k]);
      x[k] = widen(take(ring, k * kVec + 2 * kPart, h + at[k]));
      g[k] = gate ? widen(take(ring, k * kVec + kPart, gate + at[k])) : filled(1.f);
      dx[k] = dh_out ? widen(take(ring, k * kVec + 4 * kPart, dh_out + at[k])) : filled(0.f);
    }
    if (ring.stages) fetch();
    else ahead();
    float r = 1.f;
    if (a.post_w) {
      F2 s = both(0.f);
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (at[k] >= C) continue;
        const Vec v = widen(cy[k]);
#pragma unroll
        for (int e = 0; e < 4; ++e) s = fma(v.p[e], v.p[e], s);
      }
      r = rsqrtf(fmaf(block_sum(sum(s), red[0][0]), inv_c, a.eps));
    }
    // sums of x^2, pre_w dn x, p y dh_out, p y pre_w dn, p y x
    F2 t[5] = {both(0.f), both(0.f), both(0.f), both(0.f), both(0.f)};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      if (K > 1) {
        w_z = times(weight8(a.post_w, at[k]), weight8(a.scale, at[k]));
        w_pre = weight8(a.pre_w, at[k]);
      }
      const Vec v = widen(cy[k]), d = widen(cn[k]);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if (gate) g[k].p[e] = sigmoid(g[k].p[e]);
        const F2 py = mul(mul(w_z.p[e], v.p[e]), g[k].p[e]), wdn = mul(w_pre.p[e], d.p[e]);
        x[k].p[e] = fma(py, both(r), x[k].p[e]);
        t[0] = fma(x[k].p[e], x[k].p[e], t[0]);
        t[1] = fma(wdn, x[k].p[e], t[1]);
        t[2] = fma(py, dx[k].p[e], t[2]);
        t[3] = fma(py, wdn, t[3]);
        t[4] = fma(py, x[k].p[e], t[4]);
      }
    }
    float s[5];
#pragma unroll
    for (int i = 0; i < 5; ++i) s[i] = sum(t[i]);
    block_sum5(s, red[1]);
    const float q = rsqrtf(fmaf(s[0], inv_c, a.eps)), mx = s[1] * inv_c * q * q * q;
    const float my = a.post_w ? (s[2] + q * s[3] - mx * s[4]) * inv_c * r * r * r : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      if (K > 1) {
        w_z = times(weight8(a.post_w, at[k]), weight8(a.scale, at[k]));
        w_pre = weight8(a.pre_w, at[k]);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          Raw<float> v;
          v.v[0] = reinterpret_cast<const uint4*>(acc_sm + i * C + at[k])[0];
          v.v[1] = reinterpret_cast<const uint4*>(acc_sm + i * C + at[k])[1];
          acc[i] = widen(v);
        }
      }
      const Vec d = widen(cn[k]), v = widen(cy[k]);
      Vec dg, dy;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        acc[0].p[e] = fma(d.p[e], mul(x[k].p[e], both(q)), acc[0].p[e]);
        dx[k].p[e] = fma(mul(w_pre.p[e], d.p[e]), both(q), fma(x[k].p[e], both(-mx), dx[k].p[e]));
        const F2 dxg = mul(dx[k].p[e], g[k].p[e]), b = mul(mul(dxg, both(r)), v.p[e]);   // dx g y r
        acc[1].p[e] = add(acc[1].p[e], b);
        const F2 bw = mul(b, w_z.p[e]);
        dg.p[e] = sub(bw, mul(bw, g[k].p[e]));
        dy.p[e] = fma(v.p[e], both(-my), mul(mul(dxg, both(r)), w_z.p[e]));
      }
      store(a.dh + out + at[k], dx[k]);
      if (gate) store(static_cast<T*>(a.dgate) + out + at[k], dg);
      store(static_cast<T*>(a.dy) + out + at[k], dy);
      if (K > 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) store(acc_sm + i * C + at[k], acc[i]);
    }
    out += step;
    if (!a.post_w) __syncthreads();   // red[1] is written again before another barrier
  }
  // the block's partial sums
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (at[k] >= C) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float* to = a.partial + ((size_t)blockIdx.x * 2 + i) * C + at[k];
      if (K == 1) {
        store(to, acc[i]);
      } else {
        for (int j = 0; j < 2; ++j) reinterpret_cast<uint4*>(to)[j] = reinterpret_cast<const uint4*>(acc_sm + i * C + at[k])[j];
      }
    }
  }
}

// Sums of the blocks' partial rows, in order: a block 32 channels of one of the two, its warps every kSumWarps-th
// partial each.
constexpr int kSumWarps = 16;
__global__ void __launch_bounds__(32 * kSumWarps) block_norm_sum_kernel(const __grid_constant__ BlockNormArgs a, int blocks) {
  __shared__ float part[kSumWarps][32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, i = blockIdx.y, c = blockIdx.x * 32 + lane;
  const bool mine = warp == 0 && c < a.C;
  const float post = mine && a.post_w ? __ldg(a.post_w + c) : 1.f, scale = mine && a.scale ? __ldg(a.scale + c) : 1.f;
  ptx::wait_prerequisite();
  float s = 0.f;
  if (c < a.C)
#pragma unroll 10
    for (int b = warp; b < blocks; b += kSumWarps) s += __ldcg(a.partial + ((size_t)b * 2 + i) * a.C + c);
  part[warp][lane] = s;
  __syncthreads();
  if (!mine) return;
  s = 0.f;
#pragma unroll
  for (int w = 0; w < kSumWarps; ++w) s += part[w][lane];
  if (i == 0) {
    a.dpre_w[c] = s;
  } else {
    if (a.dpost_w) a.dpost_w[c] = scale * s;
    if (a.dscale) a.dscale[c] = post * s;
  }
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
  const int bytes = K * (4 * (int)(sizeof(T) / 2) + 2) * t * 16, more = K == 1 ? 0 : 2 * a.C * 4;
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
  cfg.gridDim = dim3((a.C + 31) / 32, a.post_w || a.scale ? 2 : 1);
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

size_t block_norm_backward_workspace_bytes(int C) { return (size_t)backward_blocks(C) * 2 * C * sizeof(float); }

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
