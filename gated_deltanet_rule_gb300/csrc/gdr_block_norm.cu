// What stands between two blocks of a layer, in one pass over a row (token) of C channels:
//   z = post_w y / sqrt(mean(y^2) + eps)  (or z = y),   x = h + scale sigmoid(gate) z,
//   h_out = x,   n_out = pre_w x / sqrt(mean(x^2) + eps)
// and its gradient. With g = sigmoid(gate), r = 1 / sqrt(mean(y^2) + eps), s = 1 / sqrt(mean(x^2) + eps):
//   dx = dh_out + s (pre_w dn - x s^2 mean(pre_w dn x)),     dpre_w = sum over rows of dn x s,
//   dh = dx,   dscale = sum dx g z,   dgate = dx scale z g (1 - g),   dz = dx scale g,
//   dpost_w = sum dz y r,   dy = r (post_w dz - y r^2 mean(post_w dz y))  (or dz).
//
// Measured: 8192 rows of 4096 bf16 57 us (5.9 TB/s, 86% of the copy bandwidth), their gradient 124 us (5.4 TB/s, 79%),
// that of 2731 rows of 2560 float32 without gate, scale and norm of y 34 us (4.9 TB/s), 24 rows of 2048 5.8 us (launch).
//
// Both are bound by HBM. A block takes a row at a time, a thread 8 channels of it (16 neighbouring bytes, of
// float32 twice), so that a row stays in registers from its one reading to its writing; the weights of a
// thread's channels are read once and kept. Up to four rows are on their way to a block's shared memory.
//
// The gradient's three sums of a row follow one another (mean(y^2) gives x, x gives dx, dx gives dz), but the
// last is linear in dx: with p = post_w scale g it is
//   sum(p dx y) = sum(p y dh_out) + s sum(p y pre_w dn) - s^3 mean(pre_w dn x) sum(p y x),
// so all but mean(y^2) are taken at once, and the next row's mean(y^2) with them: a row costs one exchange, not three. The weights' gradients
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
constexpr int kPairThreads = 320;  // of a block of the gradient that leaves room for another on its SM
constexpr unsigned kAll = 0xffffffffu;

// A thread's vector: 16 bytes of neighbouring channels, so that a warp reads and writes whole sectors
template <typename T>
constexpr int kCh = 16 / (int)sizeof(T);
__device__ __forceinline__ uint4 load(const void* p) {   // read once: nothing for L1 to keep
  uint4 v;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(p));
  return v;
}
template <int n>
struct Vec {   // to compute with
  F2 p[n / 2];
};
template <typename T>
__device__ __forceinline__ Vec<kCh<T>> widen(const uint4& r) {
  const uint32_t u[4] = {r.x, r.y, r.z, r.w};
  Vec<kCh<T>> x;
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int e = 0; e < 4; ++e) x.p[e] = pack(__uint_as_float(u[e] << 16), __uint_as_float(u[e] & 0xFFFF0000u));
  } else {
#pragma unroll
    for (int e = 0; e < 2; ++e) x.p[e] = pack(__uint_as_float(u[2 * e]), __uint_as_float(u[2 * e + 1]));
  }
  return x;
}
__device__ __forceinline__ void store(bf16* p, const Vec<8>& x) {
  uint32_t u[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float a, b;
    unpack(x.p[e], a, b);
    u[e] = ptx::pack_bf16x2(a, b);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(u[0], u[1], u[2], u[3]);
}
template <int n>
__device__ __forceinline__ void store(float* p, const Vec<n>& x) {
#pragma unroll
  for (int e = 0; e < n / 4; ++e) {
    float4 f;
    unpack(x.p[2 * e], f.x, f.y);
    unpack(x.p[2 * e + 1], f.z, f.w);
    reinterpret_cast<float4*>(p)[e] = f;
  }
}
template <int n>
__device__ __forceinline__ Vec<n> filled(float x) {
  Vec<n> v;
#pragma unroll
  for (int e = 0; e < n / 2; ++e) v.p[e] = both(x);
  return v;
}
template <int n>
__device__ __forceinline__ Vec<n> floats(const float* p) {
  Vec<n> x;
#pragma unroll
  for (int e = 0; e < n / 4; ++e) {
    const float4 v = reinterpret_cast<const float4*>(p)[e];
    x.p[2 * e] = pack(v.x, v.y);
    x.p[2 * e + 1] = pack(v.z, v.w);
  }
  return x;
}
template <int n>
__device__ __forceinline__ Vec<n> weights_at(const float* w, int c) { return w ? floats<n>(w + c) : filled<n>(1.f); }   // NULL: ones
template <int n>
__device__ __forceinline__ Vec<n> times(const Vec<n>& a, const Vec<n>& b) {
  Vec<n> x;
#pragma unroll
  for (int e = 0; e < n / 2; ++e) x.p[e] = mul(a.p[e], b.p[e]);
  return x;
}
// sigmoid(x) = 1 / (1 + e^-x): the exponential's and the reciprocal's approximations are good to 2 and 1 units of the last place;
// an infinite exponential gives 0.
__device__ __forceinline__ F2 exp_neg(F2 x) {
  float a, b;
  unpack(mul(x, both(-1.4426950408889634f)), a, b);
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(b));
  return pack(a, b);
}
__device__ __forceinline__ F2 sigmoid_of(F2 e) {   // (of e^-x)
  float a, b;
  unpack(add(e, both(1.f)), a, b);
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(a));
  asm("rcp.approx.ftz.f32 %0, %0;" : "+f"(b));
  return pack(a, b);
}
// A gate between its two uses: sigmoid(x), or where x is not negative 1 - sigmoid(x) = e^-x sigmoid(x) with the sign turned, so that
// neither is formed as a difference that would lose it.
__device__ __forceinline__ float gate_at(float x, float g, float rest) { return x < 0.f ? g : -rest; }
__device__ __forceinline__ F2 kept_gate(F2 x, F2 e, F2 g) {
  float x0, x1, g0, g1, r0, r1;
  unpack(x, x0, x1);
  unpack(g, g0, g1);
  unpack(mul(e, g), r0, r1);
  return pack(gate_at(x0, g0, r0), gate_at(x1, g1, r1));
}
// sigmoid(x) and 1 - sigmoid(x) of that: one of them it is, the other is 1 less that.
__device__ __forceinline__ void both_of(F2 kept, F2& g, F2& rest) {
  float s0, s1;
  unpack(kept, s0, s1);
  const int m0 = __float_as_int(s0) >> 31, m1 = __float_as_int(s1) >> 31, one = __float_as_int(1.f);
  g = add(kept, pack(__int_as_float(one & m0), __int_as_float(one & m1)));
  rest = sub(pack(__int_as_float(one & ~m0), __int_as_float(one & ~m1)), kept);
}

// A thread's 16-byte units of the rows to come, in shared memory: a ring of `stages` rows of `parts` units each, every
// unit copied (asynchronously) and read by the same thread, so that rows on their way cost neither registers nor
// barriers. Without stages (a row does not fit) a row is read when it is needed.
struct Ring {
  uint32_t base, at, end, row, unit;   // shared addresses of this thread's first unit: of the ring, the present row; bytes of a row and of a unit
  int stages;
  __device__ __forceinline__ Ring(void* sm, int stages, int parts)
      : base(ptx::smem_u32(sm) + threadIdx.x * 16), at(base), row(parts * blockDim.x * 16), unit(blockDim.x * 16), stages(stages) {
    end = base + stages * row;
  }
  __device__ __forceinline__ void wait() const {   // for the oldest row
    if (stages >= 4) ptx::cp_async_wait<3>();
    else if (stages == 3) ptx::cp_async_wait<2>();
    else if (stages == 2) ptx::cp_async_wait<1>();
    else if (stages == 1) ptx::cp_async_wait<0>();
  }
  __device__ __forceinline__ void next() {
    at += row;
    if (at == end) at = base;
  }
};
__device__ __forceinline__ void copy16(uint32_t to, const void* p) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
}
__device__ __forceinline__ uint4 shared16(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}
__device__ __forceinline__ void copy(const Ring& g, int u, const void* p) { copy16(g.at + u * g.unit, p); }
__device__ __forceinline__ uint4 take(const Ring& g, int u, const void* p) { return g.stages ? shared16(g.at + u * g.unit) : load(p); }

// float32 channels of a kernel whose threads own 8 of them (32 bytes): a warp's 1024 bytes are copied 16 bytes a lane in
// order (a lane's own 32 bytes would be two half sectors), so lanes read what others copied.
__device__ __forceinline__ void copy_wide(const Ring& g, int u, const float* row, int c, int C) {   // c: the thread's first channel
  const int lane = threadIdx.x & 31, c0 = c - 8 * lane + 4 * lane;
  const uint32_t to = g.at + u * g.unit + 16 * (threadIdx.x - lane);
#pragma unroll
  for (int j = 0; j < 2; ++j)
    if (c0 + 128 * j < C) copy16(to + 512 * j, row + c0 + 128 * j);
}
__device__ __forceinline__ Vec<8> take_wide(const Ring& g, int u, const float* p) {
  if (!g.stages) return floats<8>(p);
  const uint32_t at = g.at + u * g.unit + 16 * threadIdx.x;
  const Vec<4> a = widen<float>(shared16(at)), b = widen<float>(shared16(at + 16));
  return {a.p[0], a.p[1], b.p[0], b.p[1]};
}
// The same for a store: the warp's 1024 bytes go to shared memory and from there in one piece (whole lines: 133 -> 124 us
// for the gradient of 8192 x 4096 against two lanes' sectors at a time). Every lane of the warp calls; `stage` is the
// warp's.
__device__ __forceinline__ void store_wide(float* row, const Vec<8>& x, int c, int C, uint32_t stage) {
  const int lane = threadIdx.x & 31, first = c - 8 * lane;
  if (lane == 0) ptx::bulk_wait_read();   // the last one has been read
  __syncwarp();
  float f[8];
#pragma unroll
  for (int e = 0; e < 4; ++e) unpack(x.p[e], f[2 * e], f[2 * e + 1]);
  const uint32_t at = stage + 32 * lane;
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at), "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]) : "memory");
  asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + 16), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]) : "memory");
  ptx::fence_async_smem();
  __syncwarp();
  if (lane == 0 && first < C)
    asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(row + first), "r"(stage), "r"(min(1024, 4 * (C - first))) : "memory");
  if (lane == 0) ptx::bulk_commit();
}

// Sums over the block, the same in every thread: of one value, of two, of six. red holds 0 where there is no warp; a
// place of it is written again only after another barrier.
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
// In each step a lane gives away half of what it holds, so that 9 exchanges do for six values (lanes with the same upper
// three bits end with one value) and 5 for two, and the warps' sums are read four to a lane.
__device__ __forceinline__ void block_sum(float (&v)[2], float (*red)[16]) {
  const int lane = threadIdx.x & 31;
  float c = (lane & 16 ? v[1] : v[0]) + __shfl_xor_sync(kAll, lane & 16 ? v[0] : v[1], 16);
#pragma unroll
  for (int m = 8; m >= 1; m >>= 1) c += __shfl_xor_sync(kAll, c, m);
  if (blockDim.x > 32) {
    if ((lane & 15) == 0) red[lane >> 4][threadIdx.x >> 5] = c;
    __syncthreads();
    const float4 x = reinterpret_cast<const float4*>(red[lane >> 4])[lane & 3];
    c = (x.x + x.y) + (x.z + x.w);
    c += __shfl_xor_sync(kAll, c, 1);
    c += __shfl_xor_sync(kAll, c, 2);
  }
  v[0] = __shfl_sync(kAll, c, 0);
  v[1] = __shfl_sync(kAll, c, 16);
}
__device__ __forceinline__ void block_sum(float (&v)[6], float (*red)[16]) {
  const int lane = threadIdx.x & 31;
  float a[4], b[2], c;
#pragma unroll
  for (int i = 0; i < 4; ++i) {   // lanes without bit 4 keep values 0 .. 3, those with it 4 .. 7 (6 and 7 are none)
    const float up = i < 2 ? v[4 + i] : 0.f, got = __shfl_xor_sync(kAll, lane & 16 ? v[i] : up, 16);
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
  for (int i = 0; i < 6; ++i) v[i] = __shfl_sync(kAll, c, 4 * i);
}
template <typename T, int K>
__device__ __forceinline__ float squares(const uint4 (&y)[K], const int (&at)[K], int C) {
  F2 s = both(0.f);
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (at[k] >= C) continue;
    const Vec<kCh<T>> v = widen<T>(y[k]);
#pragma unroll
    for (int e = 0; e < kCh<T> / 2; ++e) s = fma(v.p[e], v.p[e], s);
  }
  return sum(s);
}

// One row's vectors of a thread: the k-th is vector threadIdx.x + k blockDim.x. Up to 8 channels a thread the weights are kept.
template <typename T, int K>
__global__ void __launch_bounds__(kMaxThreads, K * kCh<T> <= 8 ? 2 : 1) block_norm_kernel(const __grid_constant__ BlockNormArgs a) {
  constexpr int n = kCh<T>;
  constexpr bool kKeep = K * n <= 8;
  extern __shared__ __align__(16) uint4 dyn[];
  __shared__ __align__(16) float red[3][2][16];
  for (int i = threadIdx.x; i < 3 * 2 * 16; i += blockDim.x) (&red[0][0][0])[i] = 0.f;
  __syncthreads();
  const int C = a.C;
  const float inv_c = 1.f / (float)C;
  int at[K];
#pragma unroll
  for (int k = 0; k < K; ++k) at[k] = n * (threadIdx.x + k * blockDim.x);
  // the next row to fetch, and the present one
  const T *y = static_cast<const T*>(a.y) + blockIdx.x * a.y_row, *gate = static_cast<const T*>(a.gate), *h = static_cast<const T*>(a.h) + (size_t)blockIdx.x * C;
  if (gate) gate += blockIdx.x * a.gate_row;
  const size_t y_step = (size_t)gridDim.x * a.y_row, gate_step = (size_t)gridDim.x * a.gate_row, step = (size_t)gridDim.x * C;
  T *h_out = static_cast<T*>(a.h_out) + (size_t)blockIdx.x * C, *n_out = static_cast<T*>(a.n_out) + (size_t)blockIdx.x * C;
  long long left = (a.rows - blockIdx.x + gridDim.x - 1) / gridDim.x, to_fetch = left;
  Ring ring(dyn, a.stages, 3 * K);
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
        copy(ring, 3 * k, y + at[k]);
        if (gate) copy(ring, 3 * k + 1, gate + at[k]);
        copy(ring, 3 * k + 2, h + at[k]);
      }
      ahead();
      --to_fetch;
    }
    ptx::cp_async_commit();
    ring.next();
  };
  for (int i = 0; i < a.stages; ++i) fetch();
  Vec<n> w_pre[K], w_z[K];
  auto weigh = [&](int k) {
    w_pre[k] = floats<n>(a.pre_w + at[k]);
    w_z[k] = times(weights_at<n>(a.post_w, at[k]), weights_at<n>(a.scale, at[k]));
  };
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (kKeep && at[k] < C) weigh(k);
  // the present row's y, and its root mean square
  uint4 cy[K];
  float r = 1.f;
  auto take_y = [&] {
#pragma unroll
    for (int k = 0; k < K; ++k)
      if (at[k] < C) cy[k] = take(ring, 3 * k, y + at[k]);
  };
  ring.wait();
  take_y();
  if (a.post_w) r = rsqrtf(fmaf(block_sum(squares<T>(cy, at, C), red[2][0]), inv_c, a.eps));
  for (int turn = 0; left > 0; --left, turn ^= 1) {
    Vec<n> x[K];
    F2 s = both(0.f);
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      if (!kKeep) weigh(k);
      x[k] = widen<T>(take(ring, 3 * k + 2, h + at[k]));
      const Vec<n> z = widen<T>(cy[k]);
      Vec<n> g;
      if (gate) g = widen<T>(take(ring, 3 * k + 1, gate + at[k]));
      if (gate) {
#pragma unroll
        for (int e = 0; e < n / 2; ++e) g.p[e] = sigmoid_of(exp_neg(g.p[e]));
      } else {
        g = filled<n>(1.f);
      }
#pragma unroll
      for (int e = 0; e < n / 2; ++e) {
        x[k].p[e] = fma(mul(mul(z.p[e], both(r)), w_z[k].p[e]), g.p[e], x[k].p[e]);
        s = fma(x[k].p[e], x[k].p[e], s);
      }
      store(h_out + at[k], x[k]);
    }
    if (ring.stages) fetch();
    else ahead();
    // the next row's y comes into the same exchange
    float v[2] = {sum(s), 0.f};
    if (left > 1) {
      ring.wait();
      take_y();
      if (a.post_w) v[1] = squares<T>(cy, at, C);
    }
    if (a.post_w) {
      block_sum(v, red[turn]);
      r = rsqrtf(fmaf(v[1], inv_c, a.eps));
    } else {
      v[0] = block_sum(v[0], red[turn][0]);
    }
    const float q = rsqrtf(fmaf(v[0], inv_c, a.eps));
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      if (!kKeep) weigh(k);
#pragma unroll
      for (int e = 0; e < n / 2; ++e) x[k].p[e] = mul(mul(x[k].p[e], both(q)), w_pre[k].p[e]);
      store(n_out + at[k], x[k]);
    }
    h_out += step;
    n_out += step;
  }
}

// The two sums over the rows of a thread's channels: in registers, or (more than 8 channels a thread) in shared memory
// at the thread's own places. kGate is no test in the loops, as two blocks an SM then spill registers (8192 rows of 2048 bf16 82
// us with a test, 72 without; without a gate 85 and 70 for 2560 channels).
template <typename T, int K, bool kWide, bool kGate>
__global__ void __launch_bounds__(kWide ? kMaxThreads : kPairThreads, kWide ? 1 : 2) block_norm_backward_kernel(const __grid_constant__ BlockNormArgs a) {
  constexpr int n = kCh<T>;
  constexpr bool kKeep = K * n <= 8;
  constexpr bool kF32 = sizeof(T) == 4;
  extern __shared__ __align__(16) uint4 dyn[];
  __shared__ __align__(16) float red[3][8][16];
  for (int i = threadIdx.x; i < 3 * 8 * 16; i += blockDim.x) (&red[0][0][0])[i] = 0.f;
  __syncthreads();
  const int C = a.C;
  const float inv_c = 1.f / (float)C;
  int at[K];
#pragma unroll
  for (int k = 0; k < K; ++k) at[k] = n * (threadIdx.x + k * blockDim.x);
  const T *y = static_cast<const T*>(a.y) + blockIdx.x * a.y_row, *gate = static_cast<const T*>(a.gate);
  const T *h = static_cast<const T*>(a.h) + (size_t)blockIdx.x * C, *dn = static_cast<const T*>(a.dn) + (size_t)blockIdx.x * C;
  const float* dh_out = a.dh_out;
  if (kGate) gate += blockIdx.x * a.gate_row;
  if (dh_out) dh_out += (size_t)blockIdx.x * C;
  const size_t y_step = (size_t)gridDim.x * a.y_row, gate_step = (size_t)gridDim.x * a.gate_row, step = (size_t)gridDim.x * C;
  size_t out = (size_t)blockIdx.x * C;   // where the present row's outputs go
  long long left = (a.rows - blockIdx.x + gridDim.x - 1) / gridDim.x, to_fetch = left;
  constexpr int kUnits = kF32 ? 5 : 6;   // of a thread's vector: y, gate, h, dn, dh_out
  Ring ring(dyn, a.stages, K * kUnits);
  float* acc_sm = reinterpret_cast<float*>(dyn + (size_t)a.stages * K * kUnits * blockDim.x);   // (not kept) [2][C]
  const uint32_t stage = ptx::smem_u32(acc_sm + (kKeep ? 0 : 2 * C)) + (threadIdx.x >> 5) * K * 1024;
  auto ahead = [&] {
    y += y_step;
    if (kGate) gate += gate_step;
    h += step;
    dn += step;
    if (dh_out) dh_out += step;
  };
  auto fetch = [&] {
    if (!kF32) __syncwarp();   // (other lanes have read what is written over)
    if (to_fetch > 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) {
        if (!kF32 && dh_out) copy_wide(ring, k * kUnits + 4, dh_out, at[k], C);
        if (at[k] >= C) continue;
        copy(ring, k * kUnits, y + at[k]);
        if (kGate) copy(ring, k * kUnits + 1, gate + at[k]);
        copy(ring, k * kUnits + 2, h + at[k]);
        copy(ring, k * kUnits + 3, dn + at[k]);
        if (kF32 && dh_out) copy(ring, k * kUnits + 4, dh_out + at[k]);
      }
      ahead();
      --to_fetch;
    }
    ptx::cp_async_commit();
    ring.next();
  };
  auto arrived = [&] {
    ring.wait();
    if (!kF32) __syncwarp();
  };
  for (int i = 0; i < a.stages; ++i) fetch();
  Vec<n> w_pre[K], w_z[K], acc[2][K];
  auto weigh = [&](int k) {
    w_pre[k] = floats<n>(a.pre_w + at[k]);
    w_z[k] = times(weights_at<n>(a.post_w, at[k]), weights_at<n>(a.scale, at[k]));
  };
#pragma unroll
  for (int k = 0; k < K; ++k) {
    acc[0][k] = acc[1][k] = filled<n>(0.f);
    if (at[k] >= C) continue;
    if (kKeep) {
      weigh(k);
    } else {
      store(acc_sm + at[k], acc[0][k]);
      store(acc_sm + C + at[k], acc[1][k]);
    }
  }
  // y and dn stay as they are, and are widened where they are used; the next row's y comes early, so that its mean
  // square goes into the present row's exchange
  uint4 cy[K], next_y[K];
  float r = 1.f;
  arrived();
#pragma unroll
  for (int k = 0; k < K; ++k)
    if (at[k] < C) cy[k] = take(ring, k * kUnits, y + at[k]);
  if (a.post_w) r = rsqrtf(fmaf(block_sum(squares<T>(cy, at, C), red[2][0]), inv_c, a.eps));
  for (int turn = 0; left > 0; --left, turn ^= 1) {
    uint4 cn[K];
    Vec<n> x[K], g[K], dx[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      cn[k] = take(ring, k * kUnits + 3, dn + at[k]);
      x[k] = widen<T>(take(ring, k * kUnits + 2, h + at[k]));
      if (kGate) g[k] = widen<T>(take(ring, k * kUnits + 1, gate + at[k]));
      if constexpr (kF32) dx[k] = dh_out ? widen<float>(take(ring, k * kUnits + 4, dh_out + at[k])) : filled<n>(0.f);
      else dx[k] = dh_out ? take_wide(ring, k * kUnits + 4, dh_out + at[k]) : filled<n>(0.f);
    }
    if (ring.stages) fetch();
    else ahead();
    float s[6];
    s[5] = 0.f;
    if (left > 1) {
      arrived();
#pragma unroll
      for (int k = 0; k < K; ++k)
        if (at[k] < C) next_y[k] = take(ring, k * kUnits, y + at[k]);
      if (a.post_w) s[5] = squares<T>(next_y, at, C);
    }
    // sums of x^2, pre_w dn x, p y dh_out, p y pre_w dn, p y x
    F2 t[5] = {both(0.f), both(0.f), both(0.f), both(0.f), both(0.f)};
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] >= C) continue;
      if (!kKeep) weigh(k);
      const Vec<n> v = widen<T>(cy[k]), d = widen<T>(cn[k]);
#pragma unroll
      for (int e = 0; e < n / 2; ++e) {
        F2 py = mul(w_z[k].p[e], v.p[e]);
        const F2 wdn = mul(w_pre[k].p[e], d.p[e]);
        if constexpr (kGate) {
          const F2 ex = exp_neg(g[k].p[e]), open = sigmoid_of(ex);
          py = mul(py, open);
          g[k].p[e] = kept_gate(g[k].p[e], ex, open);
        }
        x[k].p[e] = fma(py, both(r), x[k].p[e]);
        t[0] = fma(x[k].p[e], x[k].p[e], t[0]);
        t[1] = fma(wdn, x[k].p[e], t[1]);
        t[2] = fma(py, dx[k].p[e], t[2]);
        t[3] = fma(py, wdn, t[3]);
        t[4] = fma(py, x[k].p[e], t[4]);
      }
    }
#pragma unroll
    for (int i = 0; i < 5; ++i) s[i] = sum(t[i]);
    block_sum(s, red[turn]);
    const float q = rsqrtf(fmaf(s[0], inv_c, a.eps)), mx = s[1] * inv_c * q * q * q;
    const float my = a.post_w ? (s[2] + q * s[3] - mx * s[4]) * inv_c * r * r * r : 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
      if (at[k] < C) {
        if (!kKeep) {
          weigh(k);
          acc[0][k] = floats<n>(acc_sm + at[k]);
          acc[1][k] = floats<n>(acc_sm + C + at[k]);
        }
        const Vec<n> d = widen<T>(cn[k]), v = widen<T>(cy[k]);
        Vec<n> dg, dy;
#pragma unroll
        for (int e = 0; e < n / 2; ++e) {
          acc[0][k].p[e] = fma(d.p[e], mul(x[k].p[e], both(q)), acc[0][k].p[e]);
          dx[k].p[e] = fma(mul(w_pre[k].p[e], d.p[e]), both(q), fma(x[k].p[e], both(-mx), dx[k].p[e]));
          F2 dxg = dx[k].p[e], rest;
          if constexpr (kGate) {
            F2 open;
            both_of(g[k].p[e], open, rest);
            dxg = mul(dxg, open);
          }
          const F2 b = mul(mul(dxg, both(r)), v.p[e]);   // dx g y r
          acc[1][k].p[e] = add(acc[1][k].p[e], b);
          if constexpr (kGate) dg.p[e] = mul(mul(b, w_z[k].p[e]), rest);
          dy.p[e] = fma(v.p[e], both(-my), mul(mul(dxg, both(r)), w_z[k].p[e]));
        }
        if (kGate) store(static_cast<T*>(a.dgate) + out + at[k], dg);
        store(static_cast<T*>(a.dy) + out + at[k], dy);
        if (!kKeep) {
          store(acc_sm + at[k], acc[0][k]);
          store(acc_sm + C + at[k], acc[1][k]);
        }
        if constexpr (kF32) store(a.dh + out + at[k], dx[k]);
      }
      if constexpr (!kF32) store_wide(a.dh + out, dx[k], at[k], C, stage + k * 1024);
    }
    out += step;
#pragma unroll
    for (int k = 0; k < K; ++k) cy[k] = next_y[k];
    if (a.post_w) r = rsqrtf(fmaf(s[5], inv_c, a.eps));
  }
  if ((threadIdx.x & 31) == 0) ptx::bulk_wait_all();
  // the block's partial sums
#pragma unroll
  for (int k = 0; k < K; ++k) {
    if (at[k] >= C) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i)
      store(a.partial + ((size_t)blockIdx.x * 2 + i) * C + at[k], kKeep ? acc[i][k] : floats<n>(acc_sm + i * C + at[k]));
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

// Vectors of a row, of es bytes a channel: 1, 2, 4 or 8 a thread, for up to kMaxThreads threads (8 channels a thread while
// that is enough).
int vectors_of(int C, int es) {
  int k = es / 2;
  while (C * es / 16 > k * kMaxThreads) k *= 2;
  return k;
}
int threads_of(int C, int es) { return (C * es / 16 + 32 * vectors_of(C, es) - 1) / (32 * vectors_of(C, es)) * 32; }
// Blocks of the gradient that an SM holds.
int backward_per(int C, int es) {
  const int t = threads_of(C, es);
  return t > kPairThreads || vectors_of(C, es) > es / 2 ? 1 : std::min(16, 2 * kPairThreads / t);
}
// Rows on their way to a block, of `per` on an SM: at most four.
constexpr int kSmemSM = 220 << 10;
int stages_of(int per, int bytes, int more) {
  return std::max(0, std::min(4, (kSmemSM / per - 2048 - more) / bytes));
}

template <typename T, int K>
cudaError_t forward(BlockNormArgs a, cudaStream_t s) {
  const int t = threads_of(a.C, sizeof(T)), per = std::min(32, (K * kCh<T> <= 8 ? 2 : 1) * kMaxThreads / t);
  const int bytes = 3 * K * t * 16;
  a.stages = stages_of(per, bytes, 0);
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(block_norm_kernel<T, K>), 224 << 10, done);
  if (e != cudaSuccess) return e;
  const int slot = stage_timer_begin(s, kKernBlockNorm);
  block_norm_kernel<T, K><<<(unsigned)std::min<long long>(a.rows, kNumSMs * per), t, a.stages * bytes, s>>>(a);
  stage_timer_end(slot, s);
  return cudaGetLastError();
}
template <typename T, int K, bool kWide, bool kGate>
cudaError_t backward_of(BlockNormArgs a, cudaStream_t s) {
  const int t = threads_of(a.C, sizeof(T)), per = backward_per(a.C, sizeof(T)), blocks = (int)std::min<long long>(a.rows, kNumSMs * per);
  const int bytes = K * (sizeof(T) == 4 ? 5 : 6) * t * 16, more = (K * kCh<T> <= 8 ? 0 : 2 * a.C * 4) + (sizeof(T) == 2 ? K * t * 32 : 0);
  a.stages = stages_of(per, bytes, more);
  const int smem = a.stages * bytes + more;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(block_norm_backward_kernel<T, K, kWide, kGate>), 224 << 10, done);
  if (e != cudaSuccess) return e;
  int slot = stage_timer_begin(s, kKernBlockNormBwd);
  block_norm_backward_kernel<T, K, kWide, kGate><<<blocks, t, smem, s>>>(a);
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
template <typename T, int K, bool kWide>
cudaError_t backward(const BlockNormArgs& a, cudaStream_t s) {
  return a.gate ? backward_of<T, K, kWide, true>(a, s) : backward_of<T, K, kWide, false>(a, s);
}

}  // namespace

size_t block_norm_backward_workspace_bytes(int C) {
  return (size_t)kNumSMs * std::max(backward_per(C, 2), backward_per(C, 4)) * 2 * C * sizeof(float);
}

cudaError_t launch_block_norm(const BlockNormArgs& a, cudaStream_t s) {
  const int K = vectors_of(a.C, a.bf16 ? 2 : 4);
  if (a.bf16) return K == 1 ? forward<bf16, 1>(a, s) : K == 2 ? forward<bf16, 2>(a, s) : forward<bf16, 4>(a, s);
  return K == 2 ? forward<float, 2>(a, s) : K == 4 ? forward<float, 4>(a, s) : forward<float, 8>(a, s);
}
cudaError_t launch_block_norm_backward(const BlockNormArgs& a, cudaStream_t s) {
  const int es = a.bf16 ? 2 : 4, K = vectors_of(a.C, es);
  const bool pair = backward_per(a.C, es) > 1;
  if (a.bf16) {
    if (K == 1) return pair ? backward<bf16, 1, false>(a, s) : backward<bf16, 1, true>(a, s);
    return K == 2 ? backward<bf16, 2, true>(a, s) : backward<bf16, 4, true>(a, s);
  }
  if (K == 2) return pair ? backward<float, 2, false>(a, s) : backward<float, 2, true>(a, s);
  return K == 4 ? backward<float, 4, true>(a, s) : backward<float, 8, true>(a, s);
}

}  // namespace gdr
