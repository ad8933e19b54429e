// RMS norm of every query and key head and the rotation by position, in one pass:
//   y = w x / sqrt(mean(x^2) + eps);   pair j of the first R elements turned by pos inv_freq[j];
//   elements R .. D-1 pass through.
// Pairs are (j, j + R/2), or (2j, 2j + 1) when interleaved. Forward (dense outputs, or k and v left
// in a cache's pages) and gradient.
//
// Layout: D/8 lanes hold one head, eight elements each, chosen so that both members of a pair lie in
// one lane: in the half-split form a lane of the rotated part holds four elements at 4 l and their
// partners at R/2 + 4 l, every other lane eight neighbours. Pair j of lane l is 4 l + (0..3) in both
// forms, so a lane's four angles serve every head of its token and the loop over heads needs no
// exchange but the sum of squares (shuffles over the head's lanes).
//
// Angles: pos inv_freq is formed in turns modulo one by 64-bit integer arithmetic (inv_freq / 2 pi as
// a 64-bit binary fraction, times the position, dropping whole turns), exact to 2^-32 turn at any
// 31-bit position; float32 angles would be off by 0.06 rad at position 2^20, and float64 arithmetic
// runs at 1/64 of the float32 rate here. The fraction is reduced to an eighth turn before sincospif.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdr_serve.h"
#include "ptx.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kUnroll = 4;   // heads per lane in flight: 4 x 2 loads of 8 or 16 bytes

template <typename T>
struct Raw;   // four consecutive elements as loaded
template <>
struct Raw<__nv_bfloat16> {
  uint2 u;
  __device__ void load(const __nv_bfloat16* p) { u = __ldg(reinterpret_cast<const uint2*>(p)); }
  __device__ void get(float* x) const {
    x[0] = __uint_as_float(u.x << 16);
    x[1] = __uint_as_float(u.x & 0xFFFF0000u);
    x[2] = __uint_as_float(u.y << 16);
    x[3] = __uint_as_float(u.y & 0xFFFF0000u);
  }
  __device__ static void put(__nv_bfloat16* p, const float* x) {
    *reinterpret_cast<uint2*>(p) = make_uint2(ptx::pack_bf16x2(x[0], x[1]), ptx::pack_bf16x2(x[2], x[3]));
  }
  __device__ void copy(__nv_bfloat16* p) const { *reinterpret_cast<uint2*>(p) = u; }
};
template <>
struct Raw<float> {
  float4 u;
  __device__ void load(const float* p) { u = __ldg(reinterpret_cast<const float4*>(p)); }
  __device__ void get(float* x) const { x[0] = u.x; x[1] = u.y; x[2] = u.z; x[3] = u.w; }
  __device__ static void put(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
  __device__ void copy(float* p) const { *reinterpret_cast<float4*>(p) = u; }
};

// inv_freq / (2 pi) modulo one as a 64-bit binary fraction, from the bits of the double.
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int e = (int)((bits >> 52) & 0x7FF) - 1023;
  if (e == -1023) return 0;   // zero (and subnormals: below 2^-1022 rad per position)
  const uint64_t m = (bits << 11) | 0x8000000000000000ull;                 // f = m 2^(e - 63)
  // 1 / (2 pi) = C 2^-66, C = round(2^65 / pi); m C 2^-64 2^(e - 65) = f / (2 pi)
  const uint64_t t = __umul64hi(m, 0xA2F9836E4E44152Aull);
  const int sh = e - 1;                                                    // fraction = t 2^sh mod 2^64
  uint64_t r = 0;
  if (sh >= 0) r = sh < 64 ? t << sh : 0;
  else if (sh > -64) r = t >> -sh;
  return (bits >> 63) ? 0ull - r : r;
}

// cos and sin of pos * fraction turns
__device__ __forceinline__ void turn_sincos(uint64_t frac, int pos, float& c, float& s) {
  const uint32_t t = (uint32_t)((frac * (uint64_t)(int64_t)pos) >> 32);   // turns modulo one, 2^-32 units
  const uint32_t quad = (t + 0x20000000u) >> 30;                           // nearest quarter turn
  const int32_t rem = (int32_t)(t - (quad << 30));                         // within an eighth of a turn
  float sr, cr;
  sincospif((float)rem * 4.656612873077393e-10f, &sr, &cr);               // 2^-31: turns to units of pi
  const bool swap = quad & 1;
  s = swap ? cr : sr;
  c = swap ? sr : cr;
  if ((quad & 3) == 1 || (quad & 3) == 2) c = -c;
  if (quad & 2) s = -s;
}

// What a lane holds: its two runs of four elements of a head, and its pairs' turn fractions.
template <int D>
struct Lane {
  static constexpr int kLanes = D / 8;         // lanes of one head
  static constexpr int kHeads = 32 / kLanes;   // heads of one warp
  int sub, l, off0, off1;
  bool turns;
  uint64_t frac[4];
  __device__ void init(const RopeArgs& a) {
    const int lane = threadIdx.x & 31;
    sub = lane / kLanes;
    l = lane % kLanes;
    turns = 8 * l < a.R;
    const bool split = turns && !a.interleaved;
    off0 = split ? 4 * l : 8 * l;
    off1 = split ? a.R / 2 + 4 * l : 8 * l + 4;
#pragma unroll
    for (int j = 0; j < 4; ++j) frac[j] = turns ? turn_fraction(a.inv_freq[4 * l + j]) : 0;
  }
  __device__ void angles(int pos, float* c, float* s) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) turn_sincos(frac[j], pos, c[j], s[j]);
  }
};

// Turn a lane's eight values; sgn = -1 turns back. A lane outside the rotated part has angle zero.
__device__ __forceinline__ void turn(float* y, const float* c, const float* s, bool interleaved, float sgn) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int ia = interleaved ? 2 * j : j, ib = interleaved ? 2 * j + 1 : j + 4;
    const float ya = y[ia], yb = y[ib], sj = sgn * s[j];
    y[ia] = ya * c[j] - yb * sj;
    y[ib] = yb * c[j] + ya * sj;
  }
}

template <int D>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int m = D / 16; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

__device__ __forceinline__ void load8(const float* w, int off0, int off1, float* x) {
  const float4 a = __ldg(reinterpret_cast<const float4*>(w + off0)), b = __ldg(reinterpret_cast<const float4*>(w + off1));
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
  x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}

// One warp takes a share of one token's heads (shares interleave: share p takes the head groups p,
// p + split, ...). HBM-bound: each element is read and written once.
template <typename T, int D, bool kPages, bool kInter>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a) {
  const long long unit = (long long)blockIdx.x * kWarps + (threadIdx.x >> 5);
  const long long tokens = (long long)a.B * a.N;
  if (unit >= tokens * a.split) return;
  const long long token = unit / a.split;
  const int share = (int)(unit - token * a.split);
  Lane<D> ln;
  ln.init(a);
  const int pos = __ldg(a.pos + token);
  float c[4], s[4], qw[8], kw[8];
  ln.angles(pos, c, s);
  load8(a.q_w, ln.off0, ln.off1, qw);
  load8(a.k_w, ln.off0, ln.off1, kw);
  const int heads = a.Hq + (kPages ? 2 : 1) * a.Hk;
  const int groups = (heads + Lane<D>::kHeads - 1) / Lane<D>::kHeads;
  long long slot = -1;   // the position's slot in the pages laid end to end
  if (kPages) {
    const int b = (int)(token / a.N), i = (int)(token - (long long)b * a.N);
    const int n = a.lengths ? __ldg(a.lengths + b) : a.N;
    const int ctx = __ldg(a.ctx + b);
    if (n < 0 || n > a.N || ctx < 0 || (long long)ctx + n > (long long)a.M * a.page) {
      if ((threadIdx.x & 31) == 0) atomicCAS(a.err, 0, kErrDeviceIndex);
    } else if (i < n) {
      const int at = ctx + i;
      const int pg = __ldg(a.table + (long long)b * a.M + at / a.page);
      if (pg < 0 || pg >= a.P) {
        if ((threadIdx.x & 31) == 0) atomicCAS(a.err, 0, kErrDeviceIndex);
      } else {
        slot = (long long)pg * a.page + at % a.page;
      }
    }
  }
  for (int g0 = share; g0 < groups; g0 += a.split * kUnroll) {
    Raw<T> raw[kUnroll][2];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int head = (g0 + u * a.split) * Lane<D>::kHeads + ln.sub;
      if (head >= heads) continue;
      const T* src = head < a.Hq ? static_cast<const T*>(a.q) + token * a.q_tok + head * a.q_head
                     : (!kPages || head < a.Hq + a.Hk)
                         ? static_cast<const T*>(a.k) + token * a.k_tok + (head - a.Hq) * a.k_head
                         : static_cast<const T*>(a.v) + token * a.v_tok + (head - a.Hq - a.Hk) * a.v_head;
      raw[u][0].load(src + ln.off0);
      raw[u][1].load(src + ln.off1);
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int head = (g0 + u * a.split) * Lane<D>::kHeads + ln.sub;
      if ((g0 + u * a.split) * Lane<D>::kHeads >= heads) break;   // the same in every lane
      const bool live = head < heads;
      float y[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (live) {
        raw[u][0].get(y);
        raw[u][1].get(y + 4);
      }
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(y[e], y[e], ss);
      ss = head_sum<D>(ss);
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      const bool is_q = head < a.Hq;
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = (is_q ? qw[e] : kw[e]) * y[e] * r;
      if (ln.turns) turn(y, c, s, kInter, 1.f);
      if (!live) continue;
      if (is_q) {
        T* out = static_cast<T*>(a.q_out) + (token * a.Hq + head) * D;
        Raw<T>::put(out + ln.off0, y);
        Raw<T>::put(out + ln.off1, y + 4);
      } else if (!kPages) {
        T* out = static_cast<T*>(a.k_out) + (token * a.Hk + head - a.Hq) * D;
        Raw<T>::put(out + ln.off0, y);
        Raw<T>::put(out + ln.off1, y + 4);
      } else if (slot >= 0) {
        if (head < a.Hq + a.Hk) {
          T* out = static_cast<T*>(a.k_pages) + (slot * a.Hk + head - a.Hq) * D;
          Raw<T>::put(out + ln.off0, y);
          Raw<T>::put(out + ln.off1, y + 4);
        } else {
          T* out = static_cast<T*>(a.v_pages) + (slot * a.Hk + head - a.Hq - a.Hk) * D;
          raw[u][0].copy(out + ln.off0);
          raw[u][1].copy(out + ln.off1);
        }
      }
    }
  }
}

constexpr int kBwdBlocks = kNumSMs * 4;   // blocks of the gradient, and rows of its partial sums

// Gradient, with dy = R^T dout and r = 1 / sqrt(mean(x^2) + eps):
//   dx = r (w dy - x r^2 mean(w dy x)),  dw = sum over tokens and heads of dy x r.
// Blocks walk the (token, share) units; a lane keeps the weight gradients of its eight elements in
// registers over all its units, the block adds its lanes in a fixed order and writes one row of
// partial sums [block][q | k][D], which the second kernel adds in order: no atomics, the same bits
// every time.
template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_bwd_kernel(const RopeArgs a) {
  Lane<D> ln;
  ln.init(a);
  float qw[8], kw[8], gq[8], gk[8];
  load8(a.q_w, ln.off0, ln.off1, qw);
  load8(a.k_w, ln.off0, ln.off1, kw);
#pragma unroll
  for (int e = 0; e < 8; ++e) gq[e] = gk[e] = 0.f;
  const int warp = threadIdx.x >> 5;
  const long long units = (long long)a.B * a.N * a.split;
  const int heads = a.Hq + a.Hk;
  const int groups = (heads + Lane<D>::kHeads - 1) / Lane<D>::kHeads;
  for (long long unit = (long long)blockIdx.x * kWarps + warp; unit < units; unit += (long long)gridDim.x * kWarps) {
    const long long token = unit / a.split;
    const int share = (int)(unit - token * a.split);
    float c[4], s[4];
    ln.angles(__ldg(a.pos + token), c, s);
    for (int g0 = share; g0 < groups; g0 += a.split * 2) {
      Raw<T> rx[2][2], rd[2][2];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int head = (g0 + u * a.split) * Lane<D>::kHeads + ln.sub;
        if (head >= heads) continue;
        const bool is_q = head < a.Hq;
        const T* src = is_q ? static_cast<const T*>(a.q) + token * a.q_tok + head * a.q_head
                            : static_cast<const T*>(a.k) + token * a.k_tok + (head - a.Hq) * a.k_head;
        const T* dsrc = is_q ? static_cast<const T*>(a.dq_out) + (token * a.Hq + head) * D
                             : static_cast<const T*>(a.dk_out) + (token * a.Hk + head - a.Hq) * D;
        rx[u][0].load(src + ln.off0);
        rx[u][1].load(src + ln.off1);
        rd[u][0].load(dsrc + ln.off0);
        rd[u][1].load(dsrc + ln.off1);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int head = (g0 + u * a.split) * Lane<D>::kHeads + ln.sub;
        if ((g0 + u * a.split) * Lane<D>::kHeads >= heads) break;   // the same in every lane
        const bool live = head < heads, is_q = head < a.Hq;
        float x[8], dy[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = dy[e] = 0.f;
        if (live) {
          rx[u][0].get(x);
          rx[u][1].get(x + 4);
          rd[u][0].get(dy);
          rd[u][1].get(dy + 4);
        }
        if (ln.turns) turn(dy, c, s, kInter, -1.f);
        float ss = 0.f, dot = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          ss = fmaf(x[e], x[e], ss);
          dot = fmaf((is_q ? qw[e] : kw[e]) * dy[e], x[e], dot);
        }
        ss = head_sum<D>(ss);
        dot = head_sum<D>(dot);
        if (!live) continue;
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        const float m = dot * (1.f / D) * r * r;
        float dx[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          dx[e] = r * ((is_q ? qw[e] : kw[e]) * dy[e] - x[e] * m);
          const float g = dy[e] * x[e] * r;
          if (is_q) gq[e] += g;
          else gk[e] += g;
        }
        float* out = is_q ? a.dq + (token * a.Hq + head) * D : a.dk + (token * a.Hk + head - a.Hq) * D;
        Raw<float>::put(out + ln.off0, dx);
        Raw<float>::put(out + ln.off1, dx + 4);
      }
    }
  }
  // the block's sum: lanes of equal elements within a warp, then the warps in order
  __shared__ float acc[kWarps][2 * D];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
#pragma unroll
    for (int m = 16; m >= Lane<D>::kLanes; m >>= 1) {
      gq[e] += __shfl_xor_sync(0xffffffffu, gq[e], m);
      gk[e] += __shfl_xor_sync(0xffffffffu, gk[e], m);
    }
    if (ln.sub == 0) {
      const int off = (e < 4 ? ln.off0 : ln.off1) + (e & 3);
      acc[warp][off] = gq[e];
      acc[warp][D + off] = gk[e];
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
    float sum = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) sum += acc[w][i];
    a.partial[(long long)blockIdx.x * 2 * D + i] = sum;
  }
}

// dw: 32 lanes add a column's partial rows (lane l rows l, l + 32, ...), then the lanes by a fixed tree.
__global__ void __launch_bounds__(1024) qk_norm_rope_bwd_join_kernel(const float* partial, int rows, int D, float* dq_w,
                                                                     float* dk_w) {
  __shared__ float tile[32][33];
  const int col = blockIdx.x * 32 + (threadIdx.x & 31), part = threadIdx.x >> 5;
  float sum = 0.f;
  for (int r = part; r < rows; r += 32) sum += partial[(long long)r * 2 * D + col];
  tile[part][threadIdx.x & 31] = sum;
  __syncthreads();
  sum = tile[threadIdx.x & 31][part];   // warp `part` adds column blockIdx.x * 32 + part
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  if ((threadIdx.x & 31) == 0) {
    const int c = blockIdx.x * 32 + part;
    if (c < D) dq_w[c] = sum;
    else dk_w[c - D] = sum;
  }
}

template <typename T, int D>
cudaError_t forward(RopeArgs& a, cudaStream_t s) {
  const int heads = a.Hq + (a.k_pages ? 2 : 1) * a.Hk;
  const int groups = (heads + Lane<D>::kHeads - 1) / Lane<D>::kHeads;
  const long long tokens = (long long)a.B * a.N;
  // shares of a token: enough warps to fill the GPU (48 a SM) when tokens are few, and about eight
  // head groups a warp when they are many (the angles are formed once per share)
  const long long fill = (kNumSMs * 48 + tokens - 1) / tokens;
  const int want = (int)(fill > (groups + 7) / 8 ? fill : (groups + 7) / 8);
  a.split = want < groups ? want : groups;
  const long long blocks = (tokens * a.split + kWarps - 1) / kWarps;
  const int slot = stage_timer_begin(s, kKernQkNormRope);
  if (a.k_pages) {
    if (a.interleaved) qk_norm_rope_kernel<T, D, true, true><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    else qk_norm_rope_kernel<T, D, true, false><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  } else {
    if (a.interleaved) qk_norm_rope_kernel<T, D, false, true><<<(unsigned)blocks, kThreads, 0, s>>>(a);
    else qk_norm_rope_kernel<T, D, false, false><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  stage_timer_end(slot, s);
  return e;
}

template <typename T, int D>
cudaError_t backward(RopeArgs& a, cudaStream_t s) {
  const int groups = (a.Hq + a.Hk + Lane<D>::kHeads - 1) / Lane<D>::kHeads;
  const long long tokens = (long long)a.B * a.N;
  const long long fill = (kBwdBlocks * kWarps + tokens - 1) / tokens;
  a.split = (int)(fill < groups ? fill : groups);
  long long blocks = (tokens * a.split + kWarps - 1) / kWarps;
  if (blocks > kBwdBlocks) blocks = kBwdBlocks;
  const int slot = stage_timer_begin(s, kKernQkNormRopeBwd);
  if (a.interleaved) qk_norm_rope_bwd_kernel<T, D, true><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  else qk_norm_rope_bwd_kernel<T, D, false><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess) {
    qk_norm_rope_bwd_join_kernel<<<2 * D / 32, 1024, 0, s>>>(a.partial, (int)blocks, D, a.dq_w, a.dk_w);
    e = cudaGetLastError();
  }
  stage_timer_end(slot, s);
  return e;
}

}  // namespace

size_t qk_norm_rope_backward_workspace_bytes(int D) { return (size_t)kBwdBlocks * 2 * D * sizeof(float); }

cudaError_t launch_qk_norm_rope(RopeArgs a, cudaStream_t s) {
  switch (a.D) {
    case 64: return a.bf16 ? forward<__nv_bfloat16, 64>(a, s) : forward<float, 64>(a, s);
    case 128: return a.bf16 ? forward<__nv_bfloat16, 128>(a, s) : forward<float, 128>(a, s);
    default: return a.bf16 ? forward<__nv_bfloat16, 256>(a, s) : forward<float, 256>(a, s);
  }
}

cudaError_t launch_qk_norm_rope_backward(RopeArgs a, cudaStream_t s) {
  switch (a.D) {
    case 64: return a.bf16 ? backward<__nv_bfloat16, 64>(a, s) : backward<float, 64>(a, s);
    case 128: return a.bf16 ? backward<__nv_bfloat16, 128>(a, s) : backward<float, 128>(a, s);
    default: return a.bf16 ? backward<__nv_bfloat16, 256>(a, s) : backward<float, 256>(a, s);
  }
}

}  // namespace gdr
