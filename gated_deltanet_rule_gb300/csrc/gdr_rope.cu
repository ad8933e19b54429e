// RMS norm of every query and key head and the rotation by position, in one pass:
//   y = w x / sqrt(mean(x^2) + eps);   pair j of the first R elements turned by pos inv_freq[j];
//   elements R .. D-1 pass through.
// Pairs are (j, j + R/2), or (2j, 2j + 1) when interleaved. Forward (dense outputs, or k and v left
// in a cache's pages) and gradient.
//
// Layout: D/16 lanes hold one head, two runs of eight elements each (in the gradient D/8 lanes, runs of
// four): lane l of the rotated part those at 8 l and R/2 + 8 l, the lanes of the rest likewise. So
// neighbouring lanes read and write neighbouring 16 bytes, and both members of a pair lie in one lane, in
// the half-split form (run against run) and in the interleaved one (neighbours). The head's sum of squares
// is the only exchange (shuffles).
//
// A block takes the heads of one kind (queries, keys, or values to be copied; in the gradient queries and
// then keys) of a few tokens: it forms the tokens' cosines and sines once in shared memory, one entry a
// thread, and its warps then walk the (token, head) rows. Forming them in every warp instead cost a third of
// the instructions.
//
// Angles: pos inv_freq is formed in turns modulo one by 64-bit integer arithmetic (inv_freq / 2 pi as
// a 64-bit binary fraction, times the position, dropping whole turns), to within 2^-31 turn at any 32-bit
// position (half of 2^-32 from the fraction, 2^-32 from the bits dropped behind it); float32 angles would
// be off by 0.06 rad at position 2^20, and float64 arithmetic runs at 1/64 of the float32 rate here. The
// fraction is reduced to an eighth turn before sincospif.
#include <algorithm>
#include <cstring>
#include <type_traits>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdr_serve.h"
#include "ptx.cuh"

namespace gdr {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kPairs = 2048;       // (token, pair) angles of a block
constexpr int kMostTokens = 256;   // tokens of a block
constexpr int kDepth = 4;          // rows of every lane in flight
constexpr int kDepthB = 3;         // the same, gradient

// Two floats in one register pair: the packed operations halve the instructions of this kernel, whose
// issue rate is what bounds it beside HBM.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 pack(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack(F2 x, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x.v)); }
__device__ __forceinline__ F2 mul2(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 neg2(F2 a) { return {a.v ^ 0x8000000080000000ull}; }

// kE (eight or four) consecutive elements in shared memory (staged by asynchronous copies, in pieces V that
// lie kThreads apart).
template <int kE>
__device__ __forceinline__ void get(const __nv_bfloat16* p, F2* x) {
  const auto v = *reinterpret_cast<const std::conditional_t<kE == 8, uint4, uint2>*>(p);
  uint32_t w[kE / 2];
  memcpy(w, &v, sizeof(v));
#pragma unroll
  for (int e = 0; e < kE / 2; ++e) x[e] = pack(__uint_as_float(w[e] << 16), __uint_as_float(w[e] & 0xFFFF0000u));
}
template <int kE>
__device__ __forceinline__ void get(const float* p, F2* x) {
#pragma unroll
  for (int h = 0; h < kE / 4; ++h) {
    const ulonglong2 u = reinterpret_cast<const ulonglong2*>(p)[h * kThreads];
    x[2 * h] = {u.x};
    x[2 * h + 1] = {u.y};
  }
}
// Eight elements to memory; four of the gradient's.
__device__ __forceinline__ void put(__nv_bfloat16* p, const F2* x) {
  uint32_t w[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float lo, hi;
    unpack(x[e], lo, hi);
    w[e] = ptx::pack_bf16x2(lo, hi);
  }
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// (32 bytes in one store: two of 16 would each write half of every sector)
__device__ __forceinline__ void put(float* p, const F2* x) {
  if ((reinterpret_cast<uintptr_t>(p) & 31) == 0) {
    asm volatile("st.global.v4.b64 [%0], {%1, %2, %3, %4};" ::"l"(p), "l"(x[0].v), "l"(x[1].v), "l"(x[2].v), "l"(x[3].v) : "memory");
  } else {
    reinterpret_cast<ulonglong2*>(p)[0] = make_ulonglong2(x[0].v, x[1].v);
    reinterpret_cast<ulonglong2*>(p)[1] = make_ulonglong2(x[2].v, x[3].v);
  }
}

__device__ __forceinline__ void put4(float* p, const F2* x) { *reinterpret_cast<ulonglong2*>(p) = make_ulonglong2(x[0].v, x[1].v); }

// A thread's own ring in shared memory: kDepth rows of kPieces pieces V, piece p of every thread side
// by side. Only the thread that copied a piece reads it, so a wait for its own copies is all it needs; the
// copies hold no registers, which is what bounded the rows in flight.
template <int kPieces, int kDepth, typename V>
struct Ring {
  V* mine;
  __device__ __forceinline__ explicit Ring(void* smem) : mine(static_cast<V*>(smem) + threadIdx.x) {}
  __device__ __forceinline__ V* at(int slot, int piece) const { return mine + (slot * kPieces + piece) * kThreads; }
  // n pieces from src into pieces first, first + 1, ...
  template <int n>
  __device__ __forceinline__ void copy(int slot, int first, const void* src) const {
#pragma unroll
    for (int e = 0; e < n; ++e) {
      if (sizeof(V) == 16)
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(ptx::smem_u32(at(slot, first + e))),
                     "l"(static_cast<const V*>(src) + e)
                     : "memory");
      else
        asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(ptx::smem_u32(at(slot, first + e))),
                     "l"(static_cast<const V*>(src) + e)
                     : "memory");
    }
  }
  template <typename T>
  __device__ __forceinline__ const T* row(int slot, int piece) const { return reinterpret_cast<const T*>(at(slot, piece)); }
};

__device__ __forceinline__ int exponent(double f) { return (int)(((uint64_t)__double_as_longlong(f) >> 52) & 0x7FF) - 1023; }

// f / (2 pi) modulo one as a 64-bit binary fraction, from the bits of the double, to within one unit: a
// product with enough digits of 1 / (2 pi) that those of the whole turns can be dropped (the argument
// reduction of Payne and Hanek, 1983). 1 / (2 pi) = C 2^-66 with C = 2^65 / pi, and |f| = m 2^(e - 63), so
// the fraction is m C 2^-64 2^(e - 1) modulo 2^64 (e = exponent(f)).
// kFar: any |f| < 2^62; otherwise |f| < 4.
template <bool kFar>
__device__ __forceinline__ uint64_t turn_fraction(double f) {
  const uint64_t bits = (uint64_t)__double_as_longlong(f);
  const int e = exponent(f), sh = e - 1;
  const uint64_t m = (bits << 11) | 0x8000000000000000ull;
  uint64_t r;
  if (kFar && sh > 0) {   // the bits shifted in come from 64 more bits of C, rounded
    const uint64_t c1 = 0xA2F9836E4E441529ull, c0 = 0xFC2757D1F534DDC1ull;
    const uint64_t mid = m * c1, low = mid + __umul64hi(m, c0);
    const uint64_t high = __umul64hi(m, c1) + (low < mid);
    r = (high << sh) | (low >> (64 - sh));
  } else {                // C rounded; zero and what is below 2^-64 turn per position: 0
    const uint64_t t = __umul64hi(m, 0xA2F9836E4E44152Aull);
    r = sh > -64 ? t >> (-sh & 63) : 0;
  }
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

// What a lane holds of a head: two runs of kE elements.
template <int D, int kE>
struct Lane {
  static constexpr int kLanes = D / (2 * kE);  // lanes of one head
  static constexpr int kHeads = 32 / kLanes;   // rows of one warp
  int sub, l, off0, off1;
  bool turns;
  __device__ __forceinline__ explicit Lane(const RopeArgs& a) {
    const int lane = threadIdx.x & 31;
    sub = lane / kLanes;
    l = lane % kLanes;
    turns = 2 * kE * l < a.R;
    const int first = turns ? kE * l : a.R + kE * (l - a.R / (2 * kE));
    off0 = first;
    off1 = first + (turns ? a.R : D - a.R) / 2;
  }
};

// cos and sin of a block's tokens [t0, t0 + n) into cs, R floats a token.
template <int kE>
__device__ __forceinline__ void form_angles(const RopeArgs& a, long long t0, int n, float* cs) {
  const int half = a.R / 2;
  // runs of [lane][4]: the lanes' first four cosines, (kE = 8) their last four, then sines, so that the
  // lanes of a head read neighbouring 16 bytes. Pair j is entry e of lane l: half-split j = kE l + e;
  // interleaved j = kE/2 l + e in a lane's first run, R/4 + kE/2 l + e - kE/2 in its second
  auto put_angle = [&](int t, int j, float c, float s) {
    int l = j / kE, e = j % kE;
    if (a.interleaved) {
      const int second = 4 * j >= a.R, k = second ? j - a.R / 4 : j;
      l = k / (kE / 2);
      e = kE / 2 * second + k % (kE / 2);
    }
    float* at = cs + t * a.R + (e >> 2) * (2 * a.R / kE) + l * 4 + (e & 3);
    at[0] = c;
    at[a.R / 2] = s;
  };
  bool far = false;
  for (int x = threadIdx.x; x < n * half; x += kThreads) {
    const int t = x / half, j = x - t * half;
    const double f = __ldg(a.inv_freq + j);
    far |= exponent(f) >= 2;
    float c, s;
    turn_sincos(turn_fraction<false>(f), __ldg(a.pos + t0 + t), c, s);
    put_angle(t, j, c, s);
  }
  // a thread that met 4 rad per position or more (no position encoding's frequency) forms those angles again.
  // With the choice in the loop above 8192 tokens of 32 + 8 heads took 36.4 us instead of 33.3
  if (!far) return;
#pragma unroll 1
  for (int x = threadIdx.x; x < n * half; x += kThreads) {
    const int t = x / half, j = x - t * half;
    const double f = __ldg(a.inv_freq + j);
    if (exponent(f) < 2) continue;
    float c = NAN, s = NAN;   // 2^62 and more, infinite or nan: no angle
    if (exponent(f) < 62) turn_sincos(turn_fraction<true>(f), __ldg(a.pos + t0 + t), c, s);
    put_angle(t, j, c, s);
  }
}

// A lane's pairs' cosines and sines, packed two by two.
template <int kE>
__device__ __forceinline__ void read_angles(const float* cs, int R, int l, F2* c, F2* s) {
  const ulonglong2* at = reinterpret_cast<const ulonglong2*>(cs) + l;
#pragma unroll
  for (int q = 0; q < kE / 4; ++q) {
    const ulonglong2 cv = at[q * (R / (2 * kE))], sv = at[(q + kE / 4) * (R / (2 * kE))];
    c[2 * q] = {cv.x};
    c[2 * q + 1] = {cv.y};
    s[2 * q] = {sv.x};
    s[2 * q + 1] = {sv.y};
  }
}

// Turn a lane's 2 kE values (kE packed pairs) by its angles; kBack turns back.
template <int kE, bool kInter, bool kBack>
__device__ __forceinline__ void turn(F2* y, const float* cs, int R, int l) {
  F2 c[kE / 2], s[kE / 2];
  read_angles<kE>(cs, R, l, c, s);
  if (kInter) {   // (y_2j, y_2j+1) are the members of pair j
#pragma unroll
    for (int q = 0; q < kE / 2; ++q) {
      float c0, c1, s0, s1;
      unpack(c[q], c0, c1);
      unpack(s[q], s0, s1);
      if (kBack) {
        s0 = -s0;
        s1 = -s1;
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float ya, yb;
        unpack(y[2 * q + u], ya, yb);
        const float cj = u ? c1 : c0, sj = u ? s1 : s0;
        y[2 * q + u] = pack(ya * cj - yb * sj, yb * cj + ya * sj);
      }
    }
  } else {        // y[q] holds the first members of pairs 2q and 2q + 1, y[kE/2 + q] the second ones
#pragma unroll
    for (int q = 0; q < kE / 2; ++q) {
      const F2 ya = y[q], yb = y[kE / 2 + q], sq = kBack ? neg2(s[q]) : s[q];
      y[q] = fma2(ya, c[q], neg2(mul2(yb, sq)));
      y[kE / 2 + q] = fma2(yb, c[q], mul2(ya, sq));
    }
  }
}

template <int kLanes>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int m = kLanes / 2; m >= 1; m >>= 1) v += __shfl_xor_sync(0xffffffffu, v, m);
  return v;
}

template <int kE>
__device__ __forceinline__ void load_weights(const float* w, int off0, int off1, F2* x) {
#pragma unroll
  for (int q = 0; q < kE / 4; ++q) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(w + off0) + q), b = __ldg(reinterpret_cast<const float4*>(w + off1) + q);
    x[2 * q] = pack(a.x, a.y);
    x[2 * q + 1] = pack(a.z, a.w);
    x[kE / 2 + 2 * q] = pack(b.x, b.y);
    x[kE / 2 + 2 * q + 1] = pack(b.z, b.w);
  }
}

// The (token, head) row `x` of a block's tokens: token and head by one multiplication.
__device__ __forceinline__ void row_at(int x, int H, uint32_t magic, int& t, int& h) {
  t = (int)__umulhi((uint32_t)x, magic);
  h = x - t * H;
  if (h >= H) {   // (magic = floor(2^32 / H): the quotient may be one short)
    h -= H;
    ++t;
  }
}

// One kind of heads of a block's tokens: their strides, weights and destination.
template <typename T>
struct Kind {
  const T* src;
  long long tok, head;
  const float* w;
  T* out;          // dense rows, or the pages
  int H, tokens;   // heads; tokens of a block
};

// Normed, turned and written (kPages: keys into the pages, values copied there). HBM-bound: each element
// is read and written once; every lane has kDepth rows in flight in shared memory. Measured: 8192 tokens of
// 32 + 8 heads of 128, bfloat16: 31.8 us a call among others, 78% of the copy bandwidth. As a replayed graph
// 33.3 us, a plain copy of as many bytes 28.9. (When it took 34.1: with the rows loaded into registers and
// lanes 32 bytes apart 37.6, with blocks that walk both kinds, as the gradient's do, 36.5.)
template <typename T, int D, bool kPages, bool kInter>
__global__ void __launch_bounds__(kThreads) qk_norm_rope_kernel(const RopeArgs a) {
  constexpr int kRun = 8 * sizeof(T) / 16, kPieces = 2 * kRun;   // 16-byte pieces of a run, of a lane's row
  extern __shared__ __align__(16) uint8_t stage[];
  __shared__ __align__(16) float cs[2 * kPairs];
  __shared__ long long slot[kMostTokens];
  const Ring<kPieces, kDepth, uint4> ring(stage);
  using Ln = Lane<D, 8>;
  const Ln ln(a);
  const long long tokens = (long long)a.B * a.N;
  const int kind = blockIdx.x < a.blocks[0] ? 0 : blockIdx.x < a.blocks[0] + a.blocks[1] ? 1 : 2;
  const long long block = blockIdx.x - (kind == 0 ? 0 : kind == 1 ? a.blocks[0] : a.blocks[0] + a.blocks[1]);
  Kind<T> k;
  if (kind == 0) k = {static_cast<const T*>(a.q), a.q_tok, a.q_head, a.q_w, static_cast<T*>(a.q_out), a.Hq, a.tokens[0]};
  else if (kind == 1)
    k = {static_cast<const T*>(a.k), a.k_tok, a.k_head, a.k_w, static_cast<T*>(kPages ? a.k_pages : a.k_out), a.Hk, a.tokens[1]};
  else k = {static_cast<const T*>(a.v), a.v_tok, a.v_head, nullptr, static_cast<T*>(a.v_pages), a.Hk, a.tokens[1]};
  const long long t0 = block * k.tokens;
  const int n = (int)min((long long)k.tokens, tokens - t0), rows = n * k.H;
  const uint32_t magic = k.H == 1 ? 0xFFFFFFFFu : (uint32_t)((1ull << 32) / k.H);
  const int warp = threadIdx.x >> 5, step = kWarps * Ln::kHeads;
  const bool to_pages = kPages && kind > 0;

  const T* base = k.src + t0 * k.tok;
  const int tok = (int)k.tok, head = (int)k.head;
  // the first rows are on their way while the angles are formed
  auto load = [&](int u, int x) {
    if (x < rows) {
      int t, h;
      row_at(x, k.H, magic, t, h);
      const T* src = base + (t * tok + h * head);   // (below 2^31: tokens of a block <= 256)
      ring.template copy<kRun>(u, 0, src + ln.off0);
      ring.template copy<kRun>(u, kRun, src + ln.off1);
    }
    ptx::cp_async_commit();
  };
  const int x0 = warp * Ln::kHeads + ln.sub;
#pragma unroll
  for (int u = 0; u < kDepth; ++u) load(u, x0 + u * step);
  F2 w[8];
  if (kind < 2) {
    load_weights<8>(k.w, ln.off0, ln.off1, w);
    form_angles<8>(a, t0, n, cs);
  }
  if (to_pages) {
    for (int t = threadIdx.x; t < n; t += kThreads) {
      const int b = (int)((t0 + t) / a.N), i = (int)(t0 + t - (long long)b * a.N);
      const int len = a.lengths ? __ldg(a.lengths + b) : a.N, ctx = __ldg(a.ctx + b);
      long long at = -1;   // the position's slot in the pages laid end to end
      if (len < 0 || len > a.N || ctx < 0 || (long long)ctx + len > (long long)a.M * a.page) {
        atomicCAS(a.err, 0, kErrDeviceIndex);
      } else if (i < len) {
        const int pos = ctx + i, pg = __ldg(a.table + (long long)b * a.M + pos / a.page);
        if (pg < 0 || pg >= a.P) atomicCAS(a.err, 0, kErrDeviceIndex);
        else at = (long long)pg * a.page + pos % a.page;
      }
      slot[t] = at;   // (-1: h is below H, so -H + h stays negative)
    }
  }
  __syncthreads();
  int u = 0;
  for (int xw = warp * Ln::kHeads; xw < rows; xw += step, u = u + 1 == kDepth ? 0 : u + 1) {   // the same in every lane
    const int x = xw + ln.sub;
    const bool live = x < rows;
    int t, h;
    row_at(live ? x : rows - 1, k.H, magic, t, h);
    const long long first = to_pages ? slot[t] * k.H + h : t0 * k.H + x;
    T* out = k.out + first * D;
    const bool write = live && first >= 0;
    ptx::cp_async_wait<kDepth - 1>();
    if (kPages && kind == 2) {
      if (write) {
#pragma unroll
        for (int e = 0; e < kRun; ++e) {
          reinterpret_cast<uint4*>(out + ln.off0)[e] = *ring.at(u, e);
          reinterpret_cast<uint4*>(out + ln.off1)[e] = *ring.at(u, kRun + e);
        }
      }
    } else {
      F2 y[8];
      get<8>(ring.template row<T>(u, 0), y);
      get<8>(ring.template row<T>(u, kRun), y + 4);
      F2 sq = mul2(y[0], y[0]);
#pragma unroll
      for (int e = 1; e < 8; ++e) sq = fma2(y[e], y[e], sq);
      float s0, s1;
      unpack(sq, s0, s1);
      const float ss = head_sum<Ln::kLanes>(live ? s0 + s1 : 0.f);
      const float r = rsqrtf(ss * (1.f / D) + a.eps);
      const F2 rr = pack(r, r);
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = mul2(mul2(w[e], y[e]), rr);
      if (ln.turns) turn<8, kInter, false>(y, cs + t * a.R, a.R, ln.l);
      if (write) {
        put(out + ln.off0, y);
        put(out + ln.off1, y + 4);
      }
    }
    load(u, x + kDepth * step);
  }
}

constexpr int kPerSM = 4;                       // blocks of the gradient on each SM
constexpr int kBwdBlocks = kNumSMs * kPerSM;   // blocks of the gradient (one wave), and rows of its partial sums, at most

// Gradient, with dy = R^T dout and r = 1 / sqrt(mean(x^2) + eps):
//   dx = r (w dy - x r^2 mean(w dy x)),  dw = sum over tokens and heads of dy x r.
// As the forward, but lanes hold half as much, and a block walks the queries of its tokens and then their
// keys, keeping the weight gradients of a lane's eight elements in registers; it adds its lanes in a fixed
// order and writes a row of partial sums of each kind, which the second kernel adds in order: no atomics, the
// same bits every time. Measured: 3 x 2731 tokens of 16 + 2 heads of 256, bfloat16: 57.6 us a call among
// others, 77% of the copy bandwidth. As a replayed graph 58.1 us (a plain copy of as many bytes 48.6; with
// blocks of one kind each, whose work was uneven, 65.6; with sixteen elements a lane and half the warps
// besides, 67.7).
template <typename T, int D, bool kInter>
__global__ void __launch_bounds__(kThreads, kPerSM) qk_norm_rope_bwd_kernel(const RopeArgs a) {
  using V = std::conditional_t<sizeof(T) == 2, uint2, uint4>;   // a run of four elements
  using Ln = Lane<D, 4>;
  extern __shared__ __align__(16) uint8_t stage[];
  __shared__ __align__(16) float cs[2 * kPairs];
  __shared__ float acc[kWarps][D];
  const Ring<4, kDepthB, V> ring(stage);   // x and dy, two runs each
  const Ln ln(a);
  const long long tokens = (long long)a.B * a.N;
  const int warp = threadIdx.x >> 5, step = kWarps * Ln::kHeads, per = a.tokens[1], most = a.tokens[0];
  const long long begin = (long long)blockIdx.x * per, end = min(tokens, begin + per);
#pragma unroll 1
  for (int kind = 0; kind < 2; ++kind) {
    const bool is_q = kind == 0;
    const T* src = static_cast<const T*>(is_q ? a.q : a.k);
    const T* dsrc = static_cast<const T*>(is_q ? a.dq_out : a.dk_out);
    float* dst = is_q ? a.dq : a.dk;
    const long long tok = is_q ? a.q_tok : a.k_tok, head = is_q ? a.q_head : a.k_head;
    const int H = is_q ? a.Hq : a.Hk;
    const uint32_t magic = H == 1 ? 0xFFFFFFFFu : (uint32_t)((1ull << 32) / H);
    F2 w[4], g[4];
    load_weights<4>(is_q ? a.q_w : a.k_w, ln.off0, ln.off1, w);
#pragma unroll
    for (int e = 0; e < 4; ++e) g[e] = {0};
    for (long long t0 = begin; t0 < end; t0 += most) {
      const int n = (int)min((long long)most, end - t0), rows = n * H;
      auto load = [&](int u, int x) {
        if (x < rows) {
          int t, h;
          row_at(x, H, magic, t, h);
          const T* s = src + t0 * tok + (t * (int)tok + h * (int)head);
          const T* d = dsrc + (t0 * H + x) * D;
          ring.template copy<1>(u, 0, s + ln.off0);
          ring.template copy<1>(u, 1, s + ln.off1);
          ring.template copy<1>(u, 2, d + ln.off0);
          ring.template copy<1>(u, 3, d + ln.off1);
        }
        ptx::cp_async_commit();
      };
#pragma unroll
      for (int u = 0; u < kDepthB; ++u) load(u, (warp + u * kWarps) * Ln::kHeads + ln.sub);
      if (kind == 0 || end - begin > most) {   // (the keys' angles are there already where one run holds them)
        __syncthreads();   // the run before has been walked
        form_angles<4>(a, t0, n, cs);
      }
      __syncthreads();
      int u = 0;
      for (int xw = warp * Ln::kHeads; xw < rows; xw += step, u = u + 1 == kDepthB ? 0 : u + 1) {   // the same in every lane
        const int x = xw + ln.sub;
        const bool live = x < rows;
        int t, h;
        row_at(live ? x : rows - 1, H, magic, t, h);
        ptx::cp_async_wait<kDepthB - 1>();
        F2 y[4], dy[4];
        get<4>(ring.template row<T>(u, 0), y);
        get<4>(ring.template row<T>(u, 1), y + 2);
        get<4>(ring.template row<T>(u, 2), dy);
        get<4>(ring.template row<T>(u, 3), dy + 2);
        load(u, x + kDepthB * step);
        if (ln.turns) turn<4, kInter, true>(dy, cs + t * a.R, a.R, ln.l);
        F2 sq = mul2(y[0], y[0]), dt = mul2(mul2(w[0], dy[0]), y[0]);
#pragma unroll
        for (int e = 1; e < 4; ++e) {
          sq = fma2(y[e], y[e], sq);
          dt = fma2(mul2(w[e], dy[e]), y[e], dt);
        }
        float s0, s1, d0, d1;
        unpack(sq, s0, s1);
        unpack(dt, d0, d1);
        const float ss = head_sum<Ln::kLanes>(live ? s0 + s1 : 0.f), dot = head_sum<Ln::kLanes>(live ? d0 + d1 : 0.f);
        if (!live) continue;
        const float r = rsqrtf(ss * (1.f / D) + a.eps);
        const float m = -dot * (1.f / D) * r * r;
        const F2 rr = pack(r, r), mm = pack(m, m);
        F2 dx[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          dx[e] = mul2(rr, fma2(y[e], mm, mul2(w[e], dy[e])));
          g[e] = fma2(dy[e], mul2(y[e], rr), g[e]);
        }
        float* out = dst + (t0 * H + x) * D;
        put4(out + ln.off0, dx);
        put4(out + ln.off1, dx + 2);
      }
    }
    // the block's sum: lanes of equal elements within a warp, then the warps in order
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      float g0, g1;
      unpack(g[e], g0, g1);
#pragma unroll
      for (int m = 16; m >= Ln::kLanes; m >>= 1) {
        g0 += __shfl_xor_sync(0xffffffffu, g0, m);
        g1 += __shfl_xor_sync(0xffffffffu, g1, m);
      }
      if (ln.sub == 0) {
        float* at = acc[warp] + (e < 2 ? ln.off0 : ln.off1) + 2 * (e & 1);
        at[0] = g0;
        at[1] = g1;
      }
    }
    __syncthreads();
    for (int i = threadIdx.x; i < D; i += kThreads) {
      float sum = 0.f;
#pragma unroll
      for (int v = 0; v < kWarps; ++v) sum += acc[v][i];
      a.partial[((long long)kind * gridDim.x + blockIdx.x) * D + i] = sum;
    }
  }
}

// dw: a block adds eight columns of one kind's partial rows: a thread every 128th row of one column (all of
// them in flight), then those by a fixed tree.
__global__ void __launch_bounds__(1024) qk_norm_rope_bwd_join_kernel(const RopeArgs a) {
  __shared__ float tile[8][33];
  ptx::wait_prerequisite();
  const int kind = blockIdx.y, rows = a.blocks[0];
  const int col = threadIdx.x & 7, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const float* p = a.partial + (long long)kind * rows * a.D + blockIdx.x * 8 + col;
  float sum = 0.f;
#pragma unroll 8
  for (int r = threadIdx.x >> 3; r < rows; r += 128) sum += p[(long long)r * a.D];
  sum += __shfl_xor_sync(0xffffffffu, sum, 8);
  sum += __shfl_xor_sync(0xffffffffu, sum, 16);
  if (lane < 8) tile[lane][warp] = sum;
  __syncthreads();
  if (warp >= 8) return;   // warp w adds column w
  sum = tile[warp][lane];
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, m);
  if (lane == 0) (kind ? a.dk_w : a.dq_w)[blockIdx.x * 8 + warp] = sum;
}

// Tokens of a block so that its rows come to about `rows`, within the shared memory for angles.
int tokens_of(const RopeArgs& a, int H, long long rows, long long tokens) {
  const int most = a.R > 0 && 2 * kPairs / a.R < kMostTokens ? 2 * kPairs / a.R : kMostTokens;
  long long t = (rows + H - 1) / H;
  if (t > most) t = most;
  if (t > tokens) t = tokens;
  return (int)(t < 1 ? 1 : t);
}
// Rows of a forward block: as many rounds of its lane groups as make one wave of four blocks a SM, so
// that the angles' forming and the ring's filling are spread over them; one round when there are few.
int rows_of(int D, long long rows) {
  const int round = kWarps * (32 / (D / 16));
  const long long wave = (long long)kNumSMs * 4 * round, rounds = (rows + wave - 1) / wave;
  return (int)(rounds > 32 ? 32 : rounds) * round;
}

template <typename T, int D, bool kPages, bool kInter>
cudaError_t launch_rows(const RopeArgs& a, unsigned blocks, cudaStream_t s) {
  constexpr int kSmem = kThreads * 16 * sizeof(T) * kDepth;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(qk_norm_rope_kernel<T, D, kPages, kInter>), kSmem, done);
  if (e != cudaSuccess) return e;
  const int slot = stage_timer_begin(s, kKernQkNormRope);
  qk_norm_rope_kernel<T, D, kPages, kInter><<<blocks, kThreads, kSmem, s>>>(a);
  e = cudaGetLastError();
  stage_timer_end(slot, s);
  return e;
}

template <typename T, int D>
cudaError_t forward(RopeArgs& a, cudaStream_t s) {
  const long long tokens = (long long)a.B * a.N;
  const int rows = rows_of(D, tokens * (a.Hq + (a.k_pages ? 2 : 1) * a.Hk));
  a.tokens[0] = tokens_of(a, a.Hq, rows, tokens);
  a.tokens[1] = tokens_of(a, a.Hk, rows, tokens);
  a.blocks[0] = (int)((tokens + a.tokens[0] - 1) / a.tokens[0]);
  a.blocks[1] = (int)((tokens + a.tokens[1] - 1) / a.tokens[1]);
  const unsigned blocks = a.blocks[0] + (a.k_pages ? 2 : 1) * a.blocks[1];
  if (a.k_pages) return a.interleaved ? launch_rows<T, D, true, true>(a, blocks, s) : launch_rows<T, D, true, false>(a, blocks, s);
  return a.interleaved ? launch_rows<T, D, false, true>(a, blocks, s) : launch_rows<T, D, false, false>(a, blocks, s);
}

template <typename T, int D, bool kInter>
cudaError_t backward_of(RopeArgs& a, cudaStream_t s) {
  const long long tokens = (long long)a.B * a.N;
  // one wave of blocks, each with one run of tokens, or several where a run's angles do not fit (not under
  // a round of the block's lane groups: a block's start costs more than its rows)
  long long per = (tokens + kBwdBlocks - 1) / kBwdBlocks;
  const long long least = (kWarps * Lane<D, 4>::kHeads + a.Hq - 1) / a.Hq;
  per = std::min(std::max(per, least), tokens);
  a.tokens[0] = tokens_of(a, a.Hq, per * a.Hq, tokens);
  a.tokens[1] = (int)per;
  const unsigned blocks = a.blocks[0] = (int)((tokens + per - 1) / per);
  constexpr int kSmem = kThreads * 16 * sizeof(T) * kDepthB;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(qk_norm_rope_bwd_kernel<T, D, kInter>), kSmem, done);
  if (e != cudaSuccess) return e;
  const int slot = stage_timer_begin(s, kKernQkNormRopeBwd);
  qk_norm_rope_bwd_kernel<T, D, kInter><<<blocks, kThreads, kSmem, s>>>(a);
  e = cudaGetLastError();
  if (e == cudaSuccess) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(D / 8, 2);
    cfg.blockDim = dim3(1024);
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    e = cudaLaunchKernelEx(&cfg, qk_norm_rope_bwd_join_kernel, a);
  }
  stage_timer_end(slot, s);
  return e;
}

template <typename T, int D>
cudaError_t backward(RopeArgs& a, cudaStream_t s) {
  return a.interleaved ? backward_of<T, D, true>(a, s) : backward_of<T, D, false>(a, s);
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
