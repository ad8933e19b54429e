// Tokens from logits with temperature, top-k, top-p and min-p and given uniform numbers, and the probabilities
// that are left. Per row, with w = e^((l - max) / T) and the tokens in the order of falling logits (equal ones by
// rising index):
//   top-k keeps the first k; top-p of these the tokens with less than p of the mass before them (always the
//   first); min-p of these the ones with w >= min_p. The token is the smallest index whose running sum of the
//   kept w (in index order) passes u times their total; probabilities are w / total, 0 where not kept.
// Every filter keeps the first tokens of the order, so what is kept is a border: a logit, and how many of the
// tokens that equal it (the first by index).
//
// Sums decide whole numbers (which token, where the border lies), and float32 exponentials would decide one
// row in a few hundred otherwise than their exact values. Weights are therefore formed as pairs of floats to about
// 2^-40: x = (l - ref) log2(e) / T less the same of the maximum, as a pair, x = J / 64 + s with the exact remainder s, 2^(J / 64) from a table
// of pairs, 2^s as 1 + a polynomial whose first term is a pair (table and polynomial after Tang, 1989). Products
// with log2(e) / T cancel against the maximum only where that is exact: ref = 0 where |max| log2(e) / T < 300 (the
// pair holds x to 2^-39 then), else ref = max, and logits that matter (150 binary orders: what float32 probabilities
// can show) lie within a factor of two of it, where the difference is exact. Sums are integers in units of 2^-40 of the largest weight.
// bf16: of weights that are each rounded to such a unit, so in any order, and a row has the same bits in any batch. float32: a thread
// adds up its pairs and rounds their sum (to 2^-37 of it), so a total's last units, and with them a token or border that lies that close,
// depend on how many blocks share a row, and this on how many rows there are; only a border's few candidates are added up as integers.
//
// A cluster of blocks holds a row in shared memory, read once. The border is found by counting; all blocks know all counts.
//   bf16: a bin for each value of a magnitude from 2^-8 to 127, counted as the logits arrive, before their largest is known.
//     Count times weight is a bin's exact mass, so the border's value is known at once, and how many of its equals stay (values
//     around zero and large ones, several to a bin, are weighed singly, and looked into if the border lies there). The kept mass
//     is added up through the bins' weights.
//   float32: steps of 1/128 of a binary order below the maximum. For top-k the k-th logit's step, for top-p the steps that the
//     masses' bounds leave (0.5% apart; then one pass over the exact weights, which fixes the mass above them). Their logits,
//     usually some dozens, go to all blocks, which order them and add them up. More than kList / 2 of them (equal logits): 10 bits
//     of the float at a time.
// The token is found warp, 32-unit piece, lane, entry: each a scan over lanes.
//
// Bound by instructions and by the steps' dependence, not by HBM: 256 rows of 131072 bf16 with top-p take 108 us (620 GB/s, issue
// slots 55% busy), where counting is half of a block's time; 96 rows of 131072 float32 with top-p 129 to 131 us (issue 52%), a
// third of a block's time the pass over the exact weights (42 packed operations a pair of logits), and its 768 blocks, of which
// some 256 find room at once, three rounds; 48 rows of 49999 31 to 38 us, one of 32000 18 us: five exchanges between the blocks
// and a dozen dependent steps. Weights relative to the maximum's remainder in the table, 8 operations of 42 fewer, were no faster.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>
#include <type_traits>

#include "gdr_serve.h"
#include "pairs.cuh"
#include "ptx.cuh"

namespace gdr {
namespace {

using namespace pairs;

using bf16 = __nv_bfloat16;
using u64 = unsigned long long;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 1024;
// float32: steps of a binary order in the first histogram, down to 28 orders below the largest weight, and 4 of them farther
// down: a k-th logit there is found as soon as others (the 40th, 40 orders down, of a row of 49999: 32 -> 17 us, with
// top-p 48 -> 17).
constexpr int kPerOctave = 128, kFine = 3584, kPerFar = 4;
constexpr float kFar = (float)kPerFar / kPerOctave;
constexpr float kWidth = 0.99459939f, kCoarse = 0.84089642f;   // a step's least weight over its largest: 2^(-1/128), 2^(-1/4)
constexpr unsigned kAll = 0xffffffffu;
constexpr int kTarget = 100 << 10;  // bytes of a block's part of a row: two blocks an SM

struct Table {
  float2 t[64];   // 2^(k / 64) as pairs
};

// What a row's weights are formed from.
struct Scale {
  float ch, cl;   // log2(e) / T
  float ref;      // subtracted from the logits first
  float least;    // smaller differences count as this one (a weight of 2^-152, of which no probability is left)
  float mh, ml;   // the maximum's product with log2(e) / T, as formed for every logit: its weight is exactly 1
};

// Weights of two logits in units of 2^-40, as unevaluated pairs hi + lo.
struct W2 {
  F2 hi, lo;
};
__device__ __forceinline__ W2 weights(const Scale& s, const float2* table, float l0, float l1) {
  F2 z = add(pack(l0, l1), both(-s.ref));
  {
    float a, b;
    unpack(z, a, b);
    z = pack(fmaxf(a, s.least), fmaxf(b, s.least));
  }
  // the product's negative, and what its rounding left; with the maximum's product: -(d + dl)
  const F2 np = mul(z, both(-s.ch)), pl = fma(z, both(s.cl), fma(z, both(s.ch), np));
  const F2 mh = both(s.mh), nd = add(np, mh), dd = sub(nd, np);
  const F2 dl = sub(add(pl, both(-s.ml)), add(sub(np, sub(nd, dd)), sub(mh, dd)));
  constexpr float kMagic = 196608.f;   // 1.5 2^17: the sum's last place is 1 / 64
  const F2 t = sub(both(kMagic), nd), r = sub(sub(both(kMagic), t), nd);   // r exactly
  const F2 x = add(r, dl), xl = sub(dl, sub(x, r));                        // x + xl = r + dl
  // 2^x - 1 = a + b
  constexpr float kL1 = 0.693147182464599609375f, kL1l = -1.9046542999577679e-9f;   // ln 2 as a pair
  constexpr float kL2 = 0.2402265069591007f, kL3 = 0.05550410866482158f, kL4 = 0.009618129107628477f;
  const F2 a = mul(x, both(kL1));
  F2 b = fma(x, both(kL1), mul(x, both(-kL1)));
  b = fma(x, both(kL1l), b);
  b = fma(xl, both(kL1), b);
  b = fma(mul(x, x), fma(x, fma(x, both(kL4), both(kL3)), both(kL2)), b);
  // times 2^(k / 64) 2^e: th (1 + a) and what its rounding left (th - hi is exact)
  float t0, t1;
  unpack(t, t0, t1);
  const int j0 = __float_as_int(t0) - __float_as_int(kMagic), j1 = __float_as_int(t1) - __float_as_int(kMagic);
  const float2 e0 = table[j0 & 63], e1 = table[j1 & 63];
  const float f0 = __int_as_float((127 + 40 + (j0 >> 6)) << 23), f1 = __int_as_float((127 + 40 + (j1 >> 6)) << 23);
  const F2 th = pack(e0.x, e1.x), tl = pack(e0.y, e1.y), f = pack(f0, f1);
  const F2 hi = fma(th, a, th);
  const F2 lo = add(fma(th, a, sub(th, hi)), fma(th, b, tl));
  return {mul(hi, f), mul(lo, f)};
}
__device__ __forceinline__ u64 fixed(float hi, float lo) { return (u64)(__float2ll_rn(hi) + __float2ll_rn(lo)); }
__device__ __forceinline__ u64 fixed_one(float hi, float lo) { return (u64)(__float2ll_rn(hi) + __float2int_rn(lo)); }   // (one weight's: |lo| < 2^20)
__device__ __forceinline__ u64 weight(const Scale& s, const float2* table, float l) {
  const W2 w = weights(s, table, l, l);
  float h, g, lo;
  unpack(w.hi, h, g);
  unpack(w.lo, lo, g);
  return fixed_one(h, lo);
}
__device__ __forceinline__ void weight(const Scale& s, const float2* table, float l0, float l1, u64& w0, u64& w1) {
  const W2 w = weights(s, table, l0, l1);
  float h0, h1, g0, g1;
  unpack(w.hi, h0, h1);
  unpack(w.lo, g0, g1);
  w0 = fixed_one(h0, g0);
  w1 = fixed_one(h1, g1);
}
// A running sum of pairs.
__device__ __forceinline__ void accumulate(W2& acc, F2 hi, F2 lo) {
  const F2 s = add(acc.hi, hi), bb = sub(s, acc.hi);
  const F2 e = add(sub(acc.hi, sub(s, bb)), sub(hi, bb));
  acc.hi = s;
  acc.lo = add(acc.lo, add(e, lo));
}
__device__ __forceinline__ u64 fixed(const W2& w) {
  float a, b, c, d;
  unpack(w.hi, a, b);
  unpack(w.lo, c, d);
  return fixed(a, c) + fixed(b, d);
}

// a f exactly, rounded up or down; 0 <= f.
__device__ __forceinline__ u64 times(u64 a, float f, bool up) {
  if (f >= 1.f) return a;
  const uint32_t b = __float_as_uint(f), e = b >> 23, m = (b & 0x7FFFFFu) | (e ? 0x800000u : 0u);
  const int shift = 150 - (int)max(1u, e);   // f = m 2^-shift, shift >= 24
  const u64 lo = a * m, hi = __umul64hi(a, m);
  u64 r, rest;
  if (shift < 64) {
    r = (lo >> shift) | (hi << (64 - shift));
    rest = lo << (64 - shift);
  } else {
    r = shift < 128 ? hi >> (shift - 64) : 0;
    rest = lo | (shift == 64 ? 0 : shift < 128 ? hi << (128 - shift) : hi);
  }
  return r + (up && rest ? 1 : 0);
}

// The smallest n <= most with n w >= need (a 64-bit division takes longer than the rest of a search's end).
__device__ __forceinline__ uint32_t least_ties(u64 need, u64 w, uint32_t most) {
  const float q = fminf(__fdividef((float)need, (float)w), 4e6f);
  uint32_t n = (uint32_t)fmaxf(q * (1.f - 0x1p-20f) - 1.f, 0.f);
  while (n < most && n * w < need) ++n;
  return min(n, most);
}

// Floats in order as integers (no nan, one zero).
__device__ __forceinline__ uint32_t key_of(float x) {
  const uint32_t b = __float_as_uint(x);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) { return __uint_as_float(k ^ ((k >> 31) ? 0x80000000u : 0xFFFFFFFFu)); }

// A logit as the rest takes it: nan is -inf, +inf the largest finite value, one zero.
__device__ __forceinline__ float clean(float x) { return x != x ? -INFINITY : fminf(x, FLT_MAX) + 0.f; }
constexpr float kBf16Max = 3.3895313892515355e38f;

// 16 bytes of logits.
template <typename T>
struct Unit;
template <>
struct Unit<float> {
  static constexpr int n = 4;
  static __device__ __forceinline__ void read(const uint4& u, float* x) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y); x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
  static __device__ __forceinline__ uint4 write(const float* x) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
  }
  static __device__ __forceinline__ float one(const float* p) { return *p; }
  // as the rest takes them, and the largest of them and `top`
  static __device__ __forceinline__ uint4 clean_max(const uint4& u, float& top) {
    float x[4];
    read(u, x);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[e] = clean(x[e]);
      top = fmaxf(top, x[e]);
    }
    return write(x);
  }
};
template <>
struct Unit<bf16> {
  static constexpr int n = 8;
  static __device__ __forceinline__ void read(const uint4& u, float* x) {
    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      x[2 * e] = __uint_as_float(v[e] << 16);
      x[2 * e + 1] = __uint_as_float(v[e] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ uint4 write(const float* x) {   // (bf16 values: exact, but for FLT_MAX)
    uint32_t v[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = ptx::pack_bf16x2(fminf(x[2 * e], kBf16Max), fminf(x[2 * e + 1], kBf16Max));
    return make_uint4(v[0], v[1], v[2], v[3]);
  }
  static __device__ __forceinline__ float one(const bf16* p) { return __bfloat162float(*p); }
  static __device__ __forceinline__ uint4 clean_max(const uint4& u, float& top) {   // (-0 stays: only keys tell it from 0)
    // an exponent of all ones carries into the sign's place when one is added to it
    const uint32_t hit = (((u.x & 0x7F807F80u) + 0x00800080u) | ((u.y & 0x7F807F80u) + 0x00800080u) |
                          ((u.z & 0x7F807F80u) + 0x00800080u) | ((u.w & 0x7F807F80u) + 0x00800080u)) & 0x80008000u;
    uint4 r = u;
    if (hit) {
      float x[8];
      read(u, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fminf(clean(x[e]), kBf16Max);
      r = write(x);
    }
    auto two = [](uint32_t w) { return *reinterpret_cast<const __nv_bfloat162*>(&w); };
    const __nv_bfloat162 m = __hmax2(__hmax2(two(r.x), two(r.y)), __hmax2(two(r.z), two(r.w)));
    top = fmaxf(top, fmaxf(__low2float(m), __high2float(m)));
    return r;
  }
};

__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ uint4 ld_cluster4(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared::cluster.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster4(uint32_t addr, const uint4& v) {
  asm volatile("st.shared::cluster.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ __forceinline__ void st_cluster64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

// bf16: a bin for each value of a magnitude from 2^-8 to 127, so that logits are counted as they arrive, before their
// largest is known. v = 0 for smaller magnitudes, 1 .. kTop - 1 by magnitude, kTop for larger ones; a positive value's bin
// lies at ~v, a negative one's at v (modulo 4096), which two packed minima and a mask give for two logits at once. In the
// order of falling logits (steps) they follow one another from kFirstBin on: kTop - v, and kTop + 1 + v for negative ones.
constexpr int kLeast = (127 - 8) << 7;             // the code of 2^-8
constexpr int kTop = 1919;
constexpr int kMiddleStep = kTop;                  // around zero (and the step after it, which is counted with it)
constexpr int kFirstBin = 4095 - kTop;
constexpr float kLarge = 127.f;                    // the magnitude with v = kTop
constexpr int kMaxSteps = 4096;
template <typename T>
struct Bins;
template <>
struct Bins<float> {
  static constexpr int n = kMaxSteps;              // steps of 1 / kPerOctave of a binary order of the weight
};
template <>
struct Bins<bf16> {
  static constexpr int n = 2 * kTop + 2;           // large ones, positive values falling, around zero, negative values, the rest
};

constexpr int kList = 2048;                  // candidates of a row: places, shared out evenly to its blocks
constexpr int kOthers = 256;
constexpr int kDirect = 384;
struct Shared {
  float2 table[64];
  union {
    struct {
      uint4 hist[kBins];                     // counts, and masses in two words: this block's,
      uint4 hist_all[kBins];                 // all blocks'
    };
    struct {
      uint32_t steps[kMaxSteps];             // counts of the first histogram: this block's,
      uint32_t all[kMaxSteps];               // all blocks'
    };
    u64 list[kList];                         // candidates, by block; other blocks write them, while this one may still
                                             // read `all`: they lie over `steps`, which everyone has read by then
    u64 weight[kMaxSteps];                   // bf16: the weight of each bin's value (0: not kept)
  };
  float others[kOthers];                     // bf16: logits around zero
  double min_p;                              // T ln(min_p)
  float tops[kMaxCluster];
  u64 sums[2][3][kMaxCluster];   // the blocks' totals, by turns
  int listed[kMaxCluster];
  u64 warps[kWarps], chunks[kWarps];
  uint32_t equals[kWarps], chunk_equals[kWarps];
  u64 scan_m[kWarps];
  float scan_f[kWarps];
  uint32_t scan_n[kWarps];
  uint32_t edge[2];
  float reds[kWarps];
  // answers of a search
  int bin, bin2;
  uint32_t bin_n, above_n;
  u64 bin_m, above_m;
  int mine;
  int cut;
};
static_assert(kFirstBin % 8 == 0 && kMaxSteps == 8 * kThreads && Bins<bf16>::n <= kMaxSteps && kList * sizeof(u64) <= kMaxSteps * sizeof(uint32_t), "bins and lists fit");

// v of two bf16 logits (16 bits each), and their bins.
__device__ __forceinline__ uint32_t magnitudes(uint32_t w) {
  constexpr uint32_t kOff = (uint32_t)(uint16_t)(1 - kLeast) * 0x10001u;
  return __viaddmin_s16x2_relu(w & 0x7FFF7FFFu, kOff, (uint32_t)kTop * 0x10001u);
}
__device__ __forceinline__ uint32_t bins(uint32_t w, uint32_t v) {
  uint32_t negative;   // the signs, over each half
  asm("prmt.b32 %0, %1, 0, 0xBB99;" : "=r"(negative) : "r"(w));
  return (v ^ ~negative) & 0x0FFF0FFFu;
}

template <typename T>
struct Row {
  using U = Unit<T>;
  static constexpr int kSteps = Bins<T>::n;
  static constexpr bool kValues = sizeof(T) == 2;   // a step is one value (but for the middle and the last)
  const T* tile;     // this block's part of the row
  int first;         // index of its first entry (may be before the row: such entries are -inf)
  int units;         // of 16 bytes
  int rank, ranks;
  Shared* sh;
  Scale s;
  float top, steps;  // maximum, steps of the first histogram a unit of logits
  uint32_t all_n;    // of the last block_scan
  u64 all_m;
  float all_f;
  int turn_s;

  // The step of a logit: it rises as the logit falls.
  __device__ __forceinline__ int step_of(float l) const {
    if constexpr (kValues) {
      const int b = (int)(__float_as_uint(l) >> 16), v = min(max((b & 0x7FFF) - (kLeast - 1), 0), kTop);
      return b & 0x8000 && v > 0 ? kMiddleStep + 1 + v : kMiddleStep - v;
    } else {
      return (int)place(l);
    }
  }
  // float32: the same before it is cut to a step.
  __device__ __forceinline__ float place(float l) const {
    const float y = (top - l) * steps;
    return fminf(fminf(y, fmaf(y, kFar, kFine * (1.f - kFar))), (float)(kSteps - 1));
  }
  // float32: the largest weight of a step.
  static __device__ __forceinline__ float most_of(int step) {
    const float s = (float)step;
    return ptx::ex2_approx(fminf(s * (-1.f / kPerOctave), fmaf(s, -1.f / kPerFar, (float)kFine / kPerFar - (float)kFine / kPerOctave)));
  }
  // Whether a step holds one value (kValues), and which.
  __device__ __forceinline__ bool one_value(int step) const {
    return kValues && step != 0 && step != kMiddleStep && step != kMiddleStep + 1 && step < kSteps - 1;
  }
  __device__ __forceinline__ float value_of(int step) const {
    const int v = step > kMiddleStep ? step - kMiddleStep - 1 : kMiddleStep - step;
    return __uint_as_float(((uint32_t)(v + kLeast - 1) | (step > kMiddleStep ? 0x8000u : 0u)) << 16);
  }

  // All blocks' v (n of them), in order of rank: sums before this block, and of all.
  template <int n>
  __device__ __forceinline__ void cluster_sums(const u64 (&v)[n], u64 (&before)[n], u64 (&total)[n]) {
    if (threadIdx.x < ranks)
      for (int i = 0; i < n; ++i) st_cluster64(ptx::dsmem_addr(&sh->sums[turn_s][i][rank], threadIdx.x), v[i]);
    ptx::cluster_sync_all();
    for (int i = 0; i < n; ++i) {
      before[i] = total[i] = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r) {
        const u64 x = r < ranks ? sh->sums[turn_s][i][r] : 0;
        if (r < rank) before[i] += x;
        total[i] += x;
      }
    }
    turn_s ^= 1;
  }
  // Sum over the block, in every thread (u64: any order); the warps' stay in sh->warps.
  __device__ __forceinline__ u64 block_sum(u64 v) {
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(kAll, v, m);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh->warps[threadIdx.x >> 5] = v;
    __syncthreads();
    v = sh->warps[threadIdx.x & (kWarps - 1)];
#pragma unroll
    for (int m = kWarps / 2; m >= 1; m >>= 1) v += __shfl_xor_sync(kAll, v, m);
    return v;
  }
  // Sums over the threads before this one, of three kinds at once; the sums of all in all_n, all_m, all_f.
  __device__ __forceinline__ void block_scan(uint32_t n, u64 m, float f, uint32_t& bn, u64& bm, float& bf) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t in = n;
    u64 im = m;
    float jf = f;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t un = __shfl_up_sync(kAll, in, d);
      const u64 um = __shfl_up_sync(kAll, im, d);
      const float uf = __shfl_up_sync(kAll, jf, d);
      if (lane >= d) {
        in += un;
        im += um;
        jf += uf;
      }
    }
    if (lane == 31) {
      sh->scan_n[warp] = in;
      sh->scan_m[warp] = im;
      sh->scan_f[warp] = jf;
    }
    __syncthreads();
    // the warps before this one, and all: every warp scans their sums
    uint32_t wn = lane < kWarps ? sh->scan_n[lane] : 0;
    u64 wm = lane < kWarps ? sh->scan_m[lane] : 0;
    float wf = lane < kWarps ? sh->scan_f[lane] : 0.f;
#pragma unroll
    for (int d = 1; d < kWarps; d <<= 1) {
      const uint32_t un = __shfl_up_sync(kAll, wn, d);
      const u64 um = __shfl_up_sync(kAll, wm, d);
      const float uf = __shfl_up_sync(kAll, wf, d);
      if (lane >= d) {
        wn += un;
        wm += um;
        wf += uf;
      }
    }
    const int prev = max(warp - 1, 0);
    const uint32_t pn = __shfl_sync(kAll, wn, prev);
    const u64 pm = __shfl_sync(kAll, wm, prev);
    const float pf = __shfl_sync(kAll, wf, prev);
    bn = in - n + (warp ? pn : 0);
    bm = im - m + (warp ? pm : 0);
    bf = jf - f + (warp ? pf : 0.f);
    all_n = __shfl_sync(kAll, wn, kWarps - 1);
    all_m = __shfl_sync(kAll, wm, kWarps - 1);
    all_f = __shfl_sync(kAll, wf, kWarps - 1);
    __syncthreads();
  }

  // bf16: the weights of two neighbouring bins' values (of an even step and the next; 0 where a bin holds more than a value)
  // into sh->weight.
  __device__ __forceinline__ void weigh(int step, u64& w0, u64& w1) const {
    gdr::weight(s, sh->table, value_of(step), value_of(step + 1), w0, w1);
    if (!one_value(step)) w0 = 0;
    if (!one_value(step + 1)) w1 = 0;
    *reinterpret_cast<ulonglong2*>(sh->weight + ((step + kFirstBin) & (kMaxSteps - 1))) = make_ulonglong2(w0, w1);
  }

  // Calls f(x[n], index of x[0]) for the block's units, a thread's share.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    for (int i = threadIdx.x; i < units; i += kThreads) {
      float x[U::n];
      U::read(reinterpret_cast<const uint4*>(tile)[i], x);
      f(x, first + i * U::n);
    }
  }
  // The mass of the thread's share where on(x) holds: each weight rounded for itself, as a search through them adds them up (sums
  // of pairs, rounded once a thread, can pass a border that the search then does not find).
  template <typename F>
  __device__ __forceinline__ u64 mass_where(F on) const {
    u64 mass = 0;
    each([&](const float* x, int) {
      bool some = false;
#pragma unroll
      for (int e = 0; e < U::n; ++e) some |= on(x[e]);
      if (!some) return;
#pragma unroll
      for (int e = 0; e < U::n; e += 2) {
        u64 w0, w1;
        gdr::weight(s, sh->table, on(x[e]) ? x[e] : -INFINITY, on(x[e + 1]) ? x[e + 1] : -INFINITY, w0, w1);
        mass += w0 + w1;
      }
    });
    return mass;
  }

  // Counts of the row's logits by step: this block's, then over all blocks, of this thread's steps (kMine neighbours).
  // Each block adds up a part of the steps and hands the sums to all (reading every block's counts everywhere took five
  // times as long). bf16 with `masses`: the masses of the steps that hold more than a value, too.
  static constexpr int kMine = kMaxSteps / kThreads;
  __device__ __forceinline__ void start_counts() {   // (before a barrier)
    for (int i = threadIdx.x; i < kMaxSteps / 4; i += kThreads) reinterpret_cast<uint4*>(sh->steps)[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) sh->mine = 0;
  }
  __device__ __forceinline__ void count_logit(float x) const {
    if (x > -INFINITY) atomicAdd(&sh->steps[step_of(x)], 1u);
  }
  // bf16: eight logits by their bins (-inf among the rest), those around zero listed
  __device__ __forceinline__ void count_unit(const uint4& u) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    uint32_t zero = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t v = magnitudes(w[e]), at = bins(w[e], v);
      atomicAdd(&sh->steps[at & 0xFFFFu], 1u);
      atomicAdd(&sh->steps[at >> 16], 1u);
      zero |= (v - 0x00010001u) & ~v;
    }
    if (zero & 0x80008000u) {   // (or next to one: looked at again)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const uint32_t h = w[e >> 1] >> (16 * (e & 1));
        if ((int)(h & 0x7FFFu) >= kLeast) continue;
        const int i = atomicAdd(&sh->mine, 1);
        if (i < kOthers) sh->others[i] = __uint_as_float(h << 16);
      }
    }
  }
  // (after a cluster barrier behind the counting) bf16: the masses of the steps that hold more than a value: large logits,
  // those around zero, the rest
  __device__ __forceinline__ void finish_counts(bool masses, uint32_t (&n)[kMine], u64 (&mass)[3]) {
    if (kValues && masses) {
      u64 v[3] = {0, 0, 0};
      const int count = sh->mine;
      if (count > kOthers) v[1] = mass_where([&](float x) { return fabsf(x) < 0x1p-8f; });
      else if (threadIdx.x < count) v[1] = gdr::weight(s, sh->table, sh->others[threadIdx.x]);
      if (count) v[1] = block_sum(v[1]);
      if (top >= kLarge) v[0] = block_sum(mass_where([&](float x) { return x >= kLarge; }));
      if ((-kLarge - top) * s.ch > -64.f) v[2] = block_sum(mass_where([&](float x) { return x <= -kLarge && x > -INFINITY; }));
#pragma unroll
      for (int i = 0; i < 3; ++i)
        if (threadIdx.x < ranks) st_cluster64(ptx::dsmem_addr(&sh->sums[turn_s][i][rank], threadIdx.x), v[i]);
    }
    // (parts of whole 16 bytes)
    const int part = (kMaxSteps / 4 + ranks - 1) / ranks, end = min((rank + 1) * part, kMaxSteps / 4);
    for (int at = rank * part + threadIdx.x; at < end; at += kThreads) {
      uint4 t = make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) {
        if (q >= ranks) continue;
        const uint4 x = ld_cluster4(ptx::dsmem_addr(&sh->steps[4 * at], q));
        t.x += x.x;
        t.y += x.y;
        t.z += x.z;
        t.w += x.w;
      }
      for (int q = 0; q < ranks; ++q) st_cluster4(ptx::dsmem_addr(&sh->all[4 * at], q), t);
    }
    ptx::cluster_sync_all();
    if (kValues && masses) {
#pragma unroll
      for (int i = 0; i < 3; ++i) {
        mass[i] = 0;
        for (int q = 0; q < ranks; ++q) mass[i] += sh->sums[turn_s][i][q];
      }
      turn_s ^= 1;
    }
#pragma unroll
    for (int i = 0; i < kMine; i += 4) {
      // (a thread's steps lie side by side in the order of bins, too)
      const uint4 x = reinterpret_cast<const uint4*>(sh->all)[((threadIdx.x * kMine + i + (kValues ? kFirstBin : 0)) & (kMaxSteps - 1)) / 4];
      n[i] = x.x;
      n[i + 1] = x.y;
      n[i + 2] = x.z;
      n[i + 3] = x.w;
    }
    __syncthreads();   // (what lies in the same place is written next)
  }

  // Zeroes this block's histogram, to be filled by `fill`; then finds the first bin at which the running count (or mass)
  // over all blocks reaches `need`. False if the whole does not. (Added up in parts, as the steps are.)
  template <bool kMass, typename F>
  __device__ bool border(u64 need, F fill) {
    for (int i = threadIdx.x; i < kBins; i += kThreads) sh->hist[i] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) sh->bin = -1;
    __syncthreads();
    fill(sh->hist);
    ptx::cluster_sync_all();
    const int part = (kBins + ranks - 1) / ranks, end = min((rank + 1) * part, kBins);
    for (int at = rank * part + threadIdx.x; at < end; at += kThreads) {
      uint32_t n = 0;
      u64 m = 0;
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) {
        if (q >= ranks) continue;
        const uint4 x = ld_cluster4(ptx::dsmem_addr(&sh->hist[at], q));
        n += x.x;
        m += (u64)x.y + ((u64)x.z << 32);
      }
      const uint4 t = make_uint4(n, (uint32_t)m, (uint32_t)(m >> 32), 0);
      for (int q = 0; q < ranks; ++q) st_cluster4(ptx::dsmem_addr(&sh->hist_all[at], q), t);
    }
    ptx::cluster_sync_all();
    // two neighbouring bins a thread
    const int b0 = 2 * threadIdx.x;
    uint32_t n[2];
    u64 m[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const uint4 x = sh->hist_all[b0 + i];
      n[i] = x.x;
      m[i] = (u64)x.y + ((u64)x.z << 32);
    }
    uint32_t bn;
    u64 bm;
    float bf;
    block_scan(n[0] + n[1], m[0] + m[1], 0.f, bn, bm, bf);
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u64 a = kMass ? bm : bn, b = a + (kMass ? m[i] : n[i]);
      if (a < need && b >= need) {
        sh->bin = b0 + i;
        sh->bin_n = n[i];
        sh->above_n = bn;
        sh->above_m = bm;
      }
      bn += n[i];
      bm += m[i];
    }
    __syncthreads();
    return sh->bin >= 0;
  }

  // Key range of a step: it falls with the key, so its ends are found by bisection.
  __device__ void step_keys(int step, uint32_t& lo, uint32_t& hi) {
    __syncthreads();
    if (threadIdx.x < 2) {
      const int b = step - (int)threadIdx.x;   // the smallest key whose step is at most b
      uint32_t l = key_of(-FLT_MAX), r = key_of(top);
      if (b < 0 || step_of(top) > b) {
        l = r + 1;
      } else {
        while (l < r) {
          const uint32_t mid = l + (r - l) / 2;
          if (step_of(of_key(mid)) <= b) r = mid;
          else l = mid + 1;
        }
      }
      sh->edge[threadIdx.x] = l;
    }
    __syncthreads();
    lo = sh->edge[0];
    hi = sh->edge[1] - 1;
  }

  // Among the entries with keys in [lo, hi], from the largest down: the key at which the running count (mass)
  // reaches `need`; what lies above it in the range is taken off `need`, and n is how many entries have it.
  template <bool kMass>
  __device__ bool refine(uint32_t lo, uint32_t hi, u64& need, uint32_t& key, uint32_t& n) {
    for (;;) {
      const int bits = 32 - __clz(hi - lo), shift = max(0, bits - 10);
      const bool got = border<kMass>(need, [&](uint4* h) {
        each([&](const float* x, int) {
#pragma unroll
          for (int e = 0; e < U::n; ++e) {
            const uint32_t k = key_of(x[e] + 0.f);
            if (k >= lo && k <= hi) count<kMass>(h, (hi - k) >> shift, x[e]);
          }
        });
      });
      if (!got) return false;
      need -= kMass ? sh->above_m : sh->above_n;
      const uint32_t b = (uint32_t)sh->bin;
      n = sh->bin_n;
      const uint32_t h2 = hi - (b << shift), w = (1u << shift) - 1;
      __syncthreads();   // (the answer has been read)
      lo = h2 - lo > w ? h2 - w : lo;
      hi = h2;
      if (shift == 0) {
        key = hi;
        return true;
      }
    }
  }
  template <bool kMass>
  __device__ __forceinline__ void count(uint4* h, uint32_t b, float l) const {
    atomicAdd(&h[b].x, 1u);
    if (!kMass) return;
    const u64 w = gdr::weight(s, sh->table, l);
    const uint32_t old = atomicAdd(&h[b].y, (uint32_t)w);
    const uint32_t up = (uint32_t)(w >> 32) + (old + (uint32_t)w < old);
    if (up) atomicAdd(&h[b].z, up);
  }
};

// What is kept of a row: logits above `value`, and those equal to it up to index `cut`.
struct Border {
  float value;
  uint32_t ties, equal;   // how many of the equal ones are kept, and how many there are
  int cut;
  bool known;             // cut is given (ties and equal are not needed)
  bool weighed;           // bf16: the weights of the row's values lie in Shared::weight
  u64 mass;               // of what is kept, where it came about (0: not)
};

// The border of top-k (0: none) and top-p (1: none) in a row whose logits are counted by step.
template <typename T>
__device__ __forceinline__ Border find_border(Row<T>& r, int k, float p) {
  using U = Unit<T>;
  constexpr int kMine = Row<T>::kMine, kSteps = Row<T>::kSteps;
  Shared& sh = *r.sh;
  const int tid = threadIdx.x, s0 = tid * kMine;
  Border out = {-INFINITY, 0, 0, -1, false, false, 0};
  const bool cuts_k = k > 0, cuts_p = p < 1.f;
  uint32_t n[kMine];
  u64 others[3] = {0, 0, 0};
  r.finish_counts(p < 1.f, n, others);
  if constexpr (Row<T>::kValues) {
    // negative zeros' neighbours belong to the middle; -inf is among the rest, which matters only where the k-th logit does
    constexpr int kA = kMiddleStep, kB = kMiddleStep + 1, kLast = kSteps - 1;
    static_assert(kA / kMine + 1 == kB / kMine && kB % kMine == 0, "the middle's two steps lie in neighbouring threads");
    if (tid == kB / kMine) {
      sh.bin_n = n[0];
      n[0] = 0;
    }
    __syncthreads();
    if (tid == kA / kMine) n[kA % kMine] += sh.bin_n;
    uint32_t finite = 0;
    if (cuts_k) {
      uint32_t c = 0;
      if (tid != kLast / kMine)
#pragma unroll
        for (int i = 0; i < kMine; ++i) c += n[i];
      else
#pragma unroll
        for (int i = 0; i < kLast % kMine; ++i) c += n[i];
      if (r.block_sum(c) <= (u64)k) {   // (the same in every block)
        u64 mine = 0;
        r.each([&](const float* x, int) {
#pragma unroll
          for (int e = 0; e < U::n; ++e) mine += x[e] <= -kLarge && x[e] > -INFINITY;
        });
        const u64 v[1] = {r.block_sum(mine)};
        u64 before[1], sum[1];
        r.cluster_sums(v, before, sum);
        finite = (uint32_t)sum[0];
      }
    }
    if (tid == kLast / kMine) n[kLast % kMine] = finite;
  }

  // counts above this thread's steps; masses: of each step's value, or (float32) bounds that the steps' width gives
  uint32_t sum_n = 0, bn;
  u64 m[kMine], sum_m = 0, bm;
  float sum_f = 0.f, bf;
#pragma unroll
  for (int i = 0; i < kMine; ++i) {
    sum_n += n[i];
    m[i] = 0;
    if (!Row<T>::kValues) sum_f += (float)n[i] * Row<T>::most_of(s0 + i);
  }
  if (Row<T>::kValues && cuts_p) {
    // (the kept mass is added up from these weights, too; of bins that hold nothing none is needed)
    uint32_t some = 0;
#pragma unroll
    for (int i = 0; i < kMine; ++i) some |= n[i];
    if (some)
#pragma unroll
    for (int i = 0; i < kMine; i += 2) {
      u64 w0, w1;
      r.weigh(s0 + i, w0, w1);
      m[i] = n[i] * w0;
      m[i + 1] = n[i + 1] * w1;
      sum_m += m[i] + m[i + 1];
    }
    out.weighed = true;
  }
  if (Row<T>::kValues) {
    constexpr int at[3] = {0, kMiddleStep, kSteps - 1};
#pragma unroll
    for (int i = 0; i < 3; ++i)
      if (at[i] / kMine == tid) {
        m[at[i] % kMine] = others[i];
        sum_m += others[i];
      }
  }
  r.block_scan(sum_n, sum_m, sum_f, bn, bm, bf);

  // ------------------------------------------------------------------ the step of the k-th logit
  const uint32_t total_n = r.all_n;
  const u64 total_m = r.all_m;
  const float total_f = r.all_f;
  const bool k_on = cuts_k && (uint32_t)k < total_n;
  int k_step = kSteps;
  uint32_t k_above = 0, k_equal = 0;
  u64 k_mass = 0;      // (values) mass above that step
  if (k_on) {
    uint32_t at = bn;
    u64 am = bm;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      if (at < (uint32_t)k && at + n[i] >= (uint32_t)k) {
        sh.bin = s0 + i;
        sh.bin_n = n[i];
        sh.above_n = at;
        sh.above_m = am;
      }
      at += n[i];
      am += m[i];
    }
    __syncthreads();
    k_step = sh.bin;
    k_equal = sh.bin_n;
    k_above = sh.above_n;
    k_mass = sh.above_m;
    __syncthreads();
  }

  if constexpr (Row<T>::kValues) {
    // a step is a value: the border lies in it, or (rarely) in the middle or the rest
    if (k_on) {
      u64 need = (u64)k - k_above;
      uint32_t n_key = k_equal;
      out.value = r.value_of(k_step);
      if (!r.one_value(k_step)) {
        uint32_t lo, hi, key;
        r.step_keys(k_step, lo, hi);
        r.template refine<false>(lo, hi, need, key, n_key);
        out.value = of_key(key);
        out.weighed = false;
      }
      out.ties = (uint32_t)need;
      out.equal = n_key;
    }
    if (!cuts_p) return out;
    u64 all = 0;
    if (!k_on) {
      all = total_m;
    } else if (r.one_value(k_step)) {
      all = k_mass + out.ties * weight(r.s, sh.table, out.value);
    } else {
      const float b = out.value;
      const u64 v[1] = {r.block_sum(r.mass_where([&](float x) { return x > b; }))};
      u64 before[1], mass[1];
      r.cluster_sums(v, before, mass);
      all = mass[0] + out.ties * weight(r.s, sh.table, b);
    }
    u64 need = max((u64)1, times(all, p, true)), am = bm;
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      if (am < need && am + m[i] >= need) {
        sh.bin = s0 + i;
        sh.bin_n = n[i];
        sh.above_m = am;
      }
      am += m[i];
    }
    __syncthreads();
    const int step = sh.bin;
    const uint32_t equal = sh.bin_n;
    const u64 above = sh.above_m;
    __syncthreads();
    need -= above;   // (sums of whole numbers: there is such a step, the k-th logit's at the latest)
    if (r.one_value(step)) {
      const u64 w = max((u64)1, weight(r.s, sh.table, r.value_of(step)));
      const uint32_t ties = least_ties(need, w, equal);
      if (k_on && step == k_step) {
        out.ties = min(out.ties, ties);
      } else {
        out.value = r.value_of(step);
        out.ties = ties;
        out.equal = equal;
      }
      out.mass = above + out.ties * w;
      return out;
    }
    uint32_t lo, hi, key, n_key;
    r.step_keys(step, lo, hi);
    out.weighed = false;   // (its place is written anew)
    if (r.template refine<true>(lo, hi, need, key, n_key) && (!k_on || of_key(key) >= out.value)) {
      const float b = of_key(key);
      const u64 w = max((u64)1, weight(r.s, sh.table, b));
      const uint32_t ties = least_ties(need, w, n_key);
      if (k_on && b == out.value) {
        out.ties = min(out.ties, ties);
      } else {
        out.value = b;
        out.ties = ties;
        out.equal = n_key;
      }
    }
    return out;
  } else {
    // ---------------------------------------------------------------- float32: the steps that may hold the border
    int lo_step = 0, hi_step = k_on ? k_step : kSteps - 1;
    int first_step = 0;   // narrowed down
    if (cuts_p && !k_on) {
      // Between the running sums' bounds: a step's weights lie within a factor of kWidth or kCoarse of its largest (the
      // last step's between 0 and that); 2^-10 for the sums' own roundings and those of the steps' borders.
      const float all = total_f;
      if (tid == 0) {
        sh.bin = kSteps - 1;
        sh.bin2 = kSteps - 1;
      }
      if (s0 == kFine) sh.reds[0] = bf;
      __syncthreads();
      const float low = kWidth * sh.reds[0] + kCoarse * fmaxf(0.f, all - sh.reds[0]);
      const float least = p * low * (1.f - 0x1p-10f) - 0x1p-14f, most = p * all * (1.f + 0x1p-10f) + 0x1p-14f;
      // The first step whose sum reaches each of the two, of all steps that do: a thread's last sum and the next thread's first
      // one are added up in different orders, so a limit may lie between them, and a step at which the sum passes it need
      // not be anywhere. (The border's own step reaches `least` whatever the sums' roundings.)
      int lo = kSteps, hi = kSteps;
      float at = bf;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        at += (float)n[i] * Row<T>::most_of(s0 + i);
        if (at >= least) lo = min(lo, s0 + i);
        if (s0 + i < kFine && at * kWidth >= most) hi = min(hi, s0 + i);
      }
      lo = __reduce_min_sync(kAll, lo);
      hi = __reduce_min_sync(kAll, hi);
      if ((tid & 31) == 0 && lo < kSteps) atomicMin(&sh.bin, lo);
      if ((tid & 31) == 0 && hi < kSteps) atomicMin(&sh.bin2, hi);
      __syncthreads();
      lo_step = sh.bin;
      hi_step = max(sh.bin2, lo_step);
      first_step = lo_step;
      __syncthreads();
    }
    u64 all = 0, above = 0;   // the mass of all (of the first k), and above lo_step
    // Candidates: the logits of steps first_step .. hi_step, handed to every block. How many the steps hold:
    const int room = kList / r.ranks;
    auto held = [&](int from, int to) {
      if (tid == 0) {
        sh.above_n = sh.bin_n = 0;
        sh.mine = 0;
      }
      __syncthreads();
      uint32_t at = bn;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        if (s0 + i == from) sh.bin_n = at;
        at += n[i];
        if (s0 + i == to) sh.above_n = at;
      }
      __syncthreads();
      return sh.above_n - sh.bin_n;
    };
    auto hand = [&](float x, int index) {
      const int i = atomicAdd(&sh.mine, 1);
      const u64 c = ((u64)key_of(x) << 32) | (0xFFFFFFFFu - (uint32_t)index);
      if (i < room)
        for (int q = 0; q < r.ranks; ++q) st_cluster64(ptx::dsmem_addr(&sh.list[r.rank * room + i], q), c);
    };
    // how many each block has handed over, and whether they fit
    int offset[kMaxCluster + 1];
    bool fits = true;
    auto handed = [&](int slot) {
      offset[0] = 0;
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q) {
        const int c = q < r.ranks ? (int)sh.sums[r.turn_s][slot][q] : 0;
        fits = fits && c <= room;
        offset[q + 1] = offset[q] + c;
      }
    };
    // Top-p alone: a few hundred of them go along with the weighing of all, more are narrowed down first (a row of 49999: 57000
    // cycles instead of 68700).
    bool direct = false;
    if (cuts_p && !k_on) {
      direct = held(lo_step, hi_step) <= kDirect;
      W2 acc = {{0}, {0}}, acc_above = {{0}, {0}};
      const float lo_edge = (float)lo_step, hi_edge = direct ? hi_step == kSteps - 1 ? INFINITY : (float)(hi_step + 1) : lo_edge;
      r.each([&](const float* x, int at) {
#pragma unroll
        for (int e = 0; e < U::n; e += 2) {
          const W2 w = weights(r.s, sh.table, x[e], x[e + 1]);
          accumulate(acc, w.hi, w.lo);
          const float y0 = r.place(x[e]), y1 = r.place(x[e + 1]);
          if (y0 < hi_edge || y1 < hi_edge) {
            const F2 up = pack(y0 < lo_edge ? 1.f : 0.f, y1 < lo_edge ? 1.f : 0.f);
            accumulate(acc_above, mul(w.hi, up), mul(w.lo, up));
            if (y0 >= lo_edge && y0 < hi_edge && x[e] > -INFINITY) hand(x[e], at + e);
            if (y1 >= lo_edge && y1 < hi_edge && x[e + 1] > -INFINITY) hand(x[e + 1], at + e + 1);
          }
        }
      });
      const u64 mine_all = r.block_sum(fixed(acc)), v[3] = {mine_all, r.block_sum(fixed(acc_above)), (u64)sh.mine};
      if (tid < r.ranks)
        for (int i = 0; i < 3; ++i) st_cluster64(ptx::dsmem_addr(&sh.sums[r.turn_s][i][r.rank], tid), v[i]);
      ptx::cluster_sync_all();
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q)
        if (q < r.ranks) {
          all += sh.sums[r.turn_s][0][q];
          above += sh.sums[r.turn_s][1][q];
        }
      handed(2);
      r.turn_s ^= 1;
    }
    if (cuts_p && !k_on && !direct) {
      // With these the doubt is about the window's own mass alone: usually one or two steps are left.
      const u64 want = max((u64)1, times(all, p, true));
      const float need = want > above ? (float)(want - above) * 0x1p-40f : 0.f, slack = (float)all * 0x1p-58f;
      if (tid == 0) {
        sh.bin = hi_step;
        sh.bin2 = hi_step;
        sh.reds[0] = 0.f;
      }
      __syncthreads();
      float at = bf;
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        if (s0 + i == lo_step) sh.reds[0] = at;   // the float sums' value where the window begins
        at += (float)n[i] * Row<T>::most_of(s0 + i);
      }
      __syncthreads();
      at = bf - sh.reds[0];
#pragma unroll
      for (int i = 0; i < kMine; ++i) {
        const float up = at + (float)n[i] * Row<T>::most_of(s0 + i);
        const int step = s0 + i;
        if (step >= lo_step && step <= hi_step) {
          if (up + slack >= need * (1.f - 0x1p-10f)) atomicMin(&sh.bin, step);
          if ((up - slack) * (step < kFine ? kWidth : kCoarse) >= need * (1.f + 0x1p-10f)) atomicMin(&sh.bin2, step);
        }
        at = up;
      }
      __syncthreads();
      first_step = min(sh.bin, hi_step);
      hi_step = max(min(sh.bin2, hi_step), first_step);
      __syncthreads();
    }
    if (!direct) {
      const bool few = held(first_step, hi_step) <= kList / 2;
      u64 between = 0;
      W2 acc = {{0}, {0}};
      const float w_edge = (float)lo_step, lo_edge = (float)first_step, hi_edge = (float)(hi_step + 1);
      const bool open = hi_step == kSteps - 1, mass = first_step > lo_step;
      r.each([&](const float* x, int at) {
        float y[U::n];
        bool some = false, part = false;
#pragma unroll
        for (int e = 0; e < U::n; ++e) {
          y[e] = r.place(x[e]);
          some |= y[e] >= lo_edge && (y[e] < hi_edge || open);
          part |= y[e] >= w_edge && y[e] < lo_edge;
        }
        if (mass && part)
#pragma unroll
          for (int e = 0; e < U::n; e += 2) {
            const W2 w = weights(r.s, sh.table, y[e] >= w_edge && y[e] < lo_edge ? x[e] : -INFINITY,
                                 y[e + 1] >= w_edge && y[e + 1] < lo_edge ? x[e + 1] : -INFINITY);
            accumulate(acc, w.hi, w.lo);
          }
        if (few && some)
#pragma unroll
          for (int e = 0; e < U::n; ++e)
            if (y[e] >= lo_edge && (y[e] < hi_edge || open) && x[e] > -INFINITY) hand(x[e], at + e);
      });
      between = fixed(acc);
      const u64 mine_between = r.block_sum(between), v[2] = {mine_between, (u64)sh.mine};
      if (tid < r.ranks)
        for (int i = 0; i < 2; ++i) st_cluster64(ptx::dsmem_addr(&sh.sums[r.turn_s][i][r.rank], tid), v[i]);
      ptx::cluster_sync_all();
#pragma unroll
      for (int q = 0; q < kMaxCluster; ++q)
        if (q < r.ranks) above += sh.sums[r.turn_s][0][q];
      fits = few;
      handed(1);
      r.turn_s ^= 1;
    }
    {
      if (fits) {
        // ------------------------------------------------------------ few: in order, every block for itself
        const int count = offset[kMaxCluster];   // (one at least: the border's)
        // packed into the list's first half; then each to the place that the number of larger ones gives
        constexpr int kEach = kList / 2 / kThreads;
        u64 mine[kEach], *packed = sh.list, *sorted = sh.list + kList / 2;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          const int i = tid + j * kThreads;
          mine[j] = 0;
          if (i < count) {
            int q = 0;
#pragma unroll
            for (int z = 1; z < kMaxCluster; ++z) q += i >= offset[z];
            mine[j] = sh.list[q * room + i - offset[q]];
          }
        }
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kEach; ++j)
          if (tid + j * kThreads < count) packed[tid + j * kThreads] = mine[j];
        __syncthreads();
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          if (tid + j * kThreads >= count) continue;
          int place = 0;
#pragma unroll 8
          for (int i = 0; i < count; ++i) place += packed[i] > mine[j];
          sorted[place] = mine[j];
        }
        __syncthreads();
        // neighbours' weights and their running sums
        u64 w[kEach], mass = 0, before;
        uint32_t un;
        float uf;
#pragma unroll
        for (int j = 0; j < kEach; ++j) {
          const int i = tid * kEach + j;
          w[j] = i < count && cuts_p && !(k_on && i >= k) ? weight(r.s, sh.table, of_key((uint32_t)(sorted[i] >> 32))) : 0;
          mass += w[j];
        }
        if (cuts_p) {
          r.block_scan(0, mass, 0.f, un, before, uf);
          if (k_on) all = r.all_m;
        }
        const int most = k_on ? min(k, count) : count;
        if (tid == 0) sh.bin = most - 1;
        __syncthreads();
        if (cuts_p) {
          const u64 want = max((u64)1, times(all, p, true)), need = want > above ? want - above : 1;
          u64 at = before;
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            const int i = tid * kEach + j;
            if (i < most && at < need && at + w[j] >= need) atomicMin(&sh.bin, i);
            at += w[j];
          }
          __syncthreads();
          at = before;
#pragma unroll
          for (int j = 0; j < kEach; ++j) {
            at += w[j];
            if (tid * kEach + j == sh.bin) sh.above_m = at;
          }
          __syncthreads();
          out.mass = above + sh.above_m;
        }
        const u64 last = sorted[sh.bin];
        out.value = of_key((uint32_t)(last >> 32));
        out.cut = (int)(0xFFFFFFFFu - (uint32_t)last);
        out.known = true;
        return out;
      }
    }
    // ---------------------------------------------------------------- many: histograms of the doubtful steps' floats
    if (k_on) {
      u64 need = (u64)k - k_above;
      uint32_t lo, hi, key, n_key = 0;
      r.step_keys(k_step, lo, hi);
      r.template refine<false>(lo, hi, need, key, n_key);
      out.value = of_key(key);
      out.ties = (uint32_t)need;
      out.equal = n_key;
      if (!cuts_p) return out;
      const float b = out.value;
      const u64 v[1] = {r.block_sum(r.mass_where([&](float x) { return x > b; }))};
      u64 before[1], mass[1];
      r.cluster_sums(v, before, mass);
      all = mass[0] + out.ties * weight(r.s, sh.table, b);
      const u64 want = max((u64)1, times(all, p, true));
      if (want > mass[0]) {   // inside the tokens that equal the k-th
        const u64 w = max((u64)1, weight(r.s, sh.table, b));
        out.ties = least_ties(want - mass[0], w, out.ties);
        return out;
      }
    }
    if (!cuts_p) return out;
    u64 need = max((u64)1, times(all, p, true)) - above;   // (what lies above first_step is less by `least`'s margin)
    uint32_t lo, hi, ends, key, n_key;
    r.step_keys(first_step, ends, hi);
    if (k_on) lo = key_of(out.value) + 1;
    else r.step_keys(hi_step, lo, ends);
    if (r.template refine<true>(lo, hi, need, key, n_key)) {
      out.value = of_key(key);
      const u64 w = max((u64)1, weight(r.s, sh.table, out.value));
      out.ties = least_ties(need, w, n_key);
      out.equal = n_key;
    }
    return out;
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a, const __grid_constant__ Table tab) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Shared sh;
  using U = Unit<T>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ranks = a.cluster, rank = (int)ptx::cluster_ctarank(), row = blockIdx.x / ranks;
  const T* logits = static_cast<const T*>(a.logits) + (long long)row * a.stride;

  float temperature = __ldg(a.temperature + row);
  int k = a.top_k ? __ldg(a.top_k + row) : 0;
  float p = a.top_p ? __ldg(a.top_p + row) : 1.f;
  const float min_p = a.min_p ? __ldg(a.min_p + row) : 0.f;
  if (!(temperature >= 0.f) || k < 0 || !(p >= 0.f && p <= 1.f) || !(min_p >= 0.f && min_p <= 1.f)) {   // (the same in the whole cluster)
    if (tid == 0) atomicCAS(a.err, 0, kErrDeviceIndex);
    return;
  }
  if (temperature == 0.f) {   // the best token alone
    k = 1;
    p = 1.f;
  } else {   // (log2(e) / T stays a float; above, the lowest logit would have weight, and -inf, which stands for what is not kept, is taken for it)
    temperature = fminf(fmaxf(temperature, 1.5e-30f), 1e36f);
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // (waited for before the first remote write)
  if (tid < 64) sh.table[tid] = tab.t[tid];
  if (tid == kThreads - 1 && min_p > 0.f) sh.min_p = (double)temperature * log((double)min_p);   // (read after barriers)

  Row<T> r;
  r.tile = reinterpret_cast<const T*>(dyn);
  r.sh = &sh;
  r.rank = rank;
  r.ranks = ranks;
  r.turn_s = 0;
  // 16-byte units from the aligned address at or before the row's first entry
  const int skew = (int)((reinterpret_cast<uintptr_t>(logits) & 15) / sizeof(T));
  const int all = (a.V + skew + U::n - 1) / U::n, per = (all + ranks - 1) / ranks;
  const int u0 = min(all, rank * per);
  r.units = min(all, u0 + per) - u0;
  r.first = u0 * U::n - skew;

  const bool filters = (k > 0 && k < a.V) || p < 1.f;
  if (!(k > 0 && k < a.V)) k = 0;
  if (filters) r.start_counts();
  __syncthreads();
  // the row into shared memory, and its largest entry (bf16: and the counts of its values)
  float top = -INFINITY;
  {
    uint4* to = reinterpret_cast<uint4*>(dyn);
    const uint4* from = reinterpret_cast<const uint4*>(logits + r.first);
    constexpr int kAhead = 8;
    for (int i0 = tid; i0 < r.units; i0 += kAhead * kThreads) {
      uint4 v[kAhead];
#pragma unroll
      for (int c = 0; c < kAhead; ++c) {
        const int i = i0 + c * kThreads, at = r.first + i * U::n;
        if (i >= r.units) continue;
        if (at >= 0 && at + U::n <= a.V) {
          v[c] = __ldg(from + i);
        } else {
          float x[U::n];
#pragma unroll
          for (int e = 0; e < U::n; ++e) x[e] = at + e >= 0 && at + e < a.V ? clean(U::one(logits + at + e)) : -INFINITY;
          v[c] = U::write(x);
        }
      }
#pragma unroll
      for (int c = 0; c < kAhead; ++c) {
        const int i = i0 + c * kThreads;
        if (i >= r.units) continue;
        const uint4 x = U::clean_max(v[c], top);
        to[i] = x;
        if constexpr (Row<T>::kValues)
          if (filters) r.count_unit(x);
      }
    }
  }
#pragma unroll
  for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, m));
  if (lane == 0) sh.reds[warp] = top;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh.reds[w]);
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (tid < ranks) st_cluster(ptx::dsmem_addr(&sh.tops[rank], tid), __float_as_uint(top));
  ptx::cluster_sync_all();
  for (int i = 0; i < ranks; ++i) top = fmaxf(top, sh.tops[i]);
  top += 0.f;
  r.top = top;

  u64 total = 0;
  if (top > -INFINITY) {
    {
      const float t = temperature == 0.f ? 1.f : temperature;
      // log2(e) / T as a pair: the quotient, and what it leaves over T
      constexpr float kLog2e = 1.44269502162933349609375f, kLog2eLow = 1.9259629911266174681e-8f;
      r.s.ch = kLog2e / t;
      r.s.cl = (fmaf(-r.s.ch, t, kLog2e) + kLog2eLow) / t;
      const bool near = fabsf(top) * r.s.ch < 300.f;
      r.s.ref = near ? 0.f : top;
      const float z = near ? top : 0.f;
      r.s.mh = __fmul_rn(z, r.s.ch);
      r.s.ml = __fmaf_rn(z, r.s.cl, __fmaf_rn(z, r.s.ch, -r.s.mh));
      r.s.least = fmaxf((r.s.mh - 152.f) / r.s.ch, -FLT_MAX);
      r.steps = r.s.ch * (float)kPerOctave;
    }
    Border edge = {-INFINITY, 0, 0, -1, false, false, 0};
    if (filters) {
      if (!Row<T>::kValues) {
        r.each([&](const float* x, int) {
#pragma unroll
          for (int e = 0; e < U::n; ++e) r.count_logit(x[e]);
        });
        ptx::cluster_sync_all();
      }
      edge = find_border(r, k, p);
    }

    // ---------------------------------------------------------------- min-p
    if (min_p > 0.f && temperature > 0.f) {
      const double least = (double)top + sh.min_p;
      const float f = __double2float_ru(least) + 0.f;   // the smallest logit that is kept
      if (f > edge.value) {
        edge = {of_key(key_of(f) - (f == 0.f ? 2 : 1)), 0, 0, -1, true, edge.weighed, 0};   // the float below it
      }
    }
    const float border = edge.value;

    // ---------------------------------------------------------------- the kept mass, the token
    // Of the entries that equal the border the first `ties` are kept; where that is not all of them, they are counted along
    // with the mass of the others, and a running sum is the mass so far and the border's weight for each kept one of them.
    const bool part = !edge.known && edge.ties > 0 && edge.ties < edge.equal;
    int cut = edge.known ? edge.cut : edge.ties > 0 && !part ? 0x7fffffff : -1;   // the last index of them that is kept (part: none yet)
    const u64 tie = part ? weight(r.s, sh.table, border) : 0;
    auto kept = [&](float x, int at) { return x > border || (x == border && x > -INFINITY && at <= cut); };
    total = edge.mass;
    const bool sums = a.token || total == 0, find_cut = part && a.probs;
    // a warp's run of units
    const int run = (r.units + kWarps - 1) / kWarps, w0 = min(r.units, warp * run), w1 = min(r.units, w0 + run);
    const uint4* tile = reinterpret_cast<const uint4*>(dyn);
    if (sums || find_cut) {
      if constexpr (Row<T>::kValues) {
        // the weights of the bins' values that may be kept, once
        __syncthreads();
        const int last = min(border > -INFINITY ? r.step_of(border) : Row<T>::kSteps - 2, Row<T>::kSteps - 2);
        u64 unused0, unused1;
        for (int i = 2 * tid; !edge.weighed && i <= last; i += 2 * kThreads) r.weigh(i, unused0, unused1);
        if (tid == 0) sh.weight[0] = sh.weight[kMaxSteps - 1] = sh.weight[kTop] = 0;   // (around zero, and the rest)
        __syncthreads();
      }
      auto weight_of = [&](float x) -> u64 {
        if constexpr (Row<T>::kValues) {
          const int step = r.step_of(x);
          if (r.one_value(step)) return sh.weight[(step + kFirstBin) & (kMaxSteps - 1)];
        }
        return weight(r.s, sh.table, x);
      };
      u64 mine = 0;
      uint32_t equal = 0;
      if constexpr (Row<T>::kValues) {
        // two at once: those that are not kept at a bin without weight, as are those whose bin holds more than one value; kept
        // ones of these (few, or none) are added by themselves
        const __nv_bfloat162 b2 = __bfloat162bfloat162(__float2bfloat16_rd(border));   // (above the one is above the other)
        const bool all_ties = edge.ties > 0 && !part;
        for (int i = w0 + lane; i < w1; i += 32) {
          const uint4 u = tile[i];
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
          uint32_t odd = 0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 x2 = *reinterpret_cast<const __nv_bfloat162*>(&w[e]);
            const uint32_t same = __heq2_mask(x2, b2), on = __hgt2_mask(x2, b2) | (all_ties ? same : 0u);
            const uint32_t v = magnitudes(w[e]), at = bins(w[e], v) & on;
            mine += sh.weight[at & 0xFFFFu];
            mine += sh.weight[at >> 16];
            equal += __popc(same);
            odd |= ((v - 0x00010001u) | (v + (0x8000u - kTop) * 0x10001u)) & on;   // v = 0 (or next to one), v = kTop
          }
          if (odd & 0x80008000u) {
            float x[U::n];
            U::read(u, x);
            const int at = r.first + i * U::n;
#pragma unroll
            for (int e = 0; e < U::n; ++e)
              if (kept(x[e], at + e) && !r.one_value(r.step_of(x[e]))) mine += weight(r.s, sh.table, x[e]);
          }
        }
        equal = part ? equal / 16 : 0;
      } else {
        W2 acc = {{0}, {0}};
        for (int i = w0 + lane; i < w1; i += 32) {
          float x[U::n];
          U::read(tile[i], x);
          const int at = r.first + i * U::n;
          bool some = false;
#pragma unroll
          for (int e = 0; e < U::n; ++e) some |= x[e] >= border;
          if (!some) continue;
          if (part)
#pragma unroll
            for (int e = 0; e < U::n; ++e) equal += x[e] == border;
          if (!sums) continue;
#pragma unroll
          for (int e = 0; e < U::n; e += 2) {
            const W2 w = weights(r.s, sh.table, kept(x[e], at + e) ? x[e] : -INFINITY, kept(x[e + 1], at + e + 1) ? x[e + 1] : -INFINITY);
            // (what is not drawn, a weight that rounds to 0 units, adds nothing: where a sum passes there is an entry to find)
            float h0, h1;
            unpack(w.hi, h0, h1);
            accumulate(acc, pack(h0 > 0.5f ? h0 : 0.f, h1 > 0.5f ? h1 : 0.f), w.lo);
          }
        }
        mine = fixed(acc);
      }
      {   // the warps' sums stay in sh.warps and sh.equals
        equal = __reduce_add_sync(kAll, equal);
        if (lane == 0) sh.equals[warp] = equal;
        mine = r.block_sum(mine);   // (its barriers are behind this write, too)
        u64 e64;
        e64 = sh.equals[lane & (kWarps - 1)];
#pragma unroll
        for (int m = kWarps / 2; m >= 1; m >>= 1) e64 += __shfl_xor_sync(kAll, e64, m);
        const u64 v[2] = {mine, e64};
        u64 before[2], sum[2];
        r.cluster_sums(v, before, sum);
        if (sums) total = sum[0] + edge.ties * tie;
        // The entry at which the running sum passes target: its index goes to `found` in the one block that holds it.
        // kMass false: the running count of the border's equals instead.
        auto search = [&](auto mass, u64 target, auto found) {
          constexpr bool kMass = decltype(mass)::value;
          const u64 each_tie = kMass ? tie : 1;
          auto sum_at = [&](u64 m, u64 n) { return (kMass ? m : 0) + min(n, (u64)edge.ties) * each_tie; };
          // the first of kWarps parts (lane's: pm, pn) that passes; m and n are then what lies before it, or before the last
          // part that holds anything where none passes (their sums differ from the whole's by roundings)
          u64 m = before[0], n = before[1];
          auto first_part = [&](u64 pm, uint32_t pn, bool& none) {
            u64 im = pm;
            uint32_t in = pn;
#pragma unroll
            for (int d = 1; d < kWarps; d <<= 1) {
              const u64 um = __shfl_up_sync(kAll, im, d);
              const uint32_t un = __shfl_up_sync(kAll, in, d);
              if (lane >= d) {
                im += um;
                in += un;
              }
            }
            const u64 m0 = m + im - pm, n0 = n + in - pn;
            const unsigned over = __ballot_sync(kAll, lane < kWarps && sum_at(m + im, n + in) > target);
            const unsigned holds = __ballot_sync(kAll, lane < kWarps && (pm || (pn && n0 < edge.ties)));
            none = over == 0;
            const int who = over ? __ffs(over) - 1 : holds ? 31 - __clz(holds) : 0;
            m = __shfl_sync(kAll, m0, who);
            n = __shfl_sync(kAll, n0, who);
            return who;
          };
          if (sum_at(m, n) > target) return;
          bool none;
          const int w = first_part(sh.warps[lane & (kWarps - 1)], sh.equals[lane & (kWarps - 1)], none);
          if (none) return;
          // the warps share that run: a 32-unit piece each
          const int i0 = min(r.units, w * run) + warp * 32 + lane, end = min(r.units, (w + 1) * run);
          const int base = r.first + i0 * U::n;
          const bool there = warp * 32 < run && i0 < end;
          float x[U::n];
          u64 vm[U::n], im = 0;
          uint32_t in = 0;
          if (there) U::read(tile[i0], x);
#pragma unroll
          for (int e = 0; e < U::n; ++e) {
            vm[e] = kMass && there && kept(x[e], base + e) ? weight_of(x[e]) : 0;
            im += vm[e];
            in += part && there && x[e] == border;
          }
          const u64 own_m = im;
          const uint32_t own_n = in;
#pragma unroll
          for (int d = 1; d < 32; d <<= 1) {
            const u64 um = __shfl_up_sync(kAll, im, d);
            const uint32_t un = __shfl_up_sync(kAll, in, d);
            if (lane >= d) {
              im += um;
              in += un;
            }
          }
          if (lane == 31) {
            sh.chunks[warp] = im;
            sh.chunk_equals[warp] = in;
          }
          __syncthreads();
          const int c = first_part(sh.chunks[lane & (kWarps - 1)], sh.chunk_equals[lane & (kWarps - 1)], none);
          if (warp == c) {
            const bool holds = own_m > 0 || (own_n > 0 && n + in - own_n < edge.ties);
            const unsigned over = __ballot_sync(kAll, none ? holds : sum_at(m + im, n + in) > target);
            if (over && lane == (none ? 31 - __clz(over) : __ffs(over) - 1)) {
              u64 sm = m + im - own_m, sn = n + in - own_n;
              int hit = -1;
#pragma unroll
              for (int e = 0; e < U::n; ++e) {
                const bool eq = part && x[e] == border && sn < edge.ties;
                sm += vm[e];
                sn += part && x[e] == border;
                if ((vm[e] || eq) && (none || (sum_at(sm, sn) > target && hit < 0))) hit = base + e;
              }
              found(hit);
            }
          }
          __syncthreads();
        };
        if (a.token) {
          const float u = __ldg(a.u + row);
          search(std::true_type(), u > 0.f ? min(times(total, u, false), total - 1) : 0, [&](int i) { a.token[row] = i; });
        }
        if (find_cut) {
          search(std::false_type(), edge.ties - 1, [&](int at) {
            for (int i = 0; i < ranks; ++i) st_cluster(ptx::dsmem_addr(&sh.cut, i), (uint32_t)at);
          });
          ptx::cluster_sync_all();
          cut = sh.cut;
        }
      }
    }
    if (a.probs) {
      float* out = a.probs + (long long)row * a.V;
      const float inv = 1.f / (float)total;
      const int n = r.units * U::n;
      for (int i = tid; i < n; i += 2 * kThreads) {
        const int j = i + kThreads, ai = r.first + i, aj = r.first + j;
        const float x = U::one(r.tile + i), y = j < n ? U::one(r.tile + j) : -INFINITY;
        const bool kx = kept(x, ai), ky = kept(y, aj);
        float px = 0.f, py = 0.f;
        if (kx || ky) {
          const W2 w = weights(r.s, sh.table, x, y);
          unpack(mul(add(w.hi, w.lo), both(inv)), px, py);
        }
        if (ai >= 0 && ai < a.V) out[ai] = kx ? px : 0.f;
        if (j < n && aj >= 0 && aj < a.V) out[aj] = ky ? py : 0.f;
      }
    }
  } else {   // nothing to draw from
    if (a.token && rank == 0 && tid == 0) a.token[row] = -1;
    if (a.probs)
      for (int i = tid; i < r.units * U::n; i += kThreads) {
        const int at = r.first + i;
        if (at >= 0 && at < a.V) a.probs[(long long)row * a.V + at] = 0.f;
      }
  }
  ptx::cluster_sync_all();   // no block leaves while another may write to its shared memory
}

const Table& table() {
  static const Table t = [] {
    Table t;
    for (int k = 0; k < 64; ++k) {
      const double x = std::exp2(k / 64.0);
      t.t[k].x = (float)x;
      t.t[k].y = (float)(x - (double)t.t[k].x);
    }
    return t;
  }();
  return t;
}

// Blocks of a row, `bytes(c)` each of c: all at once if that can be, one an SM or (at about 1.35 the time) two, whichever
// should end sooner. Clusters leave gaps: of more than two blocks only some 128 find an SM each, 256 a half of one. Otherwise
// parts that two an SM can hold, or one. (us by 1, 2, 3, 4, 5, 6, 8 blocks, rows of 32000 float32, top-k and top-p: 25 rows 29, 22,
// 20, 19, 19, 22, 22; 38 rows 29, 22, 20, 23, 23, 23, 35; 48 rows 30, 23, 26, 24, 24, 37, 40; 76 rows 29, 23, 26, 37, 38, 42, 55;
// 150 rows 29, 29, 46, 56, 62, 77, 92. Rows of 50000, top-p alone, 48 rows by 2, 4, 5, 8: 52, 52, 47, 61.)
template <typename F>
int blocks_of(int R, F bytes) {
  constexpr int kPart = 128 << 10, kHalf = 76 << 10;   // of a block, and of one that leaves room for another
  int best = 0;
  float least = 0.f;
  for (int c = 1; c <= kMaxCluster; ++c) {
    const int b = bytes(c);
    const long long blocks = (long long)R * c;
    if (b > kPart || (c > 1 && bytes(c - 1) <= 16 * kThreads)) continue;   // (or a thread has less than a unit)
    const bool alone = blocks <= (c == 1 || (c == 2 && b <= kTarget) ? kNumSMs : 128);
    if (!alone && (b > kHalf || blocks > (c <= 2 ? 2 * kNumSMs : 256))) continue;
    const float us = (16.f + 0.2f / 1024 * b) * (alone ? 1.f : 1.35f);
    if (!best || us < least) {
      best = c;
      least = us;
    }
  }
  if (!best)
    for (best = 1; best < kMaxCluster && bytes(best) > kTarget;) best *= 2;
  return best;
}

template <typename T>
cudaError_t launch(SampleArgs a, cudaStream_t s) {
  auto bytes = [&](int c) { return (((a.V + Unit<T>::n - 1) / Unit<T>::n + 1 + c - 1) / c) * 16; };
  a.cluster = blocks_of(a.R, bytes);
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(sample_kernel<T>), 160 << 10, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)a.R * a.cluster);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes(a.cluster);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = a.cluster;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int slot = stage_timer_begin(s, kKernSample);
  e = cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, table());
  stage_timer_end(slot, s);
  return e;
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s) { return a.bf16 ? launch<bf16>(a, s) : launch<float>(a, s); }

}  // namespace gdr
