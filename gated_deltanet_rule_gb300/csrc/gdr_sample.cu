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
// can show) lie within a factor of two of it, where the difference is exact. Sums are kept in integers of 2^-40 (associative: no order, no rounding).
//
// A cluster of blocks holds a row in shared memory, read once. The border is found by counting: a histogram over
// 1024 steps of 1/32 of a binary order below the maximum finds the step of the k-th logit, histograms over the
// step's own floats (two, rarely more) the logit. For top-p the counts bound the mass above each step to 2.2%,
// so one pass over all weights takes the total, the mass above the doubtful steps and a histogram of masses over
// those; the rest as for top-k, with masses. The token is found block, warp, run of 16-byte units, lane, entry.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cfloat>
#include <cmath>

#include "gdr_serve.h"
#include "ptx.cuh"

namespace gdr {
namespace {

using bf16 = __nv_bfloat16;
using u64 = unsigned long long;
constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 1024;
constexpr int kPerOctave = 32;      // steps of a binary order in the first histogram
constexpr unsigned kAll = 0xffffffffu;
constexpr int kTarget = 100 << 10;  // bytes of a block's part of a row: two blocks an SM

struct Table {
  float2 t[64];   // 2^(k / 64) as pairs
};

// Two floats in one register pair.
struct F2 {
  u64 v;
};
__device__ __forceinline__ F2 pack(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ F2 both(float x) { return pack(x, x); }
__device__ __forceinline__ void unpack(F2 x, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x.v)); }
__device__ __forceinline__ F2 add(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 mul(F2 a, F2 b) {
  F2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}
__device__ __forceinline__ F2 fma(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 sub(F2 a, F2 b) { return fma(b, both(-1.f), a); }

// What a row's weights are formed from.
struct Scale {
  float ch, cl;   // log2(e) / T
  float ref;      // subtracted from the logits first
  float least;    // smaller differences count as this one (a weight of 2^-150)
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
  const F2 ch = both(s.ch), ph = mul(z, ch), pl = fma(z, both(s.cl), fma(z, ch, mul(ph, both(-1.f))));
  // less the maximum's product: d + dl
  const F2 mh = both(-s.mh), d = add(ph, mh), dd = sub(d, ph);
  const F2 dl = add(add(sub(ph, sub(d, dd)), sub(mh, dd)), add(pl, both(-s.ml)));
  constexpr float kMagic = 196608.f;   // 1.5 2^17: the sum's last place is 1 / 64
  const F2 t = add(d, both(kMagic)), r = sub(d, add(t, both(-kMagic)));   // r exactly
  const F2 x = add(r, dl), xl = sub(dl, sub(x, r));                       // x + xl = r + dl
  // 2^x - 1 = a + b
  constexpr float kL1 = 0.693147182464599609375f, kL1l = -1.9046542999577679e-9f;   // ln 2 as a pair
  constexpr float kL2 = 0.2402265069591007f, kL3 = 0.05550410866482158f, kL4 = 0.009618129107628477f;
  const F2 a = mul(x, both(kL1));
  F2 b = fma(x, both(kL1), mul(a, both(-1.f)));
  b = fma(x, both(kL1l), b);
  b = fma(xl, both(kL1), b);
  b = fma(mul(x, x), fma(x, fma(x, both(kL4), both(kL3)), both(kL2)), b);
  // times 2^(k / 64) 2^e
  float t0, t1;
  unpack(t, t0, t1);
  const int j0 = __float_as_int(t0) - __float_as_int(kMagic), j1 = __float_as_int(t1) - __float_as_int(kMagic);
  const float2 e0 = table[j0 & 63], e1 = table[j1 & 63];
  const float f0 = __int_as_float((127 + 40 + (j0 >> 6)) << 23), f1 = __int_as_float((127 + 40 + (j1 >> 6)) << 23);
  const F2 th = pack(e0.x, e1.x), tl = pack(e0.y, e1.y), f = pack(f0, f1);
  const F2 m = mul(th, a), hi = add(th, m);
  F2 lo = add(sub(m, sub(hi, th)), fma(th, a, mul(m, both(-1.f))));
  lo = add(lo, fma(th, b, tl));
  return {mul(hi, f), mul(lo, f)};
}
__device__ __forceinline__ u64 fixed(float hi, float lo) { return (u64)(__float2ll_rn(hi) + __float2ll_rn(lo)); }
__device__ __forceinline__ u64 weight(const Scale& s, const float2* table, float l) {
  const W2 w = weights(s, table, l, l);
  float h, g, lo;
  unpack(w.hi, h, g);
  unpack(w.lo, lo, g);
  return fixed(h, lo);
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
};

__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, uint32_t v) {
  asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void st_cluster64(uint32_t addr, u64 v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

struct Hist {
  uint32_t n[kBins], lo[kBins], hi[kBins];   // counts, and masses in two words
};
struct Shared {
  float2 table[64];
  Hist hist[2];              // by turns: a block may still read its neighbours' last one
  float tops[kMaxCluster];
  u64 sums[2][3][kMaxCluster];   // the blocks' totals, by turns
  u64 warps[kWarps], chunks[kWarps];
  u64 scan_m[kWarps];
  uint32_t scan_n[kWarps];
  uint32_t edge[2];
  float reds[kWarps];
  // a border search's answer
  int bin;
  uint32_t bin_n, above_n;
  u64 bin_m, above_m;
  int bin2;
  int cut;
};

template <typename T>
struct Row {
  const T* tile;     // this block's part of the row
  int first;         // index of its first entry (may be before the row: such entries are -inf)
  int units;         // of 16 bytes
  int rank, ranks;
  Shared* sh;
  Scale s;
  float top, steps;  // maximum, steps of the first histogram a unit of logits
  int turn_h, turn_s;

  __device__ __forceinline__ int bin_of(float l) const { return (int)fminf((top - l) * steps, (float)(kBins - 1)); }

  // All blocks' v (n of them), in order of rank: sums before this block, and of all.
  template <int n>
  __device__ __forceinline__ void cluster_sums(const u64 (&v)[n], u64 (&before)[n], u64 (&total)[n]) {
    if (threadIdx.x < ranks)
      for (int i = 0; i < n; ++i) st_cluster64(ptx::dsmem_addr(&sh->sums[turn_s][i][rank], threadIdx.x), v[i]);
    ptx::cluster_sync_all();
    for (int i = 0; i < n; ++i) {
      before[i] = total[i] = 0;
      for (int r = 0; r < ranks; ++r) {
        const u64 x = sh->sums[turn_s][i][r];
        if (r < rank) before[i] += x;
        total[i] += x;
      }
    }
    turn_s ^= 1;
  }
  // Sum over the block, in every thread (u64: any order).
  __device__ __forceinline__ u64 block_sum(u64 v) {
    for (int m = 16; m >= 1; m >>= 1) v += __shfl_xor_sync(kAll, v, m);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) sh->warps[threadIdx.x >> 5] = v;
    __syncthreads();
    v = 0;
    for (int w = 0; w < kWarps; ++w) v += sh->warps[w];
    return v;
  }

  // Calls f(x[n], index of x[0]) for the block's units, a thread's share.
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    constexpr int n = Unit<T>::n;
    for (int i = threadIdx.x; i < units; i += kThreads) {
      float x[n];
      Unit<T>::read(reinterpret_cast<const uint4*>(tile)[i], x);
      f(x, first + i * n);
    }
  }

  // Zeroes the histogram of this turn (each block its own), to be filled by `fill`; then finds the first bin at
  // which the running count (or mass) over all blocks reaches `need`. False if the whole does not.
  template <bool kMass, typename F>
  __device__ bool border(u64 need, F fill) {
    Hist& h = sh->hist[turn_h];
    for (int i = threadIdx.x; i < kBins; i += kThreads) {
      h.n[i] = 0;
      if (kMass) h.lo[i] = h.hi[i] = 0;
    }
    if (threadIdx.x == 0) sh->bin = -1;
    __syncthreads();
    fill(h);
    ptx::cluster_sync_all();
    // two neighbouring bins a thread
    const int b0 = 2 * threadIdx.x, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t n[2] = {0, 0};
    u64 m[2] = {0, 0};
    for (int r = 0; r < ranks; ++r) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        n[i] += ld_cluster(ptx::dsmem_addr(&h.n[b0 + i], r));
        if (kMass)
          m[i] += (u64)ld_cluster(ptx::dsmem_addr(&h.lo[b0 + i], r)) + ((u64)ld_cluster(ptx::dsmem_addr(&h.hi[b0 + i], r)) << 32);
      }
    }
    uint32_t in = n[0] + n[1];
    u64 im = m[0] + m[1];
    for (int d = 1; d < 32; d <<= 1) {
      const uint32_t un = __shfl_up_sync(kAll, in, d);
      const u64 um = kMass ? __shfl_up_sync(kAll, im, d) : 0;
      if (lane >= d) {
        in += un;
        im += um;
      }
    }
    if (lane == 31) {
      sh->scan_n[warp] = in;
      sh->scan_m[warp] = im;
    }
    __syncthreads();
    uint32_t bn = in - n[0] - n[1];
    u64 bm = im - m[0] - m[1];
    for (int w = 0; w < warp; ++w) {
      bn += sh->scan_n[w];
      bm += sh->scan_m[w];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u64 a = kMass ? bm : bn, b = a + (kMass ? m[i] : n[i]);
      if (a < need && b >= need) {
        sh->bin = b0 + i;
        sh->bin_n = n[i];
        sh->above_n = bn;
        sh->bin_m = m[i];
        sh->above_m = bm;
      }
      bn += n[i];
      bm += m[i];
    }
    __syncthreads();
    turn_h ^= 1;
    return sh->bin >= 0;
  }

  // Key range of a step of the first histogram: it falls with the key, so its ends are found by bisection.
  __device__ void step_keys(int bin, uint32_t& lo, uint32_t& hi) {
    __syncthreads();
    if (threadIdx.x < 2) {
      const int b = bin - (int)threadIdx.x;   // the smallest key whose step is at most b
      uint32_t l = key_of(-FLT_MAX), r = key_of(top);
      if (b < 0) {
        l = r + 1;
      } else {
        while (l < r) {
          const uint32_t mid = l + (r - l) / 2;
          if (bin_of(of_key(mid)) <= b) r = mid;
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
      const bool got = border<kMass>(need, [&](Hist& h) {
        each([&](const float* x, int) {
#pragma unroll
          for (int e = 0; e < Unit<T>::n; ++e) {
            const uint32_t k = key_of(x[e]);
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
  __device__ __forceinline__ void count(Hist& h, uint32_t b, float l) const {
    if (!kMass) {
      atomicAdd(&h.n[b], 1u);
      return;
    }
    atomicAdd(&h.n[b], 1u);
    const u64 w = weight(s, sh->table, l);
    const uint32_t old = atomicAdd(&h.lo[b], (uint32_t)w);
    const uint32_t up = (uint32_t)(w >> 32) + (old + (uint32_t)w < old);
    if (up) atomicAdd(&h.hi[b], up);
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a, const __grid_constant__ Table tab) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Shared sh;
  using U = Unit<T>;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int ranks = a.cluster, rank = (int)ptx::cluster_ctarank(), row = blockIdx.x / ranks;
  const T* logits = static_cast<const T*>(a.logits) + (long long)row * a.stride;

  const float temperature = __ldg(a.temperature + row);
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
  }
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");   // (waited for before the first remote write)
  if (tid < 64) sh.table[tid] = tab.t[tid];

  Row<T> r;
  r.tile = reinterpret_cast<const T*>(dyn);
  r.sh = &sh;
  r.rank = rank;
  r.ranks = ranks;
  r.turn_h = r.turn_s = 0;
  // 16-byte units from the aligned address at or before the row's first entry
  const int skew = (int)((reinterpret_cast<uintptr_t>(logits) & 15) / sizeof(T));
  const int all = (a.V + skew + U::n - 1) / U::n, per = (all + ranks - 1) / ranks;
  const int u0 = min(all, rank * per);
  r.units = min(all, u0 + per) - u0;
  r.first = u0 * U::n - skew;

  // the row into shared memory, and its largest entry
  float top = -INFINITY;
  {
    uint4* to = reinterpret_cast<uint4*>(dyn);
    const uint4* from = reinterpret_cast<const uint4*>(logits + r.first);
    constexpr int kAhead = 4;
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
        float x[U::n];
        U::read(v[c], x);
#pragma unroll
        for (int e = 0; e < U::n; ++e) {
          x[e] = clean(x[e]);
          top = fmaxf(top, x[e]);
        }
        to[i] = U::write(x);
      }
    }
  }
  if (sizeof(T) == 2) top = fminf(top, kBf16Max);   // (as it was written)
  for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(kAll, top, m));
  if (lane == 0) sh.reds[warp] = top;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sh.reds[w]);
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (tid < ranks) st_cluster(ptx::dsmem_addr(&sh.tops[rank], tid), __float_as_uint(top));
  ptx::cluster_sync_all();
  for (int i = 0; i < ranks; ++i) top = fmaxf(top, sh.tops[i]);
  r.top = top;

  u64 total = 0;
  float border = -INFINITY;   // kept: above it, and the first `ties` that equal it
  uint32_t ties = 0, equal = 0;
  if (top > -INFINITY) {
    {
      const double c = temperature == 0.f ? 1.4426950408889634 : fmin(1.4426950408889634 / (double)temperature, 1e30);
      r.s.ch = (float)c;
      r.s.cl = (float)(c - (double)r.s.ch);
      const bool near = fabsf(top) * r.s.ch < 300.f;
      r.s.ref = near ? 0.f : top;
      const float z = near ? top : 0.f;
      r.s.mh = __fmul_rn(z, r.s.ch);
      r.s.ml = __fmaf_rn(z, r.s.cl, __fmaf_rn(z, r.s.ch, -r.s.mh));
      r.s.least = fmaxf((r.s.mh - 150.f) / r.s.ch, -FLT_MAX);
      r.steps = r.s.ch * (float)kPerOctave;
    }

    // ---------------------------------------------------------------- top-k
    const bool cuts_k = k > 0 && k < a.V, cuts_p = p < 1.f;
    int last_bin = kBins - 1;    // steps that hold kept tokens
    bool counted = false;
    if (cuts_k) {
      auto fill = [&](Hist& h) {
        r.each([&](const float* x, int) {
#pragma unroll
          for (int e = 0; e < U::n; ++e)
            if (x[e] > -INFINITY) atomicAdd(&h.n[r.bin_of(x[e])], 1u);
        });
      };
      if (r.template border<false>((u64)k, fill)) {
        u64 need = (u64)k - sh.above_n;
        last_bin = sh.bin;
        uint32_t lo, hi, key, n;
        r.step_keys(last_bin, lo, hi);
        r.template refine<false>(lo, hi, need, key, n);
        border = of_key(key);
        ties = (uint32_t)need;
        equal = n;
        counted = true;
      }
    }

    // ---------------------------------------------------------------- top-p: of the tokens above the border
    if (cuts_p) {
      // the mass above the border, and a histogram of it
      u64 mine = 0;
      {
        W2 acc = {{0}, {0}};
        r.each([&](const float* x, int) {
          bool some = false;
#pragma unroll
          for (int e = 0; e < U::n; ++e) some |= x[e] > border;
          if (!some) return;
#pragma unroll
          for (int e = 0; e < U::n; e += 2) {
            const W2 w = weights(r.s, sh.table, x[e], x[e + 1]);
            const F2 on = pack(x[e] > border ? 1.f : 0.f, x[e + 1] > border ? 1.f : 0.f);
            accumulate(acc, mul(w.hi, on), mul(w.lo, on));
          }
        });
        mine = fixed(acc);
      }
      const u64 v[1] = {r.block_sum(mine)};
      u64 before[1], sum[1];
      r.cluster_sums(v, before, sum);
      const u64 each_tie = counted ? weight(r.s, sh.table, border) : 0;
      const double mass = (double)(sum[0] + ties * each_tie) * (double)p;
      u64 need = max((u64)1, (u64)ceil(mass));
      auto fill = [&](Hist& h) {
        r.each([&](const float* x, int) {
#pragma unroll
          for (int e = 0; e < U::n; ++e)
            if (x[e] > border) r.template count<true>(h, r.bin_of(x[e]), x[e]);
        });
      };
      if (r.template border<true>(need, fill)) {
        need -= sh.above_m;
        const int bin = sh.bin;
        uint32_t lo, hi, key, n;
        r.step_keys(bin, lo, hi);
        if (counted) lo = max(lo, key_of(border) + 1);
        if (r.template refine<true>(lo, hi, need, key, n)) {
          border = of_key(key);
          const u64 w = max((u64)1, weight(r.s, sh.table, border));
          ties = (uint32_t)min((u64)n, (need + w - 1) / w);
          equal = n;
        }
      } else if (counted && each_tie > 0 && need > sum[0]) {   // inside the tokens that equal the k-th
        ties = (uint32_t)min((u64)ties, (need - sum[0] + each_tie - 1) / each_tie);
      }
    }

    // ---------------------------------------------------------------- min-p
    if (min_p > 0.f && temperature > 0.f) {
      const double least = (double)top + (double)temperature * log((double)min_p);
      const float f = __double2float_ru(least) + 0.f;   // the smallest logit that is kept
      if (f > border) {
        border = of_key(key_of(f) - (f == 0.f ? 2 : 1));   // the float below it
        ties = 0;
      }
    }

    // ---------------------------------------------------------------- which of the equal ones
    const bool part = ties > 0 && ties < equal;
    int cut = ties > 0 ? 0x7fffffff : -1;   // the last index of them that is kept
    // a warp's run of units
    const int run = (r.units + kWarps - 1) / kWarps, w0 = min(r.units, warp * run), w1 = min(r.units, w0 + run);
    const uint4* tile = reinterpret_cast<const uint4*>(dyn);
    // The entry at which the running sum of g(x, index) over the row passes target: its index goes to `found` in
    // the one block that holds it (the warps' sums being in sh.warps, those before this block `before`).
    auto search = [&](u64 target, u64 before, auto g, auto found) {
      u64 at = before;
      int w = 0;
      for (; w < kWarps && at + sh.warps[w] <= target; ++w) at += sh.warps[w];
      if (before > target || w == kWarps) return;
      // the warps share that run: a 32-unit piece each
      const int i0 = min(r.units, w * run) + warp * 32 + lane, end = min(r.units, (w + 1) * run);
      float x[U::n];
      u64 v[U::n], mine = 0;
      const int base = r.first + i0 * U::n;
      if (warp * 32 < run) {
        if (i0 < end) U::read(tile[i0], x);
#pragma unroll
        for (int e = 0; e < U::n; ++e) {
          v[e] = i0 < end ? g(x[e], base + e) : 0;
          mine += v[e];
        }
      }
      u64 incl = mine;
      for (int d = 1; d < 32; d <<= 1) {
        const u64 up = __shfl_up_sync(kAll, incl, d);
        if (lane >= d) incl += up;
      }
      if (lane == 31) sh.chunks[warp] = incl;
      __syncthreads();
      int c = 0, last = 0;
      u64 from = at;
      for (; c < kWarps && from + sh.chunks[c] <= target; ++c) {
        from += sh.chunks[c];
        if (sh.chunks[c]) last = c;
      }
      const bool none = c == kWarps;   // (sums of pieces and of the run differ by roundings: then the last entry)
      if (warp == (none ? last : c)) {
        const unsigned over = __ballot_sync(kAll, none ? mine > 0 : from + incl > target);
        if (over && lane == (none ? 31 - __clz(over) : __ffs(over) - 1)) {
          u64 s = from + incl - mine;
          int hit = -1;
#pragma unroll
          for (int e = 0; e < U::n; ++e) {
            s += v[e];
            if (v[e] && (none || (s > target && hit < 0))) hit = base + e;
          }
          found(hit);
        }
      }
      __syncthreads();
    };
    if (part) {
      auto is = [&](float x, int) { return (u64)(x == border); };
      u64 n = 0;
      for (int i = w0 + lane; i < w1; i += 32) {
        float x[U::n];
        U::read(tile[i], x);
#pragma unroll
        for (int e = 0; e < U::n; ++e) n += is(x[e], 0);
      }
      u64 v[1] = {r.block_sum(n)}, before[1], sum[1];
      r.cluster_sums(v, before, sum);
      search(ties - 1, before[0], is, [&](int at) {
        for (int i = 0; i < ranks; ++i) st_cluster(ptx::dsmem_addr(&sh.cut, i), (uint32_t)at);
      });
      ptx::cluster_sync_all();
      cut = sh.cut;
    }

    // ---------------------------------------------------------------- the kept mass, the token
    auto kept = [&](float x, int at) { return x > border || (x == border && x > -INFINITY && at <= cut); };
    u64 mine = 0;
    {
      W2 acc = {{0}, {0}};
      for (int i = w0 + lane; i < w1; i += 32) {
        float x[U::n];
        U::read(tile[i], x);
        const int at = r.first + i * U::n;
        bool some = false;
#pragma unroll
        for (int e = 0; e < U::n; ++e) some |= kept(x[e], at + e);
        if (!some) continue;
#pragma unroll
        for (int e = 0; e < U::n; e += 2) {
          const W2 w = weights(r.s, sh.table, x[e], x[e + 1]);
          const F2 on = pack(kept(x[e], at + e) ? 1.f : 0.f, kept(x[e + 1], at + e + 1) ? 1.f : 0.f);
          accumulate(acc, mul(w.hi, on), mul(w.lo, on));
        }
      }
      mine = fixed(acc);
    }
    const u64 v[1] = {r.block_sum(mine)};
    u64 before[1], sum[1];
    r.cluster_sums(v, before, sum);
    total = sum[0];
    if (a.token) {
      const float u = __ldg(a.u + row);
      const double at = u > 0.f ? (double)fminf(u, 1.f) * (double)total : 0.0;
      const u64 target = min((u64)at, total - 1);
      search(target, before[0], [&](float x, int i) { return kept(x, i) ? weight(r.s, sh.table, x) : (u64)0; },
             [&](int i) { a.token[row] = i; });
    }
    if (a.probs) {
      float* out = a.probs + (long long)row * a.V;
      const float inv = 1.f / (float)total;
      const T* x = r.tile;
      for (int i = tid; i < r.units * U::n; i += kThreads) {
        const int at = r.first + i;
        if (at < 0 || at >= a.V) continue;
        const float l = U::one(x + i);
        float w = 0.f;
        if (kept(l, at)) {
          const W2 both_w = weights(r.s, sh.table, l, l);
          float h, g;
          unpack(add(both_w.hi, both_w.lo), h, g);
          w = h * inv;
        }
        out[at] = w;
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

template <typename T>
cudaError_t launch(SampleArgs a, cudaStream_t s) {
  // Blocks of a row: enough for their parts to fit two an SM, and more of them while there are few rows.
  auto bytes = [&](int c) { return (((a.V + Unit<T>::n - 1) / Unit<T>::n + 1 + c - 1) / c) * 16; };
  a.cluster = 1;
  while (a.cluster < kMaxCluster && (bytes(a.cluster) > kTarget || (a.R * a.cluster < 2 * kNumSMs && bytes(a.cluster) > 16 * kThreads)))
    a.cluster *= 2;
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
