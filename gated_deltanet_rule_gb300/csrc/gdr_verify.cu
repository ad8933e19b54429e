// Verification of drafted tokens against the target's probabilities (speculative sampling over a
// tree, a chain being the tree of one child each).
//
// The walk starts at the root. At a node with target distribution p the candidates are its children
// in index order; with (c, Z) = (0, 1) at first and rho = max(p - c q, 0), candidate t is accepted if
//   u q(t) Z < rho(t),
// and a refusal takes the residual on. Normalised residuals max(rho / Z - q, 0) keep this form: they
// are max(p - c' q, 0) / Z' with c' = c + Z and Z' = sum max(p - c' q, 0), so the whole state of a
// node is two numbers and each refusal costs one pass over the vocabulary (none for given drafts,
// q NULL: there a refused token's probability is taken out and Z loses it). A residual with nothing
// left is dropped: the state stays as it was. When no candidate is left the next token is the
// smallest index whose running sum of rho passes u_next times the total.
//
// One cluster of eight blocks takes a row: every block walks the tree on the same scalars (gathered
// once, so the walk runs in shared memory), and a pass splits the vocabulary over the cluster's 64
// warps, each a contiguous run of 128-entry chunks (four entries a lane, 16-byte loads where rows are
// aligned), whose sums the blocks exchange through distributed shared memory. The token is then found
// step by step: block, warp, an eighth of its run, ... , and then chunk, lane and entry at once.
// A pass is bound by the latency of its loads and, over many rows, by its arithmetic (about 20
// instructions an entry); blocks of 256 threads keep 48 rows of 131072 entries resident at once.
// Measured: a float32 chain of 6 over 32000 entries 8.9 us, 48 float32 trees of 24 over 131072 35 to 46 us by
// how many drafts the inputs have refused. Steps (on one input):
// float64 reductions and scalars 17.8 / 104 us; pairs of floats in the passes, four entries a lane,
// asynchronous copies 12.4 / 41.0 us; pairs in the walk and the search as well 10.2 / 39 us; the last chunks
// searched at once by one warp, first nodes read along with the length 8.5 / 39 us. Clusters of sixteen
// shorten a row's pass but no longer keep the rows resident: 12.4 / 50.5 us against 12.4 / 41.0. Two chunks
// at a time spill: 11.0 / 44.1 us.
//
// Sums decide whole numbers, so they are carried to about 2^-46: unevaluated pairs of floats (Knuth's
// error-free sum of two floats) throughout. Float64, at 1/64 of the float32 rate, took longer for the walk's and the
// search's few scalars than the passes did for the vocabulary.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdr_serve.h"
#include "ptx.cuh"

namespace gdr {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kChunk4 = 128;   // entries of a chunk: four a lane
constexpr int kAhead = 8;      // chunks of p and q on their way to a thread
constexpr int kLast = 4;       // chunks that one warp searches at once
constexpr unsigned kAll = 0xffffffffu;

__device__ __forceinline__ float above_zero(float x) { return x > 0.f ? x : 0.f; }   // nan and negatives count as 0
__device__ __forceinline__ float prob(const float* p) { return above_zero(__ldg(p)); }
__device__ __forceinline__ float prob(const __nv_bfloat16* p) { return above_zero(__bfloat162float(*p)); }

// Entries i .. i + 3 of a row of V (0 past its end); kVec: V and the rows are multiples of four entries.
template <bool kVec>
__device__ __forceinline__ void load4(const float* p, int i, int V, float* x) {
  if (kVec) {
    const float4 v = i < V ? __ldg(reinterpret_cast<const float4*>(p + i)) : make_float4(0.f, 0.f, 0.f, 0.f);
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = i + e < V ? __ldg(p + i + e) : 0.f;
  }
}
template <bool kVec>
__device__ __forceinline__ void load4(const __nv_bfloat16* p, int i, int V, float* x) {
  if (kVec) {
    const uint2 v = i < V ? __ldg(reinterpret_cast<const uint2*>(p + i)) : make_uint2(0u, 0u);
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xFFFF0000u);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] = i + e < V ? __bfloat162float(p[i + e]) : 0.f;
  }
}

// Four entries copied asynchronously to shared memory, and read from there.
__device__ __forceinline__ void copy4(void* to, const float* from) { ptx::cp_async16_zfill(to, from, 16); }
__device__ __forceinline__ void copy4(void* to, const __nv_bfloat16* from) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(ptx::smem_u32(to)), "l"(from) : "memory");
}
__device__ __forceinline__ void read4(const float* p, bool there, float* x) {
  const float4 v = there ? *reinterpret_cast<const float4*>(p) : make_float4(0.f, 0.f, 0.f, 0.f);
  x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
}
__device__ __forceinline__ void read4(const __nv_bfloat16* p, bool there, float* x) {
  const uint2 v = there ? *reinterpret_cast<const uint2*>(p) : make_uint2(0u, 0u);
  x[0] = __uint_as_float(v.x << 16);
  x[1] = __uint_as_float(v.x & 0xFFFF0000u);
  x[2] = __uint_as_float(v.y << 16);
  x[3] = __uint_as_float(v.y & 0xFFFF0000u);
}

// A sum as an unevaluated pair hi + lo.
struct Pair {
  float hi, lo;
};
// a + b as s + e exactly
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float bb = __fadd_rn(s, -a);
  e = __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -bb)), __fadd_rn(b, -bb));
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  float s, e;
  two_sum(a.hi, b.hi, s, e);
  return {s, __fadd_rn(__fadd_rn(a.lo, b.lo), e)};
}
__device__ __forceinline__ Pair negative(Pair a) { return {-a.hi, -a.lo}; }
__device__ __forceinline__ Pair times(float x, Pair a) {
  const float h = __fmul_rn(x, a.hi), l = __fmaf_rn(x, a.lo, __fmaf_rn(x, a.hi, -h)), s = __fadd_rn(h, l);
  return {s, __fadd_rn(l, -__fadd_rn(s, -h))};
}
// whether a > b (false where a difference is nan: an infinite b, an infinite total)
__device__ __forceinline__ bool above(Pair a, Pair b) {
  float s, e;
  two_sum(a.hi, -b.hi, s, e);
  return __fadd_rn(s, __fadd_rn(e, __fadd_rn(a.lo, -b.lo))) > 0.f;
}
template <int kLanes>
__device__ __forceinline__ Pair lanes_sum(Pair v) {   // the same in every lane of the group
#pragma unroll
  for (int m = kLanes / 2; m >= 1; m >>= 1) v = add(v, {__shfl_xor_sync(kAll, v.hi, m), __shfl_xor_sync(kAll, v.lo, m)});
  return v;
}

// Two floats in one register pair: a pass over many rows is bound by its arithmetic, which the packed
// operations halve.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 pack(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
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
__device__ __forceinline__ F2 sub(F2 a, F2 b) { return fma(b, pack(-1.f, -1.f), a); }   // a - b, one rounding
// a + b as s + e exactly, and a - b
__device__ __forceinline__ void two_sum(F2 a, F2 b, F2& s, F2& e) {
  s = add(a, b);
  const F2 bb = sub(s, a);
  e = add(sub(a, sub(s, bb)), sub(b, bb));
}
__device__ __forceinline__ void two_diff(F2 a, F2 b, F2& s, F2& e) {
  s = sub(a, b);
  const F2 bb = sub(s, a);
  e = sub(sub(a, sub(s, bb)), add(b, bb));
}

// Two sums at once.
struct Pair2 {
  F2 hi, lo;
};
__device__ __forceinline__ Pair2 add(Pair2 a, Pair2 b) {
  F2 s, e;
  two_sum(a.hi, b.hi, s, e);
  return {s, add(add(a.lo, b.lo), e)};
}
__device__ __forceinline__ void halves(Pair2 x, Pair& a, Pair& b) {
  unpack(x.hi, a.hi, b.hi);
  unpack(x.lo, a.lo, b.lo);
}
__device__ __forceinline__ Pair both(Pair2 x) {
  Pair a, b;
  halves(x, a, b);
  return add(a, b);
}

// rho of four entries: max(p - c q, 0) with c = ch + cl (q NULL or c = 0: p), or 0 for a token taken out.
template <typename T, bool kVec>
struct Dist {
  const T* p;
  const T* q;
  float ch, cl;
  const int* gone;
  int n_gone, V;
  __device__ __forceinline__ void of(const float* pv, const float* qv, int i, Pair2* rho) const {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const F2 x = pack(above_zero(pv[2 * h]), above_zero(pv[2 * h + 1]));
      rho[h] = {x, {0}};
      if (q) {
        const F2 y = pack(above_zero(qv[2 * h]), above_zero(qv[2 * h + 1]));
        F2 s, r;
        if (ch == 1.f && cl == 0.f) {   // the first refusal
          two_diff(x, y, s, r);
        } else {
          const F2 c = pack(ch, ch), t = mul(c, y);
          two_diff(x, t, s, r);
          r = sub(r, fma(pack(cl, cl), y, fma(c, y, sub({0}, t))));   // less the product's own error
        }
        float s0, s1, r0, r1, g0, g1;
        unpack(add(s, r), g0, g1);
        unpack(s, s0, s1);
        unpack(r, r0, r1);
        rho[h] = {pack(g0 > 0.f ? s0 : 0.f, g1 > 0.f ? s1 : 0.f), pack(g0 > 0.f ? r0 : 0.f, g1 > 0.f ? r1 : 0.f)};
      }
    }
    for (int g = 0; g < n_gone; ++g) {
      const int at = gone[g] - i;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float s0, s1;
        unpack(rho[h].hi, s0, s1);
        rho[h].hi = pack(at == 2 * h ? 0.f : s0, at == 2 * h + 1 ? 0.f : s1);   // (given drafts: lo is 0)
      }
    }
  }
  // Sum of chunks [c0, c1), the same in every lane. The latency of the loads is what a pass costs: with
  // aligned rows each thread keeps kAhead chunks on their way into its own places of `ring`, else four in
  // registers.
  __device__ __forceinline__ Pair sum(int c0, int c1, uint8_t* ring) const {
    const int lane = threadIdx.x & 31;
    Pair2 acc[2] = {{{0}, {0}}, {{0}, {0}}};
    auto take = [&](const float* pv, const float* qv, int i) {
      Pair2 rho[2];
      of(pv, qv, i, rho);
#pragma unroll
      for (int h = 0; h < 2; ++h) acc[h] = add(acc[h], rho[h]);
    };
    if constexpr (kVec) {
      constexpr int kPiece = 4 * sizeof(T);   // bytes of four entries
      uint8_t* mine = ring + threadIdx.x * kPiece;
      auto place = [&](int slot, int of_q) { return mine + (2 * slot + of_q) * kThreads * kPiece; };
      auto copy = [&](int c, int slot) {
        const int i = c * kChunk4 + 4 * lane;
        if (c < c1 && i < V) {
          copy4(place(slot, 0), p + i);
          if (q) copy4(place(slot, 1), q + i);
        }
        ptx::cp_async_commit();
      };
#pragma unroll
      for (int k = 0; k < kAhead; ++k) copy(c0 + k, k);
      int slot = 0;
      for (int c = c0; c < c1; ++c, slot = slot + 1 == kAhead ? 0 : slot + 1) {
        ptx::cp_async_wait<kAhead - 1>();
        const int i = c * kChunk4 + 4 * lane;
        float pv[4], qv[4];
        read4(reinterpret_cast<const T*>(place(slot, 0)), i < V, pv);
        if (q) read4(reinterpret_cast<const T*>(place(slot, 1)), i < V, qv);
        copy(c + kAhead, slot);
        take(pv, qv, i);
      }
    } else {
      constexpr int kBatch = 4;
      for (int c = c0; c < c1; c += kBatch) {
        float pv[kBatch][4], qv[kBatch][4];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
          const int i = c + k < c1 ? (c + k) * kChunk4 + 4 * lane : V;
          load4<kVec>(p, i, V, pv[k]);
          if (q) load4<kVec>(q, i, V, qv[k]);
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k) take(pv[k], qv[k], c + k < c1 ? (c + k) * kChunk4 + 4 * lane : V);
      }
    }
    return lanes_sum<32>(both(add(acc[0], acc[1])));
  }
};

// Of kParts <= 32 parts (lane r holds part r's sum), the first whose running sum passes the target; the
// target then counts from that part's start. Where none passes (the sums agree with the whole only to
// rounding, or u_next is not below 1) the last part that holds anything, and the target becomes infinite,
// so that later steps do the same. -1 if every part is empty.
template <int kParts>
__device__ __forceinline__ int pick(Pair v, Pair& target) {
  const int lane = threadIdx.x & 31;
  if (lane >= kParts) v = {0.f, 0.f};
  const bool holds = v.hi > 0.f;
  Pair incl = v;
#pragma unroll
  for (int m = 1; m < kParts; m <<= 1) {
    const Pair up = {__shfl_up_sync(kAll, incl.hi, m), __shfl_up_sync(kAll, incl.lo, m)};
    if (lane >= m) incl = add(up, incl);
  }
  const unsigned over = __ballot_sync(kAll, holds && above(incl, target)), any = __ballot_sync(kAll, holds);
  if (over) {
    const int who = __ffs(over) - 1, from = who > 0 ? who - 1 : 0;
    const Pair before = {__shfl_sync(kAll, incl.hi, from), __shfl_sync(kAll, incl.lo, from)};
    if (who > 0) target = add(target, negative(before));
    return who;
  }
  target = {INFINITY, 0.f};
  return any ? 31 - __clz(any) : -1;
}

// Bytes before the ring: seven words a node.
__host__ __device__ constexpr int ring_at(int N) { return (N * 28 + 15) & ~15; }

struct Shared {
  Pair ctas[2][kCluster];   // totals of the cluster's blocks, by pass parity
  Pair warps[kWarps];
  Pair c, target;
  int cur, n_gone, act, found, c0, c1;
};

template <typename T, bool kVec>
__global__ void __launch_bounds__(kThreads, 3) __cluster_dims__(kCluster, 1, 1) verify_kernel(const VerifyArgs a) {
  extern __shared__ __align__(16) uint8_t dyn[];
  __shared__ Shared sh;
  float* s_p = reinterpret_cast<float*>(dyn);          // p and q of node i's token at its parent
  float* s_q = s_p + a.N;
  float* s_u = s_q + a.N;
  int* s_parent = reinterpret_cast<int*>(s_u + a.N);   // -1: not a candidate
  int* s_token = s_parent + a.N;
  int* s_path = s_token + a.N;
  int* s_gone = s_path + a.N;
  uint8_t* ring = dyn + ring_at(a.N);
  const int b = blockIdx.x / kCluster, rank = (int)ptx::cluster_ctarank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const size_t row = (size_t)b * a.N;
  // (a thread's first node is read along with the length)
  const int n = __ldg(a.lengths + b);
  const bool there = tid + 1 < a.N;
  const int parent1 = there ? __ldg(a.parents + row + tid + 1) : 0, token1 = there ? __ldg(a.tokens + row + tid + 1) : 0;
  const float u1 = there ? __ldg(a.u + row + tid + 1) : 0.f;
  if (n < 0 || n > a.N) {   // the same in every block of the cluster
    if (rank == 0 && tid == 0) atomicCAS(a.err, 0, kErrDeviceIndex);
    return;
  }
  // (no block writes to another's shared memory before that one has started: arrived here, waited for below)
  asm volatile("barrier.cluster.arrive.relaxed.aligned;" ::: "memory");
  const T* P = static_cast<const T*>(a.p) + row * a.V;
  const T* Q = a.q ? static_cast<const T*>(a.q) + row * a.V : nullptr;
  const float u_next = __ldg(a.u_next + b);
  for (int i = tid + 1; i < n; i += kThreads) {
    int parent = i == tid + 1 ? parent1 : __ldg(a.parents + row + i);
    const int t = i == tid + 1 ? token1 : __ldg(a.tokens + row + i);
    s_u[i] = i == tid + 1 ? u1 : __ldg(a.u + row + i);
    if (parent < 0 || parent >= i || t < 0 || t >= a.V) {
      atomicCAS(a.err, 0, kErrDeviceIndex);
      parent = -1;
    } else {
      s_p[i] = prob(P + (size_t)parent * a.V + t);
      s_q[i] = Q ? prob(Q + (size_t)parent * a.V + t) : 1.f;
    }
    s_parent[i] = parent;
    s_token[i] = t;
  }
  __syncthreads();
  asm volatile("barrier.cluster.wait.aligned;" ::: "memory");

  // the vocabulary's chunks, in contiguous runs: block r's, and of those warp w's
  const int chunks = (a.V + kChunk4 - 1) / kChunk4;
  auto first = [&](int w) { return (int)((long long)chunks * w / (kCluster * kWarps)); };
  const int run0 = first(rank * kWarps + warp), run1 = first(rank * kWarps + warp + 1);

  // warp 0's walk, the same in all its lanes
  int cur = 0, i = 1, count = 0, n_gone = 0, pass = 0;
  Pair c = {0.f, 0.f}, Z = {1.f, 0.f}, c_new = {0.f, 0.f};
  bool fresh = true;                   // (c, Z) = (0, 1)
  bool summed = false, bare = false;   // the totals at hand are the present state's; rho given up for p
  if (warp == 0 && n > 0) {
    if (lane == 0) s_path[0] = 0;
    count = 1;
  }
  enum { kRefused = 0, kSum = 1, kDone = 2 };
  if (n > 0) {
    while (true) {
      if (warp == 0) {
        int act = -1;
        while (act < 0 && i < n) {
          // the next candidate: the first node from i on whose parent is cur
          const unsigned child = __ballot_sync(kAll, i + lane < n && s_parent[min(i + lane, n - 1)] == cur);
          if (!child) {
            i += 32;
            continue;
          }
          i += __ffs(child) - 1;
          const float pi = s_p[i], qi = s_q[i], ui = s_u[i];
          bool yes;
          Pair here = {pi, 0.f};
          if (fresh) {
            // u q < p: the float product decides, or where it equals p its error does
            const float uq = __fmul_rn(ui, qi);
            yes = uq < pi || (uq == pi && __fmaf_rn(ui, qi, -uq) < 0.f);
          } else {
            if (Q) {
              here = add(here, negative(times(qi, c)));
              if (!(here.hi > 0.f)) here = {0.f, 0.f};
            }
            for (int g = 0; g < n_gone; ++g)
              if (s_gone[g] == s_token[i]) here = {0.f, 0.f};
            yes = above(here, times(ui, times(qi, Z)));
          }
          if (yes) {
            if (lane == 0) s_path[count] = i;
            ++count;
            cur = i;
            c = {0.f, 0.f};
            Z = {1.f, 0.f};
            fresh = true;
            n_gone = 0;
            summed = false;
          } else if (Q) {
            c_new = add(c, Z);
            act = kRefused;
          } else {
            Z = add(Z, negative(here));
            fresh = false;
            if (lane == 0) s_gone[n_gone] = s_token[i];
            ++n_gone;
            __syncwarp();
          }
          ++i;
        }
        if (act < 0) {
          act = summed ? kDone : kSum;
          c_new = c;
        }
        if (lane == 0) {
          sh.act = act;
          sh.cur = cur;
          sh.n_gone = n_gone;
          sh.c = c_new;
        }
      }
      __syncthreads();
      const int act = sh.act;
      if (act == kDone) break;
      const Dist<T, kVec> dist{P + (size_t)sh.cur * a.V, (Q && sh.c.hi != 0.f) ? Q + (size_t)sh.cur * a.V : nullptr,
                               sh.c.hi, sh.c.lo, s_gone, sh.n_gone, a.V};
      const Pair mine = dist.sum(run0, run1, ring);
      if (lane == 0) sh.warps[warp] = mine;
      __syncthreads();
      const int par = pass & 1;
      if (warp == 0) {   // the block's total, told to every block by a lane each
        const Pair total = lanes_sum<kWarps>(sh.warps[lane & (kWarps - 1)]);
        if (lane < kCluster)
          asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(ptx::dsmem_addr(&sh.ctas[par][rank], lane)),
                       "f"(total.hi), "f"(total.lo)
                       : "memory");
      }
      ptx::cluster_sync_all();
      ++pass;
      if (warp == 0) {
        const Pair total = lanes_sum<kCluster>(sh.ctas[par][lane & (kCluster - 1)]);
        if (act == kRefused) {
          summed = total.hi > 0.f;
          if (summed) {
            c = c_new;
            Z = total;
            fresh = false;
          }
        } else if (total.hi > 0.f || bare) {
          summed = true;
        } else {   // everything was taken out: the next token comes from p itself
          bare = true;
          n_gone = 0;
          c = {0.f, 0.f};
          fresh = true;
        }
      }
    }
    // the next token: the block, the warp, then eighths of the range down to a chunk
    if (warp == 0) {
      const int par = (pass - 1) & 1;
      const Pair mine = sh.ctas[par][lane & (kCluster - 1)];
      Pair target = times(u_next, lanes_sum<kCluster>(mine));
      const int block = pick<kCluster>(mine, target);
      int w = -1;
      if (block == rank) w = pick<kWarps>(sh.warps[lane & (kWarps - 1)], target);
      if (lane == 0) {
        sh.found = block == rank;
        sh.c0 = first(rank * kWarps + w);
        sh.c1 = first(rank * kWarps + w + 1);
        sh.target = target;
        if (block < 0 && rank == 0) a.next_token[b] = -1;   // an empty distribution
      }
    }
    __syncthreads();
    if (sh.found) {
      const Dist<T, kVec> dist{P + (size_t)sh.cur * a.V, (Q && sh.c.hi != 0.f) ? Q + (size_t)sh.cur * a.V : nullptr,
                               sh.c.hi, sh.c.lo, s_gone, sh.n_gone, a.V};
      int c0 = sh.c0, c1 = sh.c1;
      while (c1 - c0 > kLast) {   // a step down: to an eighth of the range
        const int per = (c1 - c0 + kWarps - 1) / kWarps;
        const int mine0 = min(c1, c0 + warp * per), mine1 = min(c1, mine0 + per);
        const Pair mine = dist.sum(mine0, mine1, ring);
        if (lane == 0) sh.warps[warp] = mine;
        __syncthreads();
        if (warp == 0) {
          Pair target = sh.target;
          const int w = max(0, pick<kWarps>(sh.warps[lane & (kWarps - 1)], target));
          if (lane == 0) {
            sh.c0 = c0 + w * per;
            sh.c1 = min(c1, c0 + (w + 1) * per);
            sh.target = target;
          }
        }
        __syncthreads();
        c0 = sh.c0;
        c1 = sh.c1;
      }
      if (warp == 0) {   // the last chunks at once: the chunk, the lane, the entry
        Pair target = sh.target;
        Pair rho[4], lanes[kLast], mine = {0.f, 0.f};
        float pv[kLast][4], qv[kLast][4];
#pragma unroll
        for (int k = 0; k < kLast; ++k) {
          const int i = c0 + k < c1 ? (c0 + k) * kChunk4 + 4 * lane : a.V;
          load4<kVec>(dist.p, i, a.V, pv[k]);
          if (dist.q) load4<kVec>(dist.q, i, a.V, qv[k]);
        }
#pragma unroll
        for (int k = 0; k < kLast; ++k) {
          Pair2 two[2];
          dist.of(pv[k], qv[k], c0 + k < c1 ? (c0 + k) * kChunk4 + 4 * lane : a.V, two);
          lanes[k] = both(add(two[0], two[1]));
          const Pair sum = lanes_sum<32>(lanes[k]);
          if (lane == k) mine = sum;
        }
        const int chunk = max(0, pick<kLast>(mine, target));
        Pair at_lane = lanes[0];
#pragma unroll
        for (int k = 1; k < kLast; ++k) {
          if (chunk == k) {
            at_lane = lanes[k];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              pv[0][e] = pv[k][e];
              qv[0][e] = qv[k][e];
            }
          }
        }
        const int who = max(0, pick<32>(at_lane, target));
        if (lane == who) {
          const int at = (c0 + chunk) * kChunk4 + 4 * lane;
          Pair2 two[2];
          dist.of(pv[0], qv[0], at, two);
          halves(two[0], rho[0], rho[1]);
          halves(two[1], rho[2], rho[3]);
          int token = at;
          bool found = false;
          Pair run = {0.f, 0.f};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            run = add(run, rho[e]);
            if (!found && rho[e].hi > 0.f) {
              token = at + e;           // the last that holds anything, unless one passes the target
              found = above(run, target);
            }
          }
          a.next_token[b] = token;
        }
      }
    }
  } else if (rank == 0 && tid == 0) {
    a.next_token[b] = -1;
  }
  if (rank == 0) {
    __syncthreads();
    if (tid == 0) {
      sh.n_gone = count;
      a.n_path[b] = count;
    }
    __syncthreads();
    for (int j = tid; j < a.N; j += kThreads) a.path[row + j] = j < sh.n_gone ? s_path[j] : -1;
  }
  ptx::cluster_sync_all();   // no block leaves while another may still write to its shared memory
}

template <typename T, bool kVec>
cudaError_t launch(const VerifyArgs& a, cudaStream_t s) {
  constexpr int kRing = kVec ? kAhead * 2 * kThreads * 4 * (int)sizeof(T) : 0;
  static std::atomic<uint64_t> done{0};
  const cudaError_t e = allow_smem(reinterpret_cast<const void*>(verify_kernel<T, kVec>), ring_at(kVerifyMaxNodes) + kRing, done);
  if (e != cudaSuccess) return e;
  verify_kernel<T, kVec><<<a.B * kCluster, kThreads, ring_at(a.N) + kRing, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_verify_draft(const VerifyArgs& a, cudaStream_t s) {
  const uintptr_t quad = a.bf16 ? 8 : 16;   // bytes of four entries
  const bool vec = a.V % 4 == 0 && reinterpret_cast<uintptr_t>(a.p) % quad == 0 && reinterpret_cast<uintptr_t>(a.q) % quad == 0;
  const int slot = stage_timer_begin(s, kKernVerifyDraft);
  const cudaError_t e = a.bf16 ? (vec ? launch<__nv_bfloat16, true>(a, s) : launch<__nv_bfloat16, false>(a, s))
                               : (vec ? launch<float, true>(a, s) : launch<float, false>(a, s));
  stage_timer_end(slot, s);
  return e;
}

}  // namespace gdr
