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
// by halving the range eightfold per step: block, warp, an eighth of its run, ... , chunk, lane, entry.
// A pass is bound by the latency of its loads and, over many rows, by its arithmetic (about 20
// instructions an entry); blocks of 256 threads keep 48 rows of 131072 entries resident at once.
// Measured: a row of 32000 entries and five drafts 17.8 -> VERIFY_CHAIN us, 48 trees of 24 nodes over
// 131072 entries 104 -> VERIFY_TREES us against single-entry loads, float64 reductions and 512 threads.
//
// Sums decide whole numbers, so they are carried to about 2^-46: unevaluated pairs of floats (error-free
// sums of two floats) in lanes, warps and blocks, float64 in the scalars of the walk. Float64 throughout
// would run at 1/64 of the float32 rate.
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
__device__ __forceinline__ double wide(Pair a) { return (double)a.hi + (double)a.lo; }
template <int kLanes>
__device__ __forceinline__ Pair lanes_sum(Pair v) {   // the same in every lane of the group
#pragma unroll
  for (int m = kLanes / 2; m >= 1; m >>= 1) v = add(v, {__shfl_xor_sync(kAll, v.hi, m), __shfl_xor_sync(kAll, v.lo, m)});
  return v;
}

// rho of four entries: max(p - c q, 0) with c = ch + cl (q NULL or c = 0: p), or 0 for a token taken out.
template <typename T, bool kVec>
struct Dist {
  const T* p;
  const T* q;
  float ch, cl;
  const int* gone;
  int n_gone, V;
  __device__ __forceinline__ void of(const float* pv, const float* qv, int i, Pair* rho) const {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = above_zero(pv[e]);
      rho[e] = {x, 0.f};
      if (q) {
        const float y = above_zero(qv[e]);
        const float t = __fmul_rn(ch, y), te = __fmaf_rn(cl, y, __fmaf_rn(ch, y, -t));
        float s, r;
        two_sum(x, -t, s, r);
        r = __fadd_rn(r, -te);
        const bool pos = __fadd_rn(s, r) > 0.f;
        rho[e] = {pos ? s : 0.f, pos ? r : 0.f};
      }
    }
    for (int g = 0; g < n_gone; ++g) {
      const int at = gone[g] - i;
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (at == e) rho[e] = {0.f, 0.f};
    }
  }
  // Sum of chunks [c0, c1), the same in every lane.
  __device__ __forceinline__ Pair sum(int c0, int c1) const {
    constexpr int kBatch = 4;   // chunks in flight
    const int lane = threadIdx.x & 31;
    Pair acc[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) acc[e] = {0.f, 0.f};
    for (int c = c0; c < c1; c += kBatch) {
      float pv[kBatch][4], qv[kBatch][4];
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        const int i = c + k < c1 ? (c + k) * kChunk4 + 4 * lane : V;
        load4<kVec>(p, i, V, pv[k]);
        if (q) load4<kVec>(q, i, V, qv[k]);
      }
#pragma unroll
      for (int k = 0; k < kBatch; ++k) {
        Pair rho[4];
        of(pv[k], qv[k], c + k < c1 ? (c + k) * kChunk4 + 4 * lane : V, rho);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[e] = add(acc[e], rho[e]);
      }
    }
    return lanes_sum<32>(add(add(acc[0], acc[1]), add(acc[2], acc[3])));
  }
};

// Of n <= 32 parts (lane r < n holds part r's sum), the first whose running sum passes the target; the
// target then counts from that part's start. Where none passes (the sums agree with the whole only to
// rounding, or u_next is not below 1) the last part that holds anything, and the target becomes
// infinite, so that later steps do the same. -1 if every part is empty.
__device__ __forceinline__ int pick(double v, int n, double& target) {
  const int lane = threadIdx.x & 31;
  double incl = lane < n ? v : 0.0;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    if (m >= n) break;
    const double up = __shfl_up_sync(kAll, incl, m);
    if (lane >= m) incl += up;
  }
  const unsigned over = __ballot_sync(kAll, lane < n && v > 0.0 && incl > target);
  const unsigned any = __ballot_sync(kAll, lane < n && v > 0.0);
  if (over) {
    const int who = __ffs(over) - 1;
    target -= __shfl_sync(kAll, incl - v, who);
    return who;
  }
  target = INFINITY;
  return any ? 31 - __clz(any) : -1;
}

struct Shared {
  Pair ctas[2][kCluster];   // totals of the cluster's blocks, by pass parity
  Pair warps[kWarps];
  float ch, cl;
  int cur, n_gone, act, found, c0, c1;
  double target;
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
  const int b = blockIdx.x / kCluster, rank = (int)ptx::cluster_ctarank();
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int n = __ldg(a.lengths + b);
  if (n < 0 || n > a.N) {   // the same in every block of the cluster
    if (rank == 0 && tid == 0) atomicCAS(a.err, 0, kErrDeviceIndex);
    return;
  }
  const size_t row = (size_t)b * a.N;
  const T* P = static_cast<const T*>(a.p) + row * a.V;
  const T* Q = a.q ? static_cast<const T*>(a.q) + row * a.V : nullptr;
  const double u_next = (double)__ldg(a.u_next + b);
  for (int i = tid + 1; i < n; i += kThreads) {
    int parent = __ldg(a.parents + row + i);
    const int t = __ldg(a.tokens + row + i);
    s_u[i] = __ldg(a.u + row + i);
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

  // the vocabulary's chunks, in contiguous runs: block r's, and of those warp w's
  const int chunks = (a.V + kChunk4 - 1) / kChunk4;
  auto first = [&](int w) { return (int)((long long)chunks * w / (kCluster * kWarps)); };
  const int run0 = first(rank * kWarps + warp), run1 = first(rank * kWarps + warp + 1);

  // thread 0's walk
  int cur = 0, i = 1, count = 0, n_gone = 0, pass = 0;
  double c = 0.0, Z = 1.0, c_new = 0.0;
  bool summed = false, bare = false;   // the totals at hand are the present state's; rho given up for p
  if (tid == 0 && n > 0) s_path[count++] = 0;
  enum { kRefused = 0, kSum = 1, kDone = 2 };
  if (n > 0) {
    while (true) {
      if (tid == 0) {
        int act = -1;
        for (; act < 0 && i < n; ++i) {
          if (s_parent[i] != cur) continue;
          const int t = s_token[i];
          double here = (double)s_p[i];
          if (Q) here = fmax(here - c * (double)s_q[i], 0.0);
          for (int g = 0; g < n_gone; ++g)
            if (s_gone[g] == t) here = 0.0;
          if ((double)s_u[i] * (double)s_q[i] * Z < here) {
            s_path[count++] = i;
            cur = i;
            c = 0.0;
            Z = 1.0;
            n_gone = 0;
            summed = false;
          } else if (Q) {
            c_new = c + Z;
            act = kRefused;
          } else {
            Z -= here;
            s_gone[n_gone++] = t;
          }
        }
        if (act < 0) {
          act = summed ? kDone : kSum;
          c_new = c;
        }
        sh.act = act;
        sh.cur = cur;
        sh.n_gone = n_gone;
        sh.ch = (float)c_new;
        sh.cl = (float)(c_new - (double)sh.ch);
      }
      __syncthreads();
      const int act = sh.act;
      if (act == kDone) break;
      const Dist<T, kVec> dist{P + (size_t)sh.cur * a.V, (Q && sh.ch != 0.f) ? Q + (size_t)sh.cur * a.V : nullptr,
                               sh.ch, sh.cl, s_gone, sh.n_gone, a.V};
      const Pair mine = dist.sum(run0, run1);
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
        const double total = wide(lanes_sum<kCluster>(sh.ctas[par][lane & (kCluster - 1)]));
        if (act == kRefused) {
          summed = total > 0.0;
          if (summed) {
            c = c_new;
            Z = total;
          }
        } else if (total > 0.0 || bare) {
          summed = true;
        } else {   // everything was taken out: the next token comes from p itself
          bare = true;
          n_gone = 0;
          c = 0.0;
        }
      }
    }
    // the next token: the block, the warp, then eighths of the range down to a chunk
    if (warp == 0) {
      const int par = (pass - 1) & 1;
      const Pair mine = sh.ctas[par][lane & (kCluster - 1)];
      double target = u_next * wide(lanes_sum<kCluster>(mine));
      const int block = pick(wide(mine), kCluster, target);
      int w = -1;
      if (block == rank) w = pick(wide(sh.warps[lane & (kWarps - 1)]), kWarps, target);
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
      const Dist<T, kVec> dist{P + (size_t)sh.cur * a.V, (Q && sh.ch != 0.f) ? Q + (size_t)sh.cur * a.V : nullptr,
                               sh.ch, sh.cl, s_gone, sh.n_gone, a.V};
      int c0 = sh.c0, c1 = sh.c1;
      while (c1 - c0 > 1) {
        const int per = (c1 - c0 + kWarps - 1) / kWarps;
        const Pair mine = dist.sum(min(c1, c0 + warp * per), min(c1, c0 + (warp + 1) * per));
        if (lane == 0) sh.warps[warp] = mine;
        __syncthreads();
        if (warp == 0) {
          double target = sh.target;
          const int w = max(0, pick(wide(sh.warps[lane & (kWarps - 1)]), kWarps, target));
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
      if (warp == 0) {
        const int at = c0 * kChunk4 + 4 * lane;
        float pv[4], qv[4];
        load4<kVec>(dist.p, at, a.V, pv);
        if (dist.q) load4<kVec>(dist.q, at, a.V, qv);
        Pair rho[4];
        dist.of(pv, qv, at, rho);
        double target = sh.target;
        const int who = max(0, pick(wide(add(add(rho[0], rho[1]), add(rho[2], rho[3]))), 32, target));
        if (lane == who) {
          int token = at;
          bool found = false;
          double run = 0.0;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const double x = wide(rho[e]);
            run += x;
            if (!found && x > 0.0) {
              token = at + e;           // the last that holds anything, unless one passes the target
              found = run > target;
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

template <typename T>
void launch(const VerifyArgs& a, bool vec, cudaStream_t s) {
  const size_t smem = (size_t)a.N * 7 * 4;
  if (vec) verify_kernel<T, true><<<a.B * kCluster, kThreads, smem, s>>>(a);
  else verify_kernel<T, false><<<a.B * kCluster, kThreads, smem, s>>>(a);
}

}  // namespace

cudaError_t launch_verify_draft(const VerifyArgs& a, cudaStream_t s) {
  const uintptr_t quad = a.bf16 ? 8 : 16;   // bytes of four entries
  const bool vec = a.V % 4 == 0 && reinterpret_cast<uintptr_t>(a.p) % quad == 0 && reinterpret_cast<uintptr_t>(a.q) % quad == 0;
  const int slot = stage_timer_begin(s, kKernVerifyDraft);
  if (a.bf16) launch<__nv_bfloat16>(a, vec, s);
  else launch<float>(a, vec, s);
  const cudaError_t e = cudaGetLastError();
  stage_timer_end(slot, s);
  return e;
}

}  // namespace gdr
