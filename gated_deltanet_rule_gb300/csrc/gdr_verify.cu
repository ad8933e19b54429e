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
// once, so the walk runs in shared memory), and a pass splits the vocabulary over the cluster's 128
// warps, each a contiguous run, whose sums the blocks exchange through distributed shared memory.
// The reads of a pass are latency-bound; more blocks a row would shorten it, fewer leave SMs idle at
// one row.
//
// Sums decide whole numbers, so they are carried to about 2^-46: each lane adds its terms as an
// unevaluated pair of floats (error-free sums of two floats), lanes and warps add in float64. Float64
// alone would do the same at 1/64 of the rate.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "gdr_serve.h"
#include "ptx.cuh"

namespace gdr {
namespace {

constexpr int kCluster = 8;
constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

template <typename T>
__device__ __forceinline__ float prob(const T* p);
template <>
__device__ __forceinline__ float prob<float>(const float* p) {
  const float x = __ldg(p);
  return x > 0.f ? x : 0.f;
}
template <>
__device__ __forceinline__ float prob<__nv_bfloat16>(const __nv_bfloat16* p) {
  const float x = __bfloat162float(*p);
  return x > 0.f ? x : 0.f;
}

// a + b as s + e exactly
__device__ __forceinline__ void two_sum(float a, float b, float& s, float& e) {
  s = __fadd_rn(a, b);
  const float bb = __fadd_rn(s, -a);
  e = __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -bb)), __fadd_rn(b, -bb));
}

// rho = max(p - c q, 0) as a pair of floats
__device__ __forceinline__ void residual(float p, float q, float ch, float cl, float& hi, float& lo) {
  const float t = __fmul_rn(ch, q);
  const float te = __fmaf_rn(cl, q, __fmaf_rn(ch, q, -t));
  float s, e;
  two_sum(p, -t, s, e);
  e = __fadd_rn(e, -te);
  const bool pos = __fadd_rn(s, e) > 0.f;
  hi = pos ? s : 0.f;
  lo = pos ? e : 0.f;
}

struct Shared {
  double ctas[2][kCluster];     // totals of the cluster's blocks, by pass parity
  int ctas_last[2][kCluster];   // their last index with rho > 0
  double warps[kWarps];
  int warps_last[kWarps];
  float ch, cl;
  int cur, n_gone, act, look, token;
  double target;
};

// rho of one vocabulary entry under the present state (c = 0: p without the tokens taken out)
template <typename T>
struct Dist {
  const T* p;
  const T* q;
  float ch, cl;
  const int* gone;
  int n_gone;
  __device__ __forceinline__ void at(int i, float& hi, float& lo) const {
    hi = prob(p + i);
    lo = 0.f;
    if (q) residual(hi, prob(q + i), ch, cl, hi, lo);
    for (int g = 0; g < n_gone; ++g)
      if (gone[g] == i) hi = 0.f;
  }
};

template <typename T>
__global__ void __launch_bounds__(kThreads) __cluster_dims__(kCluster, 1, 1) verify_kernel(const VerifyArgs a) {
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
  for (int i = tid + 1; i < n; i += kThreads) {
    int parent = __ldg(a.parents + row + i);
    const int t = __ldg(a.tokens + row + i);
    if (parent < 0 || parent >= i || t < 0 || t >= a.V) {
      atomicCAS(a.err, 0, kErrDeviceIndex);
      parent = -1;
    } else {
      s_p[i] = prob(P + (size_t)parent * a.V + t);
      s_q[i] = Q ? prob(Q + (size_t)parent * a.V + t) : 1.f;
    }
    s_parent[i] = parent;
    s_token[i] = t;
    s_u[i] = __ldg(a.u + row + i);
  }
  __syncthreads();

  // the vocabulary's runs: warp w of block r takes run r kWarps + w
  const int run = (((a.V + kCluster * kWarps - 1) / (kCluster * kWarps)) + 31) & ~31;
  const long long lo_ll = (long long)(rank * kWarps + warp) * run;
  const int lo = (int)(lo_ll < a.V ? lo_ll : a.V), hi = lo + run < a.V ? lo + run : a.V;

  // thread 0's walk
  int cur = 0, i = 1, count = 0, n_gone = 0, pass = 0;
  double c = 0.0, Z = 1.0, c_new = 0.0, u_next = 0.0;
  bool summed = false, bare = false;   // the totals at hand are the present state's; rho given up for p
  if (tid == 0 && n > 0) {
    s_path[count++] = 0;
    u_next = (double)__ldg(a.u_next + b);
  }
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
      const Dist<T> dist{P + (size_t)sh.cur * a.V, (Q && sh.ch != 0.f) ? Q + (size_t)sh.cur * a.V : nullptr,
                         sh.ch, sh.cl, s_gone, sh.n_gone};
      float hs = 0.f, ls = 0.f;
      int last = -1;
#pragma unroll 8
      for (int j = lo + lane; j < hi; j += 32) {
        float h, l, e;
        dist.at(j, h, l);
        if (h > 0.f) last = j;
        two_sum(hs, h, hs, e);
        ls += l + e;
      }
      double sum = (double)hs + (double)ls;
#pragma unroll
      for (int m = 16; m >= 1; m >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, m);
        last = max(last, __shfl_xor_sync(0xffffffffu, last, m));
      }
      if (lane == 0) {
        sh.warps[warp] = sum;
        sh.warps_last[warp] = last;
      }
      __syncthreads();
      const int par = pass & 1;
      if (tid < kCluster) {   // thread r tells block r
        double total = 0.0;
        int block_last = -1;
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
          total += sh.warps[w];
          block_last = max(block_last, sh.warps_last[w]);
        }
        const uint32_t da = ptx::dsmem_addr(&sh.ctas[par][rank], tid), la = ptx::dsmem_addr(&sh.ctas_last[par][rank], tid);
        asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(da), "d"(total) : "memory");
        asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(la), "r"(block_last) : "memory");
      }
      ptx::cluster_sync_all();
      ++pass;
      if (tid == 0) {
        double total = 0.0;
#pragma unroll
        for (int r = 0; r < kCluster; ++r) total += sh.ctas[par][r];
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
    // the next token: the block, then the warp, then the entry where the running sum passes the target
    const int par = (pass - 1) & 1;
    if (tid == 0) {
      double total = 0.0, before = 0.0;
      int block = -1, all_last = -1;
#pragma unroll
      for (int r = 0; r < kCluster; ++r) {
        total += sh.ctas[par][r];
        all_last = max(all_last, sh.ctas_last[par][r]);
      }
      double target = u_next * total;
#pragma unroll
      for (int r = 0; r < kCluster; ++r) {
        if (block < 0 && before + sh.ctas[par][r] > target) {
          block = r;
          target -= before;
        }
        if (block < 0) before += sh.ctas[par][r];
      }
      int w_found = -1;
      if (block == rank) {
        before = 0.0;
        int w_last = -1;
        for (int w = 0; w < kWarps; ++w) {
          if (sh.warps[w] > 0.0) w_last = w;
          if (w_found < 0 && before + sh.warps[w] > target) {
            w_found = w;
            target -= before;
          }
          if (w_found < 0) before += sh.warps[w];
        }
        if (w_found < 0) {   // by rounding alone: the block's last run with anything in it
          w_found = w_last;
          target -= before;
        }
      }
      sh.target = target;
      sh.look = w_found;   // the warp of this block that looks, if any
      sh.token = (block < 0 && rank == 0) ? all_last : -2;   // nothing passes the target (u_next of 1, an empty row)
    }
    __syncthreads();
    const Dist<T> dist{P + (size_t)sh.cur * a.V, (Q && sh.ch != 0.f) ? Q + (size_t)sh.cur * a.V : nullptr,
                       sh.ch, sh.cl, s_gone, sh.n_gone};
    if (warp == sh.look) {
      // each lane adds a 32nd of the run, a scan over lanes finds the lane, a second one the entry
      double target = sh.target;
      const int piece = run / 32;
      const int p0 = min(lo + lane * piece, hi), p1 = min(p0 + piece, hi);
      float hs = 0.f, ls = 0.f;
#pragma unroll 8
      for (int j = p0; j < p1; ++j) {
        float h, l, e;
        dist.at(j, h, l);
        two_sum(hs, h, hs, e);
        ls += l + e;
      }
      const double mine = (double)hs + (double)ls;
      double incl = mine;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const double up = __shfl_up_sync(0xffffffffu, incl, m);
        if (lane >= m) incl += up;
      }
      const unsigned over = __ballot_sync(0xffffffffu, incl > target);
      int token = sh.warps_last[warp];   // where rounding leaves nothing above the target
      if (over) {
        const int who = __ffs(over) - 1;
        target -= __shfl_sync(0xffffffffu, incl - mine, who);
        const int q0 = __shfl_sync(0xffffffffu, p0, who), q1 = __shfl_sync(0xffffffffu, p1, who);
        bool found = false;
        for (int j0 = q0; j0 < q1 && !found; j0 += 32) {
          float h = 0.f, l = 0.f;
          if (j0 + lane < q1) dist.at(j0 + lane, h, l);
          const double x = (double)h + (double)l;
          double in2 = x;
#pragma unroll
          for (int m = 1; m < 32; m <<= 1) {
            const double up = __shfl_up_sync(0xffffffffu, in2, m);
            if (lane >= m) in2 += up;
          }
          const unsigned hit = __ballot_sync(0xffffffffu, in2 > target && x > 0.0);
          const unsigned any = __ballot_sync(0xffffffffu, x > 0.0);
          if (hit) {
            token = j0 + __ffs(hit) - 1;
            found = true;
          } else if (any) {
            token = j0 + 31 - __clz(any);
          }
          target -= __shfl_sync(0xffffffffu, in2, 31);
        }
      }
      if (lane == 0) a.next_token[b] = token;
    } else if (tid == 0 && sh.token != -2) {
      a.next_token[b] = sh.token;
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

}  // namespace

cudaError_t launch_verify_draft(const VerifyArgs& a, cudaStream_t s) {
  const size_t smem = (size_t)a.N * 7 * 4;
  const int slot = stage_timer_begin(s, kKernVerifyDraft);
  if (a.bf16) verify_kernel<__nv_bfloat16><<<a.B * kCluster, kThreads, smem, s>>>(a);
  else verify_kernel<float><<<a.B * kCluster, kThreads, smem, s>>>(a);
  const cudaError_t e = cudaGetLastError();
  stage_timer_end(slot, s);
  return e;
}

}  // namespace gdr
