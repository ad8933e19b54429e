// Attention of a tree (bit masks) or a chain of drafted nodes over a cache of pages; one node is the
// plain decode step. Per row b, query head h (key head hk = h / G, G = Hq / Hk) and node i:
//   o_i = sum_j p_j v_j,  p = softmax over visible j of scale q_i . k_j,  lse_i = log sum_j e^(scale q_i . k_j)
// with j over the row's ctx committed positions and the nodes that i sees.
//
// Shape: the G query heads of a key head and the nodes of a row form the M dimension (row r = node G +
// g), so a key/value tile is read once for all of them; 128 rows are one tensor-core tile. Up to about
// 280 rows a key head the products cost less than reading K and V (HBM at 6.8 TB/s against 1.9 PFLOP/s),
// and the padding of few rows to 128 is free; above that the tensor cores and the exponentials bound it.
//
// One persistent block per SM: one warp loads (TMA boxes of a page's positions into a ring of tile
// buffers), one thread issues the products (tcgen05: S = Q K^T into one of two TMEM buffers, O += P V
// with P read from TMEM), eight warps do the softmax: warps w and w + 4 share 32 rows, each half of
// the tile's columns. S of tile t + 1 is formed while the softmax works on tile t, and P V of tile t
// while it works on tile t + 1.
//
// Work split: all (row, key head, M tile) items laid end to end are (sum of their key tiles) units; block
// c of C takes units [c U / C, (c + 1) U / C), so every SM reads the same number of tiles whatever the
// rows' lengths. An item cut across blocks leaves its parts (O / l and lse in float32) in the workspace
// and a second kernel joins them in order.
//
// The running maximum is kept as a reference that moves only when the maximum has grown by more than 8
// (in log2): P <= 2^8 then, the sums stay in range, and O in TMEM is rescaled only at those rare tiles.
// P is rounded to bf16 for the product with V (one rounding of 2^-9 relative per term, independent
// between terms); the sum l adds the unrounded P in float32.
//
// Masked places: K of an unseen position only enters a score that is replaced by -inf. V is different
// (0 times inf is nan), so tiles that reach past ctx have V cleaned in shared memory first: positions
// past the row's nodes become 0, and nodes' elements that are not finite become 0 and are added back, at
// the end, to the rows that see them.
#include <algorithm>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include "gdr_serve.h"
#include "ptx.cuh"

namespace gdr {

using namespace ptx;

namespace {

constexpr int kThreads = 384;   // warps: 0 loads, 1 products, 2-3 idle, 4-11 softmax
constexpr int kBlocks = kNumSMs;
constexpr int kM = 128;         // rows of an M tile
constexpr float kLog2e = 1.4426950408889634f;
constexpr long long kDrainBudget = 2000000000ll;   // cycles an aborting block waits for its own work

struct Args {
  const int32_t* table;
  const int32_t* ctx;
  const int32_t* lengths;
  const uint64_t* mask;
  const __nv_bfloat16* v_pages;
  float sl2;                 // scale log2(e)
  __nv_bfloat16* o;
  float* lse;
  float* part_o;             // [2 C][128][D]
  float* part_lse;           // [2 C][128]
  int B, N, Hq, Hk, G, npt, W, P, page, M;
  long long budget;
  int* err;
};

template <int D>
struct Cfg {
  static constexpr int KT = D == 256 ? 64 : 128;             // positions of a tile
  static constexpr uint32_t kTile = KT * D * 2;              // bytes of a K or V tile
  static constexpr int NS = D == 64 ? 8 : D == 128 ? 6 : 5;  // tile buffers
  static constexpr uint32_t kQ = kM * D * 2;
  static constexpr uint32_t kRing = kQ;
  static constexpr uint32_t kRed = kRing + NS * kTile;       // float [2][2][128]
  static constexpr uint32_t kBars = kRed + 2048;
  static constexpr uint32_t kSmem = kBars + 512;
  static constexpr uint32_t kTmemO = 2 * KT;                 // S buffers at columns 0 and KT
};

struct Bars {
  uint64_t full[8], empty[8];
  uint64_t q_full, q_empty;
  uint64_t s_full[2], p_full[2], pv[2];
  uint64_t clean;      // V of a masked tile has been cleaned (eight warps)
  uint64_t drain;
  uint32_t tmem;
  int bad[3];          // a cleaned node element was not finite, by segment modulo three
  // the block's first unit, found by the thread whose rows hold it
  int b0, hk0, mt0, t0;
  long long todo;
};
static_assert(sizeof(Bars) <= 512, "barriers fit their region");

// A row's nodes and context; an invalid row counts as no nodes.
__device__ __forceinline__ bool row_of(const Args& a, int b, int& n, int& ctx) {
  n = a.lengths ? __ldg(a.lengths + b) : a.N;
  ctx = __ldg(a.ctx + b);
  if (n < 0 || n > a.N || ctx < 0 || (long long)ctx + n > (long long)a.M * a.page) {
    n = 0;
    return false;
  }
  return true;
}
// Key tiles of M tile mt: a chain's M tile needs no position past its last node.
template <int KT>
__device__ __forceinline__ int tiles_of(const Args& a, int n, int ctx, int mt) {
  const int nodes = a.mask ? n : min(n, (mt + 1) * a.npt);
  return (ctx + nodes + KT - 1) / KT;
}
// Units of one key head of a row.
template <int KT>
__device__ __forceinline__ long long units_of(const Args& a, int n, int ctx) {
  if (n == 0) return 0;
  const int mts = (n + a.npt - 1) / a.npt;
  if (a.mask) return (long long)mts * tiles_of<KT>(a, n, ctx, 0);
  long long u = 0;
  for (int mt = 0; mt < mts; ++mt) u += tiles_of<KT>(a, n, ctx, mt);
  return u;
}
__device__ __forceinline__ long long first_unit(long long total, int c) { return total * c / kBlocks; }
// The block whose share holds unit x.
__device__ __forceinline__ int block_of(long long total, long long x) {
  int c = (int)min((long long)kBlocks - 1, x * kBlocks / total);
  while (first_unit(total, c + 1) <= x) ++c;
  while (first_unit(total, c) > x) --c;
  return c;
}

// Walks the block's segments: a run of key tiles [t0, t1) of one item.
template <int KT>
struct Walk {
  int b, hk, mt, t0, t1, tiles, n, ctx, index;
  long long todo;
  __device__ __forceinline__ void start(const Args& a, const Bars& s) {
    b = s.b0; hk = s.hk0; mt = s.mt0; t1 = s.t0;
    todo = s.todo;
    index = -1;
    if (todo > 0) {
      row_of(a, b, n, ctx);
      tiles = tiles_of<KT>(a, n, ctx, mt);
    }
  }
  __device__ __forceinline__ bool next(const Args& a) {
    if (todo <= 0) return false;
    if (index >= 0) {   // the last segment ended its item
      t1 = 0;
      if (++mt * a.npt >= n) {
        mt = 0;
        if (++hk == a.Hk) {
          hk = 0;
          do {
            ++b;
            row_of(a, b, n, ctx);
          } while (n == 0);   // units are left, so a row with nodes is
        }
      }
      tiles = tiles_of<KT>(a, n, ctx, mt);
    }
    t0 = t1;
    t1 = (int)min((long long)tiles, t0 + todo);
    todo -= t1 - t0;
    ++index;
    return true;
  }
};

// mbar_wait by a whole warp, with one answer for all its lanes.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, long long budget) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, budget));
}

// Sum over the block's threads (all of them call), and this thread's sum of those before it.
__device__ __forceinline__ long long block_sum(long long v, long long* warps, long long& before) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
  long long incl = v;
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const long long up = __shfl_up_sync(0xffffffffu, incl, m);
    if (lane >= m) incl += up;
  }
  if (lane == 31) warps[warp] = incl;
  __syncthreads();
  long long total = 0;
  before = incl - v;
  for (int w = 0; w < nw; ++w) {
    if (w < warp) before += warps[w];
    total += warps[w];
  }
  return total;
}

// Bits k = 0 .. 63: position pos0 + k is seen by node i (rel = pos0 - ctx).
__device__ __forceinline__ uint64_t seen(const Args& a, const uint64_t* words, int i, int n, long long rel) {
  if (rel + 64 <= 0) return ~0ull;
  uint64_t ctx_bits = 0, bits;
  int sh;         // bit k is node k - sh
  long long j0;   // first node of `bits`
  if (rel < 0) {
    sh = (int)-rel;
    ctx_bits = (1ull << sh) - 1;
    j0 = 0;
  } else {
    sh = 0;
    j0 = rel;
  }
  if (a.mask) {
    const long long w = j0 >> 6;
    const int o = (int)(j0 & 63);
    const uint64_t lo = w < a.W ? __ldg(words + w) : 0, hi = (o && w + 1 < a.W) ? __ldg(words + w + 1) : 0;
    bits = (lo >> o) | (o ? hi << (64 - o) : 0);
  } else {
    const long long k = i - j0 + 1;   // nodes j0 .. i
    bits = k <= 0 ? 0 : k >= 64 ? ~0ull : (1ull << k) - 1;
  }
  const long long left = n - j0;      // nodes that are there
  if (left <= 0) bits = 0;
  else if (left < 64) bits &= (1ull << left) - 1;
  return ctx_bits | (bits << sh);
}

// Adds the elements of seen nodes' V that are not finite (cleaned away before the product) to what the
// row's thread has just written to out[0 .. cols).
template <typename T>
__device__ __noinline__ void add_back(const Args& a, int b, int hk, int i, int n, int ctx, int lo, int hi, int D, int d0,
                                      int cols, T* out) {
  const uint64_t* words = a.mask ? a.mask + ((size_t)b * a.N + i) * a.W : nullptr;
  for (int pos = max(lo, ctx); pos < min(hi, ctx + n); ++pos) {
    const int j = pos - ctx;
    if (words ? !(words[j >> 6] >> (j & 63) & 1) : j > i) continue;
    const int pg = a.table[(size_t)b * a.M + pos / a.page];
    if (pg < 0 || pg >= a.P) continue;
    const __nv_bfloat16* v = a.v_pages + (((size_t)pg * a.page + pos % a.page) * a.Hk + hk) * D + d0;
    for (int d = 0; d < cols; ++d) {
      const float x = __bfloat162float(v[d]);
      if (!(fabsf(x) < INFINITY)) out[d] = (T)((float)out[d] + x);
    }
  }
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const Args a) {
  using C = Cfg<D>;
  constexpr int KT = C::KT, NS = C::NS, kCols = KT / 2;
  extern __shared__ __align__(1024) uint8_t sm[];
  Bars& s = *reinterpret_cast<Bars*>(sm + C::kBars);
  float* red = reinterpret_cast<float*>(sm + C::kRed);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (smem_u32(sm) & 1023u) {   // the swizzled tiles rely on it
    if (tid == 0) atomicCAS(a.err, 0, kErrTimeout);
    return;
  }

  // the block's share of the units
  {
    const int per = (a.B + kThreads - 1) / kThreads, r0 = min(a.B, tid * per), r1 = min(a.B, r0 + per);
    long long mine = 0;
    for (int b = r0; b < r1; ++b) {
      int n, ctx;
      if (!row_of(a, b, n, ctx) && blockIdx.x == 0) atomicCAS(a.err, 0, kErrDeviceIndex);
      mine += units_of<KT>(a, n, ctx) * a.Hk;
    }
    long long before;
    const long long total = block_sum(mine, reinterpret_cast<long long*>(red), before);
    const long long x0 = first_unit(total, blockIdx.x), x1 = first_unit(total, blockIdx.x + 1);
    if (tid == 0) s.todo = x1 - x0;
    if (x1 > x0 && x0 >= before && x0 < before + mine) {
      long long at = x0 - before;
      for (int b = r0; b < r1; ++b) {
        int n, ctx;
        row_of(a, b, n, ctx);
        const long long head = units_of<KT>(a, n, ctx);
        if (at >= head * a.Hk) {
          at -= head * a.Hk;
          continue;
        }
        s.b0 = b;
        s.hk0 = (int)(at / head);
        at -= s.hk0 * head;
        int mt = 0;
        while (at >= tiles_of<KT>(a, n, ctx, mt)) at -= tiles_of<KT>(a, n, ctx, mt++);
        s.mt0 = mt;
        s.t0 = (int)at;
        break;
      }
    }
  }
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    mbar_init(&s.q_full, 1);
    mbar_init(&s.q_empty, 1);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], 8);
      mbar_init(&s.pv[i], 1);
    }
    mbar_init(&s.clean, 8);
    mbar_init(&s.drain, 1);
    for (int i = 0; i < 3; ++i) s.bad[i] = 0;
    fence_mbar_init();
    prefetch_tmap(&mq);
    prefetch_tmap(&mk);
    prefetch_tmap(&mv);
  }
  if (warp == 1) tmem_alloc(&s.tmem, 512);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = s.tmem;
  launch_dependents();

  bool ok = true;
  if (warp == 0) {
    // ------------------------------------------------------------------------------ loads
    Walk<KT> w;
    w.start(a, s);
    const int rows = min(a.page, KT);                       // positions of one box
    const uint32_t box = rows * 128u;                       // its bytes in one 64-column slab
    long long it = 0;                                       // tiles loaded
    int q_loads = 0;
    while (ok && w.next(a)) {
      if (w.index > 0) ok = warp_wait(&s.q_empty, (w.index - 1) & 1, a.budget);
      if (!ok) break;
      if (lane == 0) {
        mbar_arrive_expect_tx(&s.q_full, (uint32_t)(D / 64) * a.G * a.npt * 128u);
        for (int h = 0; h < D / 64; ++h)
          tma_load_4d(sm + h * kM * 128, &mq, &s.q_full, h * 64, w.hk * a.G, w.mt * a.npt, w.b);
      }
      ++q_loads;
      const int end = w.ctx + w.n;
      const int32_t* table = a.table + (size_t)w.b * a.M;
      for (int t = w.t0; ok && t < w.t1; ++t) {
        const int base = t * KT;
        const int pieces = min(KT / rows, (end - base + rows - 1) / rows);
        int pg = -1, at = 0;
        if (lane < pieces) {
          const int pos = base + lane * rows;
          pg = __ldg(table + pos / a.page);
          at = pos % a.page;
          if (pg < 0 || pg >= a.P) {   // read as zeros (a coordinate outside the tensor) and reported
            atomicCAS(a.err, 0, kErrDeviceIndex);
            pg = -1;
          }
        }
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const int slot = (int)(it % NS);
          if (it >= NS) ok = warp_wait(&s.empty[slot], (uint32_t)(it / NS - 1) & 1, a.budget);
          if (!ok) break;
          if (lane == 0) mbar_arrive_expect_tx(&s.full[slot], pieces * box * (D / 64));
          __syncwarp();
          if (lane < pieces) {
            uint8_t* dst = sm + C::kRing + slot * C::kTile + lane * box;
            for (int h = 0; h < D / 64; ++h)
              tma_load_4d(dst + h * KT * 128, kv ? &mv : &mk, &s.full[slot], h * 64, w.hk, at, pg);
          }
        }
      }
    }
    // no copy of this block is left in flight
    for (long long i = it > NS ? it - NS : 0; i < it; ++i)
      warp_wait(&s.full[i % NS], (uint32_t)(i / NS) & 1, kDrainBudget);
    if (q_loads > 0) warp_wait(&s.q_full, (q_loads - 1) & 1, kDrainBudget);
  } else if (warp == 1) {
    // ------------------------------------------------------------------------------ products
    if (lane == 0) {
      Walk<KT> w;
      w.start(a, s);
      constexpr uint32_t kIdS = idesc_bf16(kM, KT, false, false), kIdO = idesc_bf16(kM, D, false, true);
      const uint32_t qb = smem_u32(sm), ring = smem_u32(sm + C::kRing);
      long long g = 0;   // tiles begun, over all segments
      while (ok && w.next(a)) {
        ok = mbar_wait(&s.q_full, w.index & 1, a.budget);
        const int T = w.t1 - w.t0;
        // S of tile x: its buffer is free once P V of tile x - 2 is done
        auto scores = [&](long long x, bool last) {
          if (x >= 2) ok = ok && mbar_wait(&s.pv[x & 1], (uint32_t)((x - 2) >> 1) & 1, a.budget);
          const int slot = (int)((2 * x) % NS);
          ok = ok && mbar_wait(&s.full[slot], (uint32_t)((2 * x) / NS) & 1, a.budget);
          if (!ok) return;
          tc_fence_after();
          const uint32_t kb = ring + slot * C::kTile;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16(tb + (uint32_t)(x & 1) * KT, smem_desc(qb + (kk >> 2) * kM * 128 + (kk & 3) * 32, 16, 1024),
                     smem_desc(kb + (kk >> 2) * KT * 128 + (kk & 3) * 32, 16, 1024), kIdS, kk > 0);
          mma_commit(&s.s_full[x & 1]);
          mma_commit(&s.empty[slot]);
          if (last) mma_commit(&s.q_empty);
        };
        if (ok) scores(g, T == 1);
        for (int j = 0; ok && j < T; ++j, ++g) {
          if (j + 1 < T) scores(g + 1, j + 2 == T);
          ok = ok && mbar_wait(&s.p_full[g & 1], (uint32_t)(g >> 1) & 1, a.budget);
          const int slot = (int)((2 * g + 1) % NS);
          ok = ok && mbar_wait(&s.full[slot], (uint32_t)((2 * g + 1) / NS) & 1, a.budget);
          if (!ok) break;
          tc_fence_after();
          const uint32_t vb = ring + slot * C::kTile, pb = tb + (uint32_t)(g & 1) * KT;
#pragma unroll
          for (int kk = 0; kk < KT / 16; ++kk)
            mma_f16_tmem_a(tb + C::kTmemO, pb + kk * 8, smem_desc(vb + kk * 2048, KT * 128, 1024), kIdO, j > 0 || kk > 0);
          mma_commit(&s.pv[g & 1]);
          mma_commit(&s.empty[slot]);
        }
      }
      // no product of this block is left in flight
      mma_commit(&s.drain);
      mbar_wait(&s.drain, 0, kDrainBudget);
    }
  } else if (warp >= 4) {
    // ------------------------------------------------------------------------------ softmax
    Walk<KT> w;
    w.start(a, s);
    const int half = (warp - 4) >> 2, quarter = warp & 3, row = 32 * quarter + lane;
    const uint32_t lane_base = (uint32_t)(32 * quarter) << 16;
    const uint32_t pair_bar = 1 + quarter;
    const int wtid = tid - 128;
    long long g = 0;
    uint32_t cleaned = 0;   // masked tiles so far
    while (ok && w.next(a)) {
      if (wtid == 0) s.bad[(w.index + 1) % 3] = 0;   // read two segments ago, set in the next
      const int used = min(a.npt, w.n - w.mt * a.npt) * a.G;
      const bool active = 32 * quarter < used, live = row < used;
      const int i = w.mt * a.npt + (live ? row / a.G : 0), hg = live ? row % a.G : 0;
      const uint64_t* words = a.mask ? a.mask + ((size_t)w.b * a.N + i) * a.W : nullptr;
      const int end = w.ctx + w.n;
      float m_ref = -INFINITY, l = 0.f;
      bool masked_any = false;
      for (int t = w.t0; t < w.t1; ++t, ++g) {
        const bool masked = (t + 1) * KT > w.ctx;
        if (masked) {
          // clean V of positions past ctx
          masked_any = true;
          const long long vi = 2 * g + 1;
          const int slot = (int)(vi % NS);
          ok = ok && warp_wait(&s.full[slot], (uint32_t)(vi / NS) & 1, a.budget);
          if (ok) {
            uint8_t* vt = sm + C::kRing + slot * C::kTile;
            const int r0 = max(0, w.ctx - t * KT);
            bool bad = false;
            for (int x = wtid; x < (KT - r0) * (D / 8); x += 256) {
              const int r = r0 + x / (D / 8), ch = x % (D / 8);
              uint4* p = reinterpret_cast<uint4*>(vt + (ch >> 3) * KT * 128 + r * 128 + (ch & 7) * 16);
              if (t * KT + r >= end) {
                *p = make_uint4(0, 0, 0, 0);
              } else {
                uint4 v = *p;
                uint32_t* u = reinterpret_cast<uint32_t*>(&v);
                bool hit = false;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                  if ((u[e] & 0x7F80u) == 0x7F80u) {
                    u[e] &= 0xFFFF0000u;
                    hit = true;
                  }
                  if ((u[e] & 0x7F800000u) == 0x7F800000u) {
                    u[e] &= 0xFFFFu;
                    hit = true;
                  }
                }
                if (hit) {
                  *p = v;
                  bad = true;
                }
              }
            }
            if (bad) s.bad[w.index % 3] = 1;
            fence_async_smem();
          }
          __syncwarp();
          if (lane == 0) mbar_arrive(&s.clean);
          ++cleaned;
        }
        ok = ok && warp_wait(&s.s_full[g & 1], (uint32_t)(g >> 1) & 1, a.budget);
        const uint32_t sb = tb + lane_base + (uint32_t)(g & 1) * KT;
        if (active) {
          float x[kCols];
          if (ok) {
            tc_fence_after();
            if constexpr (kCols == 64) tmem_ld64(sb + half * kCols, x);
            else tmem_ld32(sb + half * kCols, x);
          }
          if (masked && live) {
            const uint64_t vis = seen(a, words, i, w.n, (long long)t * KT + half * kCols - w.ctx);
#pragma unroll
            for (int c = 0; c < kCols; ++c)
              if (!(vis >> c & 1)) x[c] = -INFINITY;
          }
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < kCols; ++c) mx = fmaxf(mx, x[c]);
          float* mine = red + (g & 1) * 256;
          mine[half * 128 + row] = mx;
          tc_fence_before();   // (P goes over scores that the other half has read)
          ok = named_bar_and(pair_bar, 64, ok);   // both halves leave together
          if (!ok) break;
          tc_fence_after();
          mx = fmaxf(mx, mine[(half ^ 1) * 128 + row]);
          // (rows past the tile's nodes hold arbitrary scores and never ask for a new reference)
          const bool need = live && mx > m_ref && (m_ref == -INFINITY || (mx - m_ref) * a.sl2 > 8.f);
          if (__any_sync(0xffffffffu, need)) {
            const float m_new = live ? fmaxf(m_ref, mx) : m_ref;
            if (t > w.t0) {
              const float f = m_ref == m_new ? 1.f : ex2_approx((m_ref - m_new) * a.sl2);
              l *= f;
              ok = warp_wait(&s.pv[(g - 1) & 1], (uint32_t)((g - 1) >> 1) & 1, a.budget);
              if (ok) {
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < D / 2; c += 32) {
                  float o[32];
                  uint32_t u[32];
                  const uint32_t at = tb + lane_base + C::kTmemO + half * (D / 2) + c;
                  tmem_ld32(at, o);
#pragma unroll
                  for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * f);
                  tmem_st32(at, u);
                }
              }
            }
            m_ref = m_new;
          }
          const float off = m_ref == -INFINITY ? 0.f : -m_ref * a.sl2;
          uint32_t p[kCols / 2];
          float sum = 0.f;
#pragma unroll
          for (int c = 0; c < kCols; c += 2) {
            const float e0 = ex2_approx(fmaf(x[c], a.sl2, off)), e1 = ex2_approx(fmaf(x[c + 1], a.sl2, off));
            sum += e0 + e1;
            p[c / 2] = pack_bf16x2(e0, e1);
          }
          l += sum;
          if (ok) {
            if constexpr (kCols == 64) {
              tmem_st32(sb + half * 32, p);
            } else {
              tmem_st16_nowait(sb + half * 16, p);
              tmem_wait_st();
            }
          }
        }
        if (!active && !ok) break;
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&s.p_full[g & 1]);
      }
      if (!ok && !active) break;
      // the segment's result
      const long long last = g - 1;
      ok = ok && warp_wait(&s.pv[last & 1], (uint32_t)(last >> 1) & 1, a.budget);
      if (masked_any) ok = ok && warp_wait(&s.clean, (cleaned - 1) & 1, a.budget);
      if (!active) continue;
      float* mine = red + (g & 1) * 256;
      mine[half * 128 + row] = l;
      ok = named_bar_and(pair_bar, 64, ok);
      if (!ok) break;
      l += mine[(half ^ 1) * 128 + row];
      tc_fence_after();
      const float inv = l > 0.f || l != l ? 1.f / l : 0.f;
      const float lse = l > 0.f || l != l ? m_ref * a.sl2 * (1.f / kLog2e) + logf(l) : -INFINITY;
      const bool whole = w.t0 == 0 && w.t1 == w.tiles;
      const bool bad = masked_any && s.bad[w.index % 3];
      const size_t orow = ((size_t)w.b * a.N + i) * a.Hq + w.hk * a.G + hg;
      const size_t prow = (size_t)(2 * blockIdx.x + (w.index > 0)) * kM + row;
#pragma unroll
      for (int c = 0; c < D / 2; c += 32) {
        float o[32];
        const int d0 = half * (D / 2) + c;
        tmem_ld32(tb + lane_base + C::kTmemO + d0, o);
        if (!live) continue;
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] *= inv;
        if (whole) {
          uint4* out = reinterpret_cast<uint4*>(a.o + orow * D + d0);
#pragma unroll
          for (int e = 0; e < 4; ++e)
            out[e] = make_uint4(pack_bf16x2(o[8 * e], o[8 * e + 1]), pack_bf16x2(o[8 * e + 2], o[8 * e + 3]),
                                pack_bf16x2(o[8 * e + 4], o[8 * e + 5]), pack_bf16x2(o[8 * e + 6], o[8 * e + 7]));
        } else {
          float4* out = reinterpret_cast<float4*>(a.part_o + prow * D + d0);
#pragma unroll
          for (int e = 0; e < 8; ++e) out[e] = make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]);
        }
      }
      if (bad && live) {
        const int d0 = half * (D / 2);
        if (whole) add_back(a, w.b, w.hk, i, w.n, w.ctx, w.t0 * KT, w.t1 * KT, D, d0, D / 2, a.o + orow * D + d0);
        else add_back(a, w.b, w.hk, i, w.n, w.ctx, w.t0 * KT, w.t1 * KT, D, d0, D / 2, a.part_o + prow * D + d0);
      }
      if (half == 0 && live) {
        if (!whole) a.part_lse[prow] = lse;
        else if (a.lse) a.lse[orow] = lse;
      }
      tc_fence_before();
    }
  }
  if (!ok && lane == 0) atomicCAS(a.err, 0, kErrTimeout);
  __syncwarp();
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    tc_fence_after();
    tmem_dealloc(tb, 512);
  }
}

// Joins the parts of items that several blocks shared, and fills the rows of absent nodes (0, -inf):
// o = sum_s e^(lse_s - lse) o_s over a row's parts. Few items have many parts each (one item is cut over
// up to every block) and few rows: kRowWarps = 8 warps then share a (node, query head) row, warp w
// taking parts w, w + 8, ... and the block adding the warps' sums in order; with many items a row has
// one to three parts and one warp takes it. Parts are read four at a time: the loop is bound by their
// latency, 33 -> 8 us for 38 parts of 224 rows of 256.
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
template <int D, int kRowWarps>
__global__ void __launch_bounds__(kJoinThreads) tree_attn_join_kernel(const Args a) {
  constexpr int KT = Cfg<D>::KT, kVec = D / 32;
  __shared__ long long sums[2][kJoinWarps];
  __shared__ float s_acc[kRowWarps > 1 ? kRowWarps : 1][D];
  __shared__ float s_sum[kJoinWarps];
  const int b = blockIdx.y, tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  long long mine = 0, before_b = 0;   // units of all rows, and of rows before b
  for (int r = tid; r < a.B; r += kJoinThreads) {
    int n, ctx;
    row_of(a, r, n, ctx);
    const long long u = units_of<KT>(a, n, ctx) * a.Hk;
    mine += u;
    if (r < b) before_b += u;
  }
  long long dummy;
  const long long total = block_sum(mine, sums[0], dummy);
  before_b = block_sum(before_b, sums[1], dummy);
  wait_prerequisite();
  const int r = kRowWarps > 1 ? blockIdx.x : blockIdx.x * kJoinWarps + warp;   // node Hq + head
  if (r >= a.N * a.Hq) return;
  const int part0 = kRowWarps > 1 ? warp : 0;
  const int i = r / a.Hq, h = r % a.Hq;
  int n, ctx;
  row_of(a, b, n, ctx);
  const size_t orow = (size_t)b * a.N * a.Hq + r;
  float acc[kVec];
#pragma unroll
  for (int e = 0; e < kVec; ++e) acc[e] = 0.f;
  float lse = -INFINITY;
  if (i < n) {
    const int hk = h / a.G, mt = i / a.npt, row = (i - mt * a.npt) * a.G + h % a.G;
    long long x0 = before_b + hk * units_of<KT>(a, n, ctx);
    for (int t = 0; t < mt; ++t) x0 += tiles_of<KT>(a, n, ctx, t);
    const long long x1 = x0 + tiles_of<KT>(a, n, ctx, mt);
    const int c0 = block_of(total, x0), c1 = block_of(total, x1 - 1);
    if (c0 == c1) return;   // written whole (the same in every warp of the row)
    // (blocks between c0 and c1 all hold a unit: the item's units are consecutive, and a block without
    // units holds none of them, which first_unit(c) == first_unit(c + 1) says)
    auto share = [&](int c) { return first_unit(total, c) < first_unit(total, c + 1); };
    // a block's first segment is its part 0: block c0's only where the item starts its share
    auto part = [&](int c) { return (size_t)(2 * c + (first_unit(total, c) < x0)) * kM + row; };
    float top = -INFINITY;
    bool nan = false;
    for (int c = c0 + lane; c <= c1; c += 32) {
      const float x = share(c) ? a.part_lse[part(c)] : -INFINITY;
      nan |= x != x;
      top = fmaxf(top, x);
    }
#pragma unroll
    for (int m = 16; m >= 1; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    nan = __any_sync(0xffffffffu, nan);
    const float ref = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    for (int cc = c0 + part0; cc <= c1; cc += 4 * kRowWarps) {
      float w[4], x[4][kVec];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = cc + u * kRowWarps;
        const bool there = c <= c1 && share(c);
        const size_t p = there ? part(c) : part(c0);
        w[u] = there ? a.part_lse[p] : -INFINITY;
        const float* po = a.part_o + p * D + lane * kVec;
#pragma unroll
        for (int e = 0; e < kVec; e += 2) {
          const float2 y = *reinterpret_cast<const float2*>(po + e);
          x[u][e] = y.x;
          x[u][e + 1] = y.y;
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = ex2_approx((w[u] - ref) * kLog2e);
        sum += f;
        if (f != 0.f) {   // a part that saw nothing may hold anything
#pragma unroll
          for (int e = 0; e < kVec; ++e) acc[e] = fmaf(f, x[u][e], acc[e]);
        }
      }
    }
    if constexpr (kRowWarps > 1) {
#pragma unroll
      for (int e = 0; e < kVec; ++e) s_acc[warp][lane * kVec + e] = acc[e];
      if (lane == 0) s_sum[warp] = sum;
      __syncthreads();   // (every warp of the block is here: they share the row)
      if (warp > 0) return;
      sum = 0.f;
#pragma unroll
      for (int e = 0; e < kVec; ++e) acc[e] = 0.f;
#pragma unroll
      for (int w = 0; w < kRowWarps; ++w) {
        sum += s_sum[w];
#pragma unroll
        for (int e = 0; e < kVec; ++e) acc[e] += s_acc[w][lane * kVec + e];
      }
    }
    const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
#pragma unroll
    for (int e = 0; e < kVec; ++e) acc[e] *= inv;
    lse = nan ? NAN : sum > 0.f ? ref + logf(sum) : -INFINITY;
  } else if (kRowWarps > 1 && warp > 0) {
    return;
  }
  __nv_bfloat16* out = a.o + orow * D + lane * kVec;
#pragma unroll
  for (int e = 0; e < kVec; e += 2) *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(acc[e], acc[e + 1]);
  if (lane == 0 && a.lse) a.lse[orow] = lse;
}

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      p = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  }();
  return fn;
}

// [d3, d2, d1, D] bf16, box of 64 columns (128-byte swizzle) x b1 x b2 x 1
bool make_map(CUtensorMap* m, const void* base, int D, int d1, int d2, int d3, int b1, int b2) {
  auto enc = encode_fn();
  if (!enc) return false;
  const cuuint64_t row = (cuuint64_t)D * 2;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)d1, (cuuint64_t)d2, (cuuint64_t)d3};
  const cuuint64_t strides[3] = {row, row * d1, row * d1 * d2};
  const cuuint32_t box[4] = {64, (cuuint32_t)b1, (cuuint32_t)b2, 1};
  const cuuint32_t es[4] = {1, 1, 1, 1};
  return enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, es,
             CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
             CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
cudaError_t launch(const TreeAttnArgs& p, cudaStream_t st) {
  using C = Cfg<D>;
  Args a{};
  a.G = p.Hq / p.Hk;
  a.npt = kM / a.G;
  if (a.npt > p.N) a.npt = p.N;
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, p.q, D, p.Hq, p.N, p.B, a.G, a.npt) ||
      !make_map(&mk, p.k_pages, D, p.Hk, p.page, p.P, 1, std::min(p.page, C::KT)) ||
      !make_map(&mv, p.v_pages, D, p.Hk, p.page, p.P, 1, std::min(p.page, C::KT)))
    return cudaErrorInvalidValue;
  a.table = p.table; a.ctx = p.ctx; a.lengths = p.lengths; a.mask = p.mask;
  a.v_pages = static_cast<const __nv_bfloat16*>(p.v_pages);
  a.sl2 = p.scale * kLog2e;
  a.o = static_cast<__nv_bfloat16*>(p.o);
  a.lse = p.lse;
  a.part_o = reinterpret_cast<float*>(p.ws);
  a.part_lse = a.part_o + (size_t)2 * kBlocks * kM * D;
  a.B = p.B; a.N = p.N; a.Hq = p.Hq; a.Hk = p.Hk; a.W = (p.N + 63) / 64; a.P = p.P; a.page = p.page; a.M = p.M;
  a.budget = wait_budget_cycles();
  a.err = p.err;
  cudaError_t e = cudaFuncSetAttribute(tree_attn_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  if (e != cudaSuccess) return e;
  int slot = stage_timer_begin(st, kKernTreeAttn);
  tree_attn_kernel<D><<<kBlocks, kThreads, C::kSmem, st>>>(mq, mk, mv, a);
  stage_timer_end(slot, st);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  // (64 items: three parts or fewer each)
  const bool few = (long long)p.B * p.Hk * ((p.N + a.npt - 1) / a.npt) <= 64;
  cfg.gridDim = dim3(few ? p.N * p.Hq : (p.N * p.Hq + kJoinWarps - 1) / kJoinWarps, p.B);
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  slot = stage_timer_begin(st, kKernTreeAttnJoin);
  e = few ? cudaLaunchKernelEx(&cfg, tree_attn_join_kernel<D, 8>, a) : cudaLaunchKernelEx(&cfg, tree_attn_join_kernel<D, 1>, a);
  stage_timer_end(slot, st);
  return e;
}

}  // namespace

size_t tree_attn_workspace_bytes(int D) { return (size_t)2 * kBlocks * kM * (D + 1) * sizeof(float); }

cudaError_t launch_tree_attn(const TreeAttnArgs& a, cudaStream_t s) {
  return a.D == 64 ? launch<64>(a, s) : a.D == 128 ? launch<128>(a, s) : launch<256>(a, s);
}

}  // namespace gdr
