// The tcgen05 attention frame: attention of a tree (bit masks) or a chain of drafted nodes over a cache of pages; one node is the
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
// buffers), one issues the products (tcgen05: S = Q K^T into TMEM, O += P V with P read from TMEM), two
// warpgroups do the softmax. Three forms share this frame:
//   kWide   D <= 128 and more than 128 rows a key head: two M tiles an item, one a warpgroup; both read the
//           same key/value tiles, the products of one run under the softmax of the other. (Tiles of 64
//           positions with two S buffers a stream, so that S is always there in time, were slower, 119
//           us against 98 then for 8 trees of 64 nodes over 16384 positions: products of N = 64 are bound by
//           reading Q from shared memory, and every product costs two waits.)
//   kNarrow D <= 128, up to 128 rows: one M tile, the warpgroups take every other key tile, each with
//           its own accumulator, maximum and sum, joined at the end of the segment.
//   kSplit  D = 256: an accumulator takes half of TMEM, so there is one: the warpgroups take half of each
//           tile's columns, S alternates between two buffers. The queries lie in TMEM's other quarter, and keys and
//           values are loaded by a warp each (512 rows a key head over 65536 positions in pages of 16: 106.5 us before,
//           90.4 with two loading warps, 87.6 with the queries in TMEM, 80.1 with seven tile buffers in their place).
// A warp of kWide and kNarrow holds whole rows of S (a row a thread): no exchange inside a tile.
// The products are issued by an elected lane of a converged warp, straight-line, from descriptors that
// are one word plus a constant: 64 cycles a 128 x 128 x 16 product, against about 100 from a branch on
// the lane index.
//
// Work split: all (row, key head, M tile or pair of them) items laid end to end are (sum of their key
// tiles) units; block c of C takes units [c U / C, (c + 1) U / C), so every SM reads the same number of
// tiles whatever the rows' lengths, but for an item's start and end (queries loaded, the softmax drained,
// results written), which count as kPad tiles. An item cut across blocks leaves its parts (O / l and lse in
// float32) in the workspace and a second kernel joins them in order.
//
// Measured (bfloat16, a call among others): one token over 700 positions 12.3 us (latency); 16 trees of 13
// nodes over up to 8192 positions, 32 / 8 heads of 128: 72.4 us, 73% of the copy bandwidth (95% while it
// streams); 8 trees of 64 nodes over up to 16384, 32 / 4 heads of 128: 93.9 us, 47% of the matrix rate; 2
// trees of 7 over 131072, 16 / 2 heads of 256: 78.5 us, 77% of the copy bandwidth. (Comparisons below that
// give slightly other times for these are of replayed graphs.)
//
// The running maximum is kept as a reference that moves only when the maximum has grown by more than 8
// (in log2): P <= 2^8 then, the sums stay in range, and O in TMEM is rescaled only at those rare tiles.
// P is rounded to bf16 for the product with V, as a matrix instruction takes both operands of one type (one
// rounding of at most 2^-8 relative per term, independent between terms: outputs are off by 0.0023 of their
// norm, with float32 weights it would be 0.0017); the sum l adds the unrounded P in float32.
//
// Masked places: K of an unseen position only enters a score that is replaced by -inf. V is different
// (0 times inf is nan), so tiles that reach past ctx have V cleaned in shared memory first: positions
// past the row's nodes become 0, and nodes' elements that are not finite become 0 and are added back, at
// the end, to the rows that see them.
//
// The same frame serves the positions that groups of forked rows share (SharedArgs): there a "row" is a group,
// its nodes are all its rows' nodes, every one of which sees the group's shared positions and nothing else; the
// table is the group's first row's. Results stay float32 with their lse, for gdr_fork_attn.cu to join with the rows'
// own positions.
#pragma once

#include <algorithm>
#include <cuda.h>
#include <cuda_bf16.h>
#include <cudaTypedefs.h>

#include "gdr_serve.h"
#include "ptx.cuh"

namespace gdr {

using namespace ptx;

namespace {

constexpr int kThreads = 384;   // warps: 0 loads (kSplit: 0 keys, 2 values), 1 products, 4-11 softmax
constexpr int kBlocks = kNumSMs;
constexpr int kM = 128;         // rows of an M tile
constexpr float kLog2e = 1.4426950408889634f;
// Units that an item's start and end count for. 16 rows of 13 nodes over up to 8192 positions with 0, 2, 3, 4
// and 6: heads of 64 53.6, 51.9, 51.5, 52.1, 53.3 us; of 128 75.3, 73.5, 73.7, 74.0, 74.5; of 256 57.9, 57.0,
// 57.0, 56.8, 56.4. 8 rows of 64 nodes over up to 16384: heads of 64 86.1, 84.5, 83.0, 83.8, 85.2; of 128
// 97.9, 94.7, 93.6, 93.4, 93.6. Two rows over 131072: within 1% from 2 on.
constexpr int kPad = 3;
constexpr long long kDrainBudget = 2000000000ll;   // cycles an aborting block waits for its own work

enum Form { kSplit = 0, kNarrow = 1, kWide = 2 };

struct Args {
  static constexpr bool kShared = false;
  const __nv_bfloat16* q;
  const int32_t* table;
  const int32_t* ctx;
  const int32_t* lengths;
  const uint64_t* mask;
  const __nv_bfloat16* v_pages;
  float sl2;                 // scale log2(e)
  __nv_bfloat16* o;
  float* lse;
  float* part_o;             // [2 C][rows of an item][D]
  float* part_lse;           // [2 C][rows of an item]
  int items;                 // B Hk mts
  int mts;                   // items of a row and key head, N nodes' worth
  int B, N, Hq, Hk, G, W, P, page, page_shift, M;
  int npt, npi;              // nodes of an M tile, of an item
  long long budget;
  int* err;
};
// Groups of rows in the place of rows: B groups, group t the rows first[t] .. first[t + 1] - 1 of N_row nodes each.
struct SharedArgs : Args {
  static constexpr bool kShared = true;
  const int32_t* first;      // [B + 1]
  const int32_t* shared;     // [B]
  int rows, N_row;
  float* dense_o;            // [rows N_row][Hq][D]
  float* dense_lse;          // [rows N_row][Hq]
};

template <int D, int kForm>
struct Cfg {
  static constexpr int KT = kForm == kSplit ? 64 : 128;      // positions of a tile
  static constexpr int kTiles = kForm == kWide ? 2 : 1;      // M tiles of an item
  // Keys and values loaded by a warp each: with pages of 16 a tile of heads of 256 takes 32 copies of 2 KB, and one warp does not
  // issue them in time (pages of 32 and more, or fewer queries: the same times).
  static constexpr bool kTwoLoad = kForm == kSplit;
  static constexpr int kRows = kTiles * kM;
  static constexpr uint32_t kTile = KT * D * 2;              // bytes of a K or V tile
  static constexpr int NS = D == 64 ? 8 : kForm == kNarrow ? 6 : kForm == kWide ? 5 : 7;   // tile buffers
  static constexpr uint32_t kQTile = kForm == kSplit ? 0 : kM * D * 2;   // (kSplit: in TMEM)
  static constexpr uint32_t kRing = kTiles * kQTile;
  static constexpr uint32_t kRed = kRing + NS * kTile;       // float [2][2][128]
  static constexpr uint32_t kBars = kRed + 2048;
  static constexpr uint32_t kSmem = kBars + 512;
  static constexpr uint32_t kTmemO = 2 * KT;                 // two S buffers at columns 0 and KT: kSplit's tiles alternate, else one a stream
  static constexpr uint32_t kTmemQ = kTmemO + D;             // (kSplit) the queries: all 512 columns
};

struct Bars {
  uint64_t full[8], empty[8];
  uint64_t q_full, q_empty, q_there;   // (q_there: kSplit's queries are in TMEM)
  uint64_t s_full[2], p_full[2], pv[2];   // by S buffer: S formed, P written, P V done
  uint64_t o_free;     // the segment's accumulators have been read
  uint64_t drain;
  uint32_t tmem;
  int bad[3];          // a cleaned node element was not finite, by segment modulo three
  // the block's first unit, found by the thread whose rows hold it
  int b0, hk0, mt0, t0;
  long long todo;
  int later;           // that unit begins an item after the share's first unit
  long long filled[2]; // the loading warps' next tiles of keys and values when they end
};
static_assert(sizeof(Bars) <= 512, "barriers fit their region");

// A group of rows that share positions: whether its entries are in range.
__device__ __forceinline__ bool group_valid(int f0, int f1, int shared, int rows, int page, int M) {
  return f0 >= 0 && f1 >= f0 && f1 <= rows && shared >= 0 && shared % page == 0 && shared <= (long long)M * page;
}
// A row's nodes and context; an invalid row counts as no nodes.
template <class A>
__device__ __forceinline__ bool row_of(const A& a, int b, int& n, int& ctx) {
  if constexpr (A::kShared) {
    const int f0 = __ldg(a.first + b), f1 = __ldg(a.first + b + 1);
    ctx = __ldg(a.shared + b);
    n = 0;
    if (!group_valid(f0, f1, ctx, a.rows, a.page, a.M)) return false;
    if (ctx > 0) n = (f1 - f0) * a.N_row;
    return true;
  }
  n = a.lengths ? __ldg(a.lengths + b) : a.N;
  ctx = __ldg(a.ctx + b);
  if (n < 0 || n > a.N || ctx < 0 || (long long)ctx + n > (long long)a.M * a.page) {
    n = 0;
    return false;
  }
  return true;
}
// Key tiles of item mt of a row: a chain's item needs no position past its last node.
template <int KT, class A>
__device__ __forceinline__ int tiles_of(const A& a, int n, int ctx, int mt) {
  const int nodes = A::kShared ? 0 : a.mask ? n : min(n, (mt + 1) * a.npi);
  return (ctx + nodes + KT - 1) / KT;
}
// Units of one key head of a row: its items' key tiles, and kPad for each item's start and end.
template <int KT, class A>
__device__ __forceinline__ long long units_of(const A& a, int n, int ctx) {
  if (n == 0) return 0;
  const int mts = (n + a.npi - 1) / a.npi;
  if (A::kShared || a.mask || mts == 1) return (long long)mts * (tiles_of<KT>(a, n, ctx, mts - 1) + kPad);
  long long u = 0;
  for (int mt = 0; mt < mts; ++mt) u += tiles_of<KT>(a, n, ctx, mt) + kPad;
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

// The item after one; units are left, so there is one.
template <class A>
__device__ __forceinline__ void next_item(const A& a, int& b, int& hk, int& mt, int& n, int& ctx) {
  if (++mt * a.npi < n) return;
  mt = 0;
  if (++hk < a.Hk) return;
  hk = 0;
  do {
    ++b;
    row_of(a, b, n, ctx);
  } while (n == 0);
}

// Walks the block's segments: a run of key tiles [t0, t1) of one item.
template <int KT>
struct Walk {
  int b, hk, mt, t0, t1, tiles, n, ctx, index;
  long long todo;   // units left (not positive: none)
  template <class A>
  __device__ __forceinline__ void start(const A& a, const Bars& s) {
    b = s.b0; hk = s.hk0; mt = s.mt0; t1 = s.t0;
    todo = s.todo;
    index = -1;
    if (todo > 0) {
      row_of(a, b, n, ctx);
      tiles = tiles_of<KT>(a, n, ctx, mt);
    }
  }
  template <class A>
  __device__ __forceinline__ bool next(const A& a) {
    if (todo <= 0) return false;
    if (index >= 0) {   // the last segment ended its item
      t1 = 0;
      next_item(a, b, hk, mt, n, ctx);
      tiles = tiles_of<KT>(a, n, ctx, mt);
    }
    t0 = t1;
    t1 = (int)min((long long)tiles, t0 + todo);
    todo -= t1 - t0 + (t1 == tiles ? kPad : 0);
    ++index;
    return true;
  }
  // M tiles of the item that have nodes
  template <class A>
  __device__ __forceinline__ int m_tiles(const A& a) const { return mt * a.npi + a.npt < n ? a.npi / a.npt : 1; }
};

// Whether the phase with this parity is complete, at once (try_wait may suspend the thread for a while).
__device__ __forceinline__ bool test_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}\n"
      : "=r"(done)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return done != 0;
}
// mbar_wait by a whole warp, with one answer for all its lanes. A budget of 0 does not wait at all.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, long long budget) {
  return __all_sync(0xffffffffu, budget == 0 ? test_wait(bar, parity) : mbar_wait(bar, parity, budget));
}
// One lane of a converged warp.
__device__ __forceinline__ bool elected() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
__device__ __forceinline__ uint64_t desc64(uint32_t lo, uint32_t hi) { return (uint64_t)lo | ((uint64_t)hi << 32); }

// Two floats in one register pair.
struct F2 {
  unsigned long long v;
};
__device__ __forceinline__ F2 pack2(float lo, float hi) {
  F2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r.v) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ void unpack2(F2 x, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(x.v)); }
__device__ __forceinline__ F2 fma2(F2 a, F2 b, F2 c) {
  F2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r.v) : "l"(a.v), "l"(b.v), "l"(c.v));
  return r;
}
__device__ __forceinline__ F2 add2(F2 a, F2 b) {
  F2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r.v) : "l"(a.v), "l"(b.v));
  return r;
}

// A place in the ring of tile buffers: the buffer, and the parity of its present use.
template <int NS>
struct Ring {
  int slot = 0;
  uint32_t parity = 0;
  __device__ __forceinline__ void step(int n) {
    slot += n;
    if (slot >= NS) {
      slot -= NS;
      parity ^= 1;
    }
  }
};

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

// The units of a thread's rows [r0, r1), of those before them, and of all (the block's threads share the rows).
struct Rows {
  int r0, r1;
  long long mine, before, total;
};
template <int KT, class A>
__device__ __forceinline__ Rows count_rows(const A& a, long long* warps, bool report) {
  const int per = (a.B + (int)blockDim.x - 1) / (int)blockDim.x;
  Rows r;
  r.r0 = min(a.B, (int)threadIdx.x * per);
  r.r1 = min(a.B, r.r0 + per);
  r.mine = 0;
  for (int b = r.r0; b < r.r1; ++b) {
    int n, ctx;
    if (!row_of(a, b, n, ctx) && report) atomicCAS(a.err, 0, kErrDeviceIndex);
    r.mine += units_of<KT>(a, n, ctx) * a.Hk;
  }
  if constexpr (A::kShared) {   // groups that do not rise could overlap: none is attended
    bool falls = false;
    for (int b = r.r0; b < r.r1; ++b) falls |= __ldg(a.first + b) > __ldg(a.first + b + 1);
    if (__syncthreads_or(falls)) r.mine = 0;
  }
  r.total = block_sum(r.mine, warps, r.before);
  return r;
}
// An item (row, key head, M tiles), and a unit's place in it.
struct Place {
  int b, hk, mt, n, ctx, tiles, unit;
};
// The place of unit x < total: true in the one thread that holds its row.
template <int KT, class A>
__device__ __forceinline__ bool locate(const A& a, const Rows& r, long long x, Place& p) {
  if (x < r.before || x >= r.before + r.mine) return false;
  long long at = x - r.before;
  for (p.b = r.r0;; ++p.b) {
    row_of(a, p.b, p.n, p.ctx);
    const long long head = units_of<KT>(a, p.n, p.ctx);
    if (at >= head * a.Hk) {
      at -= head * a.Hk;
      continue;
    }
    p.hk = (int)(at / head);
    at -= p.hk * head;
    for (p.mt = 0; at >= (p.tiles = tiles_of<KT>(a, p.n, p.ctx, p.mt)) + kPad; ++p.mt) at -= p.tiles + kPad;
    p.unit = (int)at;
    return true;
  }
}

// Bits k = 0 .. 63: position pos0 + k is seen by node i (rel = pos0 - ctx).
// words: the node's mask, word0 its first word (loaded once a segment).
template <class A>
__device__ __forceinline__ uint64_t seen(const A& a, const uint64_t* words, uint64_t word0, int i, int n, long long rel) {
  if (rel + 64 <= 0) return ~0ull;
  if constexpr (A::kShared) return rel < 0 ? (1ull << -rel) - 1 : 0;
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
    const uint64_t lo = w == 0 ? word0 : w < a.W ? __ldg(words + w) : 0, hi = (o && w + 1 < a.W) ? __ldg(words + w + 1) : 0;
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

__device__ __forceinline__ float got(const float* p) { return __ldcg(p); }
__device__ __forceinline__ float got(const __nv_bfloat16* p) {
  return __uint_as_float((uint32_t)__ldcg(reinterpret_cast<const unsigned short*>(p)) << 16);
}
__device__ __forceinline__ void put(float* p, float x) { *p = x; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float x) { *p = __float2bfloat16(x); }
// Adds the elements of seen nodes' V that are not finite (cleaned away before the product) to what the
// warp has just written to out[0 .. cols).
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
      if (!(fabsf(x) < INFINITY)) put(out + d, got(out + d) + x);
    }
  }
}

// Cleans positions from ctx on of a V tile in shared memory: past the row's nodes to 0, elements that are
// not finite to 0 as well (true if there are any). Threads [0, count) share it.
template <int D, int KT>
__device__ __forceinline__ bool clean_tile(uint8_t* vt, int t, int ctx, int end, int thread, int count) {
  const int r0 = max(0, ctx - t * KT);
  bool bad = false;
  for (int x = thread; x < (KT - r0) * (D / 8); x += count) {
    const int r = r0 + x / (D / 8), ch = x % (D / 8);
    uint4* p = reinterpret_cast<uint4*>(vt + (ch >> 3) * KT * 128 + r * 128 + (ch & 7) * 16);
    if (t * KT + r >= end) {
      *p = make_uint4(0, 0, 0, 0);
      continue;
    }
    uint4 v = *p;
    uint32_t* u = reinterpret_cast<uint32_t*>(&v);
    // an exponent of all ones carries into the sign's place when one is added to it
    uint32_t hit = 0;
#pragma unroll
    for (int e = 0; e < 4; ++e) hit |= ((u[e] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
    if (hit) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        if ((u[e] & 0x7F80u) == 0x7F80u) u[e] &= 0xFFFF0000u;
        if ((u[e] & 0x7F800000u) == 0x7F800000u) u[e] &= 0xFFFFu;
      }
      *p = v;
      bad = true;
    }
  }
  return bad;
}

// Largest of n scores, with four chains.
template <int n>
__device__ __forceinline__ float largest(const float* x) {
  float m[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
  for (int c = 4; c < n; c += 4) {
#pragma unroll
    for (int e = 0; e < 4; ++e) m[e] = fmaxf(m[e], x[c + e]);
  }
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}
// p = 2^(x sl2 + off) of n scores as bf16 pairs; returns their float32 sum.
template <int n>
__device__ __forceinline__ float weights(const float* x, float sl2, float off, uint32_t* p) {
  const F2 k = pack2(sl2, sl2), o = pack2(off, off);
  F2 sum[2] = {{0}, {0}};
#pragma unroll
  for (int c = 0; c < n; c += 2) {
    float a, b;
    unpack2(fma2(pack2(x[c], x[c + 1]), k, o), a, b);
    a = ex2_approx(a);
    b = ex2_approx(b);
    sum[(c >> 1) & 1] = add2(sum[(c >> 1) & 1], pack2(a, b));
    p[c >> 1] = pack_bf16x2(a, b);
  }
  float a, b;
  unpack2(add2(sum[0], sum[1]), a, b);
  return a + b;
}
template <int n>
__device__ __forceinline__ void hide(float* x, uint64_t seen) {
#pragma unroll
  for (int c = 0; c < n; ++c)
    if (!(seen >> c & 1)) x[c] = -INFINITY;
}
// Multiplies kCols accumulator columns of the warp's rows.
template <int kCols>
__device__ __forceinline__ void rescale(uint32_t at, float f) {
#pragma unroll 1
  for (int c = 0; c < kCols; c += 32) {
    float o[32];
    uint32_t u[32];
    tmem_ld32(at + c, o);
#pragma unroll
    for (int e = 0; e < 32; ++e) u[e] = __float_as_uint(o[e] * f);
    tmem_st32(at + c, u);
  }
}
// Four lanes hold four 16-byte units of a row each; afterwards lane q of the four holds unit q of their
// four rows.
__device__ __forceinline__ void turn_units(uint32_t (&u)[4][4]) {
  const int q = threadIdx.x & 3;
#pragma unroll
  for (int m = 1; m <= 2; m <<= 1) {
#pragma unroll
    for (int x = 0; x < 4; ++x) {
      if (x & m) continue;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t got = __shfl_xor_sync(0xffffffffu, (q & m) ? u[x][e] : u[x | m][e], m);
        if (q & m) u[x][e] = got;
        else u[x | m][e] = got;
      }
    }
  }
}
// 32 scaled accumulator columns of the warp's rows to o (bf16) or to the part (float32). A thread's columns
// are 64 or 128 bytes of one row: written as they are, a store would touch 32 rows, and the stores were two
// thirds of a segment's end. at[k]: the place of row k of the lane's four in units of 16 bytes (< 0: none).
__device__ __forceinline__ void put32(const float* o, bool whole, uint4* out, const long long (&at)[4]) {
  const int q = threadIdx.x & 3;
  if (whole) {
    uint32_t u[4][4];
#pragma unroll
    for (int x = 0; x < 4; ++x)
#pragma unroll
      for (int e = 0; e < 4; ++e) u[x][e] = pack_bf16x2(o[8 * x + 2 * e], o[8 * x + 2 * e + 1]);
    turn_units(u);
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (at[k] >= 0) out[at[k] + q] = make_uint4(u[k][0], u[k][1], u[k][2], u[k][3]);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint32_t u[4][4];
#pragma unroll
      for (int x = 0; x < 4; ++x)
#pragma unroll
        for (int e = 0; e < 4; ++e) u[x][e] = __float_as_uint(o[16 * h + 4 * x + e]);
      turn_units(u);
#pragma unroll
      for (int k = 0; k < 4; ++k)
        if (at[k] >= 0) out[at[k] + 4 * h + q] = make_uint4(u[k][0], u[k][1], u[k][2], u[k][3]);
    }
  }
}

constexpr uint32_t kSoftmaxBar = 1;   // named barrier of the eight softmax warps; 2 .. 5: pairs of kSplit
constexpr uint32_t kLoadBar = 6;      // of the two loading warps of kSplit

template <int D, int kForm, class A>
__global__ void __launch_bounds__(kThreads, 1)
    tree_attn_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                     const __grid_constant__ CUtensorMap mv, const __grid_constant__ A a) {
  using C = Cfg<D, kForm>;
  constexpr int KT = C::KT, NS = C::NS;
  extern __shared__ __align__(1024) uint8_t sm[];
  Bars& s = *reinterpret_cast<Bars*>(sm + C::kBars);
  float* red = reinterpret_cast<float*>(sm + C::kRed);
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (smem_u32(sm) & 1023u) {   // the swizzled tiles rely on it
    if (tid == 0) atomicCAS(a.err, 0, kErrTimeout);
    return;
  }

  if (tid == 64) {   // (the first warps have the first rows to count)
    for (int i = 0; i < NS; ++i) {
      mbar_init(&s.full[i], 1);
      mbar_init(&s.empty[i], 1);
    }
    mbar_init(&s.q_full, 1);
    mbar_init(&s.q_empty, 1);
    mbar_init(&s.q_there, 8);
    for (int i = 0; i < 2; ++i) {
      mbar_init(&s.s_full[i], 1);
      mbar_init(&s.p_full[i], kForm == kSplit ? 8 : 4);
      mbar_init(&s.pv[i], 1);
    }
    mbar_init(&s.o_free, 8);
    mbar_init(&s.drain, 1);
    for (int i = 0; i < 3; ++i) s.bad[i] = 0;
    fence_mbar_init();
    prefetch_tmap(&mq);
    prefetch_tmap(&mk);
    prefetch_tmap(&mv);
  }
  if (warp == 1) tmem_alloc(&s.tmem, 512);
  // the block's share of the units
  {
    if (tid == 0) s.todo = 0;
    const Rows rows = count_rows<KT>(a, reinterpret_cast<long long*>(red), blockIdx.x == 0);
    const long long x0 = first_unit(rows.total, blockIdx.x), x1 = first_unit(rows.total, blockIdx.x + 1);
    Place at;
    if (x1 > x0 && locate<KT>(a, rows, x0, at)) {
      const int skip = at.tiles + kPad - at.unit;
      const bool later = skip <= kPad;   // behind the item's last tile
      if (later && x1 - x0 > skip) {
        next_item(a, at.b, at.hk, at.mt, at.n, at.ctx);
        at.unit = 0;
      }
      s.todo = later ? x1 - x0 - skip : x1 - x0;
      s.later = later;
      s.b0 = at.b;
      s.hk0 = at.hk;
      s.mt0 = at.mt;
      s.t0 = at.unit;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tb = s.tmem;
  launch_dependents();
  __syncwarp();
  // A softmax thread holds a row of S in registers. The block was launched with 384 x 168 registers; the
  // first warpgroup gives back 128 x 88 of them, the other two take 256 x 40.
  bool ok = true;
  if (warp < 4) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
    if (warp == 0 || (C::kTwoLoad && warp == 2)) {
    // ------------------------------------------------------------------------------ loads
    const int kv0 = C::kTwoLoad ? warp >> 1 : 0, kvs = C::kTwoLoad ? 1 : 2;   // keys (0), values (1) or both in turn
    Walk<KT> w;
    w.start(a, s);
    const int rows = min(a.page, KT);                       // positions of one box
    const uint32_t box = rows * 128u;                       // its bytes in one 64-column slab
    const int most = KT / rows;                             // boxes of a tile
    Ring<NS> ring;
    ring.step(kv0);
    long long fill = kv0;                                   // of the block's tiles of keys and values, in turn
    int q_loads = 0;
    while (ok && w.next(a)) {
      const int end = A::kShared ? w.ctx : w.ctx + w.n;
      int trow = w.b, qrow = w.b, node = w.mt * a.npi;   // the table's row; the queries' place
      if constexpr (A::kShared) {
        trow = __ldg(a.first + w.b);
        qrow = 0;
        node += trow * a.N_row;
      }
      const int32_t* table = a.table + (size_t)trow * a.M;
      // this lane's box of tile t: its page, or -1 where the tile has no such box
      auto page_at = [&](int t) {
        const int pos = t * KT + lane * rows;
        return lane < most && pos < end ? __ldg(table + (pos >> a.page_shift)) : -1;
      };
      int pg = page_at(w.t0);
      for (int t = w.t0; ok && t < w.t1; ++t) {
        const int pieces = min(most, (end - t * KT + rows - 1) / rows);
        const int at = (t * KT + lane * rows) & (a.page - 1);
        int src = pg;
        if (t + 1 < w.t1) pg = page_at(t + 1);   // (in flight while this tile waits for its buffers)
        if (lane < pieces && (src < 0 || src >= a.P)) {   // read as zeros (outside the tensor) and reported
          atomicCAS(a.err, 0, kErrDeviceIndex);
          src = -1;
        }
        for (int kv = kv0; kv < kv0 + kvs; ++kv) {
          const int slot = ring.slot;
          if (fill >= NS) ok = warp_wait(&s.empty[slot], ring.parity ^ 1, a.budget);
          if (!ok) break;
          fill += 3 - kvs;
          if (lane == 0) mbar_arrive_expect_tx(&s.full[slot], pieces * box * (D / 64));
          __syncwarp();
          if (lane < pieces) {
            uint8_t* dst = sm + C::kRing + slot * C::kTile + lane * box;
#pragma unroll
            for (int h = 0; h < D / 64; ++h)
              tma_load_4d(dst + h * KT * 128, kv ? &mv : &mk, &s.full[slot], h * 64, w.hk, at, src);
          }
          __syncwarp();
          ring.step(3 - kvs);
        }
        if (!ok) break;
        if (kForm != kSplit && t == w.t0) {
          // the segment's queries, once the last segment's are done with: after the first tile, which
          // needs only free buffers, is on its way
          if (w.index > 0) ok = warp_wait(&s.q_empty, (w.index - 1) & 1, a.budget);
          if (!ok) break;
          if (lane == 0) {
            const int m_tiles = w.m_tiles(a);
            mbar_arrive_expect_tx(&s.q_full, (uint32_t)(D / 64) * m_tiles * a.G * a.npt * 128u);
            for (int m = 0; m < m_tiles; ++m)
              for (int h = 0; h < D / 64; ++h)
                tma_load_4d(sm + m * C::kQTile + h * kM * 128, &mq, &s.q_full, h * 64, w.hk * a.G, node + m * a.npt, qrow);
          }
          __syncwarp();
          ++q_loads;
        }
      }
    }
    // no copy of this block is left in flight
    if (lane == 0) {
      s.filled[kv0] = fill;
      if (!C::kTwoLoad) s.filled[1] = fill;
    }
    __syncwarp();
    if constexpr (C::kTwoLoad) named_bar_and(kLoadBar, 64, true);
    for (int i = kv0; i < NS; i += 3 - kvs) {   // (each buffer's last filling: keys have even numbers, values odd ones)
      const long long top = max(s.filled[0], s.filled[1]) - 1;
      long long f = top - (top - i + NS) % NS;
      while (f >= 0 && f >= s.filled[f & 1]) f -= NS;
      if (f >= 0) warp_wait(&s.full[i], (uint32_t)(f / NS) & 1, kDrainBudget);
    }
    if (q_loads > 0) warp_wait(&s.q_full, (q_loads - 1) & 1, kDrainBudget);
    } else if (warp == 1) {
    // ------------------------------------------------------------------------------ products
    Walk<KT> w;
    w.start(a, s);
    const bool lead = elected();
    constexpr uint32_t kIdS = idesc_bf16(kM, KT, false, false), kIdO = idesc_bf16(kM, D, false, true);
    const uint32_t q_lo = (uint32_t)smem_desc(smem_u32(sm), 16, 1024), k_lo = (uint32_t)smem_desc(smem_u32(sm + C::kRing), 16, 1024);
    const uint32_t v_lo = (uint32_t)smem_desc(smem_u32(sm + C::kRing), KT * 128, 1024);
    const uint32_t hi = (uint32_t)(smem_desc(0, 16, 1024) >> 32);   // (the strides' high word is the same for all three)
    // S[buffer] = Q[M tile] K[slot]^T; the K buffer and Q are given back by the last products that read them
    auto scores = [&](int buf, int m, int slot, bool free_k, bool free_q) {
      const uint32_t q0 = q_lo + m * (C::kQTile >> 4), k0 = k_lo + slot * (C::kTile >> 4), d = tb + buf * KT;
      tc_fence_after();
      if (lead && ok) {
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk)
        {
          const uint64_t kd = desc64(k0 + (((kk >> 2) * KT * 128 + (kk & 3) * 32) >> 4), hi);
          if constexpr (kForm == kSplit) mma_f16_tmem_a(d, tb + C::kTmemQ + kk * 8, kd, kIdS, kk > 0);
          else mma_bf16(d, desc64(q0 + (((kk >> 2) * kM * 128 + (kk & 3) * 32) >> 4), hi), kd, kIdS, kk > 0);
        }
        mma_commit(&s.s_full[buf]);
        if (free_k) mma_commit(&s.empty[slot]);
        if (kForm != kSplit && free_q) mma_commit(&s.q_empty);
      }
      __syncwarp();
    };
    // O[stream] (+)= P[buffer] V[slot]
    auto outputs = [&](int buf, int st, int slot, bool more, bool free_v) {
      const uint32_t v0 = v_lo + slot * (C::kTile >> 4), p = tb + buf * KT, d = tb + C::kTmemO + st * D;
      const uint32_t acc = more;
      tc_fence_after();
      if (lead && ok) {
#pragma unroll
        for (int kk = 0; kk < KT / 16; ++kk)
          mma_f16_tmem_a(d, p + kk * 8, desc64(v0 + ((kk * 2048) >> 4), hi), kIdO, kk > 0 ? 1u : acc);
        mma_commit(&s.pv[buf]);
        if (free_v) mma_commit(&s.empty[slot]);
      }
      __syncwarp();
    };
    // A wait without a vote: a lane whose wait ran out issues nothing more, and the warp leaves together at
    // the end of the tile. While products run, their operands fill shared memory's bandwidth and even a
    // wait that is satisfied takes 200 to 400 cycles; so what the next products need is asked for before
    // these are issued (`early`), and waited for only if it was not there yet.
    auto early = [&](uint64_t* bar, uint32_t parity) { return test_wait(bar, parity); };
    auto wait = [&](uint64_t* bar, uint32_t parity) { ok = ok && (a.budget == 0 ? test_wait(bar, parity) : mbar_wait(bar, parity, a.budget)); };
    Ring<NS> kr, vr;                // the next tile's keys and values
    vr.step(1);
    uint32_t steps[2] = {0, 0};     // scores formed for each stream so far (kSplit: in all)
    while (ok && w.next(a)) {
      wait(kForm == kSplit ? &s.q_there : &s.q_full, w.index & 1);
      // (the same in every lane: broadcast, so that loop counts, addresses and descriptors stay in uniform registers)
      const int T = __shfl_sync(0xffffffffu, w.t1 - w.t0, 0);
      const bool first = __shfl_sync(0xffffffffu, w.index, 0) == 0;
      const uint32_t o_parity = __shfl_sync(0xffffffffu, (uint32_t)(w.index - 1) & 1, 0);
      const int streams = __shfl_sync(0xffffffffu, w.m_tiles(a), 0);   // (kWide)
      if constexpr (kForm == kSplit) {
        // S of tile j + 1, then P V of tile j
        bool k_there = false, v_there = false;
        for (int j = -1; j < T; ++j) {
          if (j + 1 < T) {
            const uint32_t x = steps[0]++;
            if (!k_there) wait(&s.full[kr.slot], kr.parity);
            if (x >= 2) wait(&s.pv[x & 1], ((x - 2) >> 1) & 1);   // (P V of tile j - 1 is done)
            if (j >= 0) v_there = early(&s.full[vr.slot], vr.parity);
            scores(x & 1, 0, kr.slot, true, j + 2 == T);
            kr.step(2);
          }
          if (j >= 0) {
            const uint32_t x = steps[0] - (j + 1 < T ? 2 : 1);      // tile j
            if (j == 0 && !first) wait(&s.o_free, o_parity);
            if (!v_there || j + 1 == T) wait(&s.full[vr.slot], vr.parity);
            wait(&s.p_full[x & 1], (x >> 1) & 1);
            k_there = j + 2 < T && early(&s.full[kr.slot], kr.parity);
            outputs(x & 1, 0, vr.slot, j > 0, true);
            vr.step(2);
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
      } else if constexpr (kForm == kWide) {
        // one buffer a stream: S of a stream's next tile goes over P of its last one, once that product is
        // done; the streams take turns. What a product needs is waited for while the one before it runs.
        for (int k = 0; k <= T; ++k) {
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            if (st >= streams) break;
            const bool last = st == streams - 1;
            if (k > 0) {
              if (k == 1 && st == 0 && !first) wait(&s.o_free, o_parity);
              wait(&s.p_full[st], (steps[st] - 1) & 1);
              outputs(st, st, vr.slot, k > 1, last);
              if (last) vr.step(2);
            }
            if (k < T) {
              if (st == 0) wait(&s.full[kr.slot], kr.parity);
              if (last) wait(&s.full[vr.slot], vr.parity);
              if (steps[st] > 0) wait(&s.pv[st], (steps[st] - 1) & 1);
              scores(st, st, kr.slot, last, k == T - 1 && last);
              ++steps[st];
              if (last) kr.step(2);
            }
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
      } else {
        // the same with tiles st, st + 2, ... of one M tile; here K and V are what is waited for, so what the
        // next products need is asked for without waiting before these are issued
        bool k_there = false, v_there = false, p_there = false;
        for (int k = 0; k <= (T + 1) / 2; ++k) {
#pragma unroll
          for (int st = 0; st < 2; ++st) {
            const int j = 2 * k + st;
            if (k > 0 && j - 2 < T) {
              if (k == 1 && st == 0 && !first) wait(&s.o_free, o_parity);
              if (!v_there) wait(&s.full[vr.slot], vr.parity);
              if (!p_there) wait(&s.p_full[st], (steps[st] - 1) & 1);
              k_there = j < T && early(&s.full[kr.slot], kr.parity);
              outputs(st, st, vr.slot, k > 1, true);
              vr.step(2);
            }
            v_there = p_there = false;
            if (j < T) {
              if (!k_there) wait(&s.full[kr.slot], kr.parity);
              if (steps[st] > 0) wait(&s.pv[st], (steps[st] - 1) & 1);
              if (j > 0) {   // the products after these: P V of the other stream's last tile
                p_there = early(&s.p_full[st ^ 1], (steps[st ^ 1] - 1) & 1);
                v_there = early(&s.full[vr.slot], vr.parity);
              }
              scores(st, 0, kr.slot, true, j == T - 1);
              ++steps[st];
              kr.step(2);
            }
            k_there = false;
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
        }
      }
    }
    // no product of this block is left in flight
    if (lead) mma_commit(&s.drain);
    warp_wait(&s.drain, 0, kDrainBudget);
    } else {
      // ------------------------------------------------------------------------------ absent nodes: 0, -inf
      const int vecs = a.Hq * D / 8;
      constexpr int kWarps = C::kTwoLoad ? 1 : 2;
      for (int x = kWarps * blockIdx.x + warp - 4 + kWarps; !A::kShared && x < a.B * a.N; x += kWarps * kBlocks) {
        const int b = x / a.N, i = x - b * a.N;
        int n, ctx;
        row_of(a, b, n, ctx);
        if (i < n) continue;
        uint4* o = reinterpret_cast<uint4*>(a.o + (size_t)x * a.Hq * D);
        for (int v = lane; v < vecs; v += 32) o[v] = make_uint4(0, 0, 0, 0);
        for (int h = lane; a.lse && h < a.Hq; h += 32) a.lse[(size_t)x * a.Hq + h] = -INFINITY;
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 208;");
    // ------------------------------------------------------------------------------ softmax
    // A warp whose wait ran out (ok) goes on through the loops without touching TMEM, so that the named
    // barriers stay matched; every other wait of the block then runs out as well.
    Walk<KT> w;
    w.start(a, s);
    const int st = (warp - 4) >> 2, quarter = warp & 3, row = 32 * quarter + lane;   // st: stream, or half of the columns
    const uint32_t rows_at = tb + ((uint32_t)(32 * quarter) << 16);
    const int wtid = tid - 128;
    long long g = 0, step = 0;   // tiles of the segments before, tiles of this stream so far
    while (w.next(a)) {
      const int m = kForm == kWide ? st : 0;                     // M tile of the item
      const int node0 = w.mt * a.npi + m * a.npt;
      const int used = max(0, min(a.npt, w.n - node0)) * a.G;
      const bool active = 32 * quarter < used, live = row < used;
      const int i = node0 + (live ? row / a.G : 0), hg = live ? row % a.G : 0;
      const uint64_t* words = a.mask && live ? a.mask + ((size_t)w.b * a.N + i) * a.W : nullptr;
      const uint64_t word0 = words ? __ldg(words) : 0;
      const int end = A::kShared ? w.ctx : w.ctx + w.n;
      const int T = w.t1 - w.t0;
      const bool masked_any = w.t1 * KT > w.ctx;
      if constexpr (kForm == kSplit) {
        // The queries into TMEM, half of its row a thread: products of 64 positions that read them from shared memory are
        // bound by that (96 KB a tile), and their place holds two more tiles. All scores of the segment before, the last
        // readers, have been waited for.
        size_t qrow = ((size_t)w.b * a.N + i) * a.Hq + w.hk * a.G + hg;
        if constexpr (A::kShared) qrow = ((size_t)__ldg(a.first + w.b) * a.N_row + i) * a.Hq + w.hk * a.G + hg;
        const uint4* from = reinterpret_cast<const uint4*>(a.q + qrow * D + st * (D / 2));
        uint4 q[D / 16];
#pragma unroll
        for (int e = 0; e < D / 16; ++e) q[e] = live ? __ldg(from + e) : make_uint4(0, 0, 0, 0);
        __syncwarp();
        if (ok) {
#pragma unroll
          for (int c = 0; c < D / 64; ++c) tmem_st16_nowait(rows_at + C::kTmemQ + st * (D / 4) + c * 16, reinterpret_cast<const uint32_t*>(q + 4 * c));
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&s.q_there);
      }
      float m_ref = -INFINITY, l = 0.f;
      const bool works = kForm != kWide || st == 0 || used > 0;   // (an item's second M tile may be empty)
      constexpr int kStep = kForm == kNarrow ? 2 : 1;
      for (int j = kForm == kNarrow ? st : 0; works && j < T; j += kStep, ++step) {
        const int t = w.t0 + j;
        const bool masked = (t + 1) * KT > w.ctx;
        // this tile's buffer and how often it was used before
        const long long use = kForm == kSplit ? g + j : step;
        const int buf = kForm == kSplit ? (int)(use & 1) : st;
        const uint32_t phase = kForm == kSplit ? (uint32_t)(use >> 1) & 1 : (uint32_t)use & 1;
        // V of a masked tile (kWide: the first M tile's product with V is issued first, so its warps clean for
        // both). A parity tells a phase from the next one alone: in the ring's first round V may be asked for
        // at once, later only when S is there, whose product comes after the one with the buffer's last V.
        const long long fill = 2 * (g + j) + 1;
        auto clean = [&] {
          ok = ok && warp_wait(&s.full[fill % NS], (uint32_t)(fill / NS) & 1, a.budget);
          if (ok) {
            uint8_t* vt = sm + C::kRing + (fill % NS) * C::kTile;
            if (clean_tile<D, KT>(vt, t, w.ctx, end, kForm == kSplit ? wtid : wtid & 127, kForm == kSplit ? 256 : 128))
              s.bad[w.index % 3] = 1;
            fence_async_smem();
          }
          __syncwarp();   // the lanes' shares differ, and what follows on TMEM wants the whole warp
        };
        const bool cleans = masked && (kForm != kWide || st == 0);
        if (cleans && fill < NS) clean();
        ok = ok && warp_wait(&s.s_full[buf], phase, a.budget);
        if (cleans && fill >= NS) clean();
        const uint32_t sb = rows_at + buf * KT;
        if (active) {
          // this thread's columns of its row: all, or a half
          constexpr int kCols = kForm == kSplit ? KT / 2 : KT;
          const int col0 = kForm == kSplit ? st * kCols : 0;
          float x[kCols];
          if (ok) {
            tc_fence_after();
            if constexpr (kCols == 32) {
              tmem_ld32(sb + col0, x);
            } else {
#pragma unroll
              for (int c = 0; c < kCols; c += 64) tmem_ld64(sb + c, x + c);
            }
          }
          if (masked && live) {
            const long long rel = (long long)t * KT + col0 - w.ctx;
            if constexpr (kCols == 32) {
              hide<32>(x, seen(a, words, word0, i, w.n, rel));
            } else {
#pragma unroll
              for (int c = 0; c < kCols; c += 64) hide<64>(x + c, seen(a, words, word0, i, w.n, rel + c));
            }
          }
          float mx = largest<kCols>(x);
          __syncwarp();   // (rows differ in what they hide)
          if constexpr (kForm == kSplit) {
            float* mine = red + ((g + j) & 1) * 256;
            mine[st * 128 + row] = mx;
            tc_fence_before();   // (P goes over scores that the other half has read)
            ok = named_bar_and(2 + quarter, 64, ok);
            tc_fence_after();
            mx = fmaxf(mx, mine[(st ^ 1) * 128 + row]);
          }
          // (rows past the tile's nodes hold arbitrary scores and never ask for a new reference)
          const bool need = live && mx > m_ref && (m_ref == -INFINITY || (mx - m_ref) * a.sl2 > 8.f);
          if (__any_sync(0xffffffffu, need)) {
            const float m_new = live ? fmaxf(m_ref, mx) : m_ref;
            if (j >= kStep) {
              const float f = m_ref == m_new ? 1.f : ex2_approx((m_ref - m_new) * a.sl2);
              l *= f;
              if (kForm != kSplit) ok = ok && warp_wait(&s.pv[st], (uint32_t)(use - 1) & 1, a.budget);
              else ok = ok && warp_wait(&s.pv[buf ^ 1], (uint32_t)((use - 1) >> 1) & 1, a.budget);
              if (ok) {
                tc_fence_after();
                if (kForm == kSplit) rescale<D / 2>(rows_at + C::kTmemO + st * (D / 2), f);
                else rescale<D>(rows_at + C::kTmemO + st * D, f);
              }
            }
            m_ref = m_new;
          }
          const float off = m_ref == -INFINITY ? 0.f : -m_ref * a.sl2;
          if constexpr (kCols == 32) {
            uint32_t p[16];
            l += weights<32>(x, a.sl2, off, p);
            if (ok) tmem_st16_nowait(sb + st * 16, p);
          } else {
#pragma unroll
            for (int c = 0; c < kCols; c += 32) {
              uint32_t p[16];
              l += weights<32>(x + c, a.sl2, off, p);
              if (ok) tmem_st16_nowait(sb + c / 2, p);
            }
          }
          if (ok) tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0 && ok) mbar_arrive(&s.p_full[buf]);
      }
      // the segment's result: the last product of this stream, then what the warpgroups tell each other
      if (works && T > (kForm == kNarrow ? st : 0)) {
        if (kForm == kSplit) ok = ok && warp_wait(&s.pv[(g + T - 1) & 1], (uint32_t)((g + T - 1) >> 1) & 1, a.budget);
        else ok = ok && warp_wait(&s.pv[st], (uint32_t)(step - 1) & 1, a.budget);
      }
      float* ml = red + ((g + T) & 1) * 256;   // (kSplit: not where the last tile's maxima are)
      float2* both_ml = reinterpret_cast<float2*>(red);
      if constexpr (kForm == kSplit) ml[st * 128 + row] = l;
      if constexpr (kForm == kNarrow) both_ml[st * 128 + row] = make_float2(m_ref, l);
      __syncwarp();
      ok = named_bar_and(kSoftmaxBar, 256, ok);
      const bool bad = masked_any && s.bad[w.index % 3];
      if (wtid == 0) s.bad[(w.index + 2) % 3] = 0;   // read before this barrier, set after the next
      float self = 1.f, other = 0.f;                  // kNarrow: factors of the two streams' accumulators
      if constexpr (kForm == kSplit) l += ml[(st ^ 1) * 128 + row];
      if constexpr (kForm == kNarrow) {
        const float2 two = both_ml[(st ^ 1) * 128 + row];
        const float top = fmaxf(m_ref, two.x);
        self = m_ref == top ? 1.f : ex2_approx((m_ref - top) * a.sl2);
        other = two.x == top ? 1.f : ex2_approx((two.x - top) * a.sl2);
        l = l * self + two.y * other;
        m_ref = top;
      }
      __syncwarp();
      if constexpr (kForm != kWide) ok = named_bar_and(kSoftmaxBar, 256, ok);   // `red` may be written again
      const bool sees = l > 0.f || l != l;
      const float inv = sees ? 1.f / l : 0.f;
      const float lse = sees ? m_ref * a.sl2 * (1.f / kLog2e) + logf(l) : -INFINITY;
      const bool whole = w.t0 == 0 && w.t1 == w.tiles;
      size_t orow = ((size_t)w.b * a.N + i) * a.Hq + w.hk * a.G + hg;
      if constexpr (A::kShared) orow = ((size_t)__ldg(a.first + w.b) * a.N_row + i) * a.Hq + w.hk * a.G + hg;
      const size_t prow = (size_t)(2 * blockIdx.x + (w.index > 0 || s.later)) * C::kRows + m * kM + row;
      constexpr int kOut = kForm == kWide ? D : D / 2;           // this thread's output columns
      const int d0 = kForm == kWide ? 0 : st * (D / 2);
      if (active && ok) {
        tc_fence_after();
        const bool both = kForm == kNarrow && T > 1;             // (one tile: the second accumulator was not written)
        // the places of the rows of this lane's four: of o, or of the part
        constexpr bool kF32 = A::kShared;                        // a whole item's result stays float32
        uint4* out = reinterpret_cast<uint4*>(whole ? (void*)a.o : (void*)a.part_o);
        if constexpr (A::kShared) out = reinterpret_cast<uint4*>(whole ? a.dense_o : a.part_o);
        long long at[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const long long mine = whole && !kF32 ? (long long)orow * (D / 8) + d0 / 8
                                                : (long long)(whole ? orow : prow) * (D / 4) + d0 / 4;
          at[k] = __shfl_sync(0xffffffffu, live ? mine : -1, (lane & ~3) | k);
        }
        const float f0 = (st == 0 || kForm != kNarrow ? self : other) * inv, f1 = (st == 0 ? other : self) * inv;
#pragma unroll 1   // (a call on few positions is bound by fetching its instructions)
        for (int c = 0; c < kOut; c += 32) {
          float o[32];
          tmem_ld32(rows_at + C::kTmemO + (kForm == kWide ? st * D : 0) + d0 + c, o);
#pragma unroll
          for (int e = 0; e < 32; ++e) o[e] *= f0;
          if constexpr (kForm == kNarrow) {
            if (both) {
              float o1[32];
              tmem_ld32(rows_at + C::kTmemO + D + d0 + c, o1);
#pragma unroll
              for (int e = 0; e < 32; ++e) o[e] = fmaf(o1[e], f1, o[e]);
            }
          }
          put32(o, whole && !kF32, out + (whole && !kF32 ? c / 8 : c / 4), at);
          __syncwarp();   // (before the next load of the whole warp)
        }
        if (bad) __threadfence();   // (add_back reads what neighbouring lanes wrote)
        __syncwarp();
        tc_fence_before();
      }
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&s.o_free);
      if (active && live && ok) {
        if (!A::kShared && bad) {
          if (whole) add_back(a, w.b, w.hk, i, w.n, w.ctx, w.t0 * KT, w.t1 * KT, D, d0, kOut, a.o + orow * D + d0);
          else add_back(a, w.b, w.hk, i, w.n, w.ctx, w.t0 * KT, w.t1 * KT, D, d0, kOut, a.part_o + prow * D + d0);
        }
        if (kForm == kWide || st == 0) {
          if (!whole) a.part_lse[prow] = lse;
          else if constexpr (A::kShared) a.dense_lse[orow] = lse;
          else if (a.lse) a.lse[orow] = lse;
        }
      }
      g += T;
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

// Joins the parts of items that several blocks shared: o = sum_s e^(lse_s - lse) o_s over a row's parts.
// Grid (item, or block that begins one; share of the item's rows). What follows from the rows' lengths is
// worked out before the first kernel has ended, and the first parts are read while their greatest lse is
// found: only the parts' reading and the sum are left to wait for (both together: 86.1 -> 81.6 us for 2 rows
// of 131072 positions, 16.4 -> 14.4 us for one token). An item in eight parts or more (few items, each cut
// over many blocks) has the block's eight warps share a row, warp w taking parts w, w + 8, ... and the block
// adding the warps' sums in order; otherwise a warp takes a row. Parts are read four at a time: the loop is
// bound by their latency (38 parts of 224 rows of 256: 33 us by one warp a row, one part after the other).
constexpr int kJoinThreads = 256, kJoinWarps = kJoinThreads / 32;
// Blocks an SM: as many as fit at once, or the rest would begin their set-up only when the first kernel has
// ended. With 2, 3, 4 and 8: 16 rows of 13 nodes, heads of 64 55.3, 53.1, 51.5, 51.7 us, of 128 76.5, 74.9,
// 73.7, 75.0, of 256 66.3, 58.7, 57.0, 55.5; 8 rows of 64 nodes, heads of 64 92.5, 85.6, 83.0, 81.8, of 128
// 101.8, 95.8, 93.6, 94.2.
constexpr int kJoinPerSM = 4;
template <int D, int kRows, int KT, class A>
__global__ void __launch_bounds__(kJoinThreads) tree_attn_join_kernel(const __grid_constant__ A a) {
  constexpr int kVec = D / 32;
  __shared__ float s_acc[kJoinWarps][D];
  __shared__ float s_sum[kJoinWarps];
  __shared__ int s_part[kBlocks];
  __shared__ long long s_warps[kJoinWarps], s_unit;
  __shared__ int s_first, s_last;
  __shared__ Place s_item;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // the item, and the blocks that hold its parts: from the rows alone, before the first kernel has ended
  if (tid == 0) s_first = s_last = 0;
  const Rows rows = count_rows<KT>(a, s_warps, false);
  Place p;
  bool mine = false;   // one thread has the item, if there is one
  long long unit;
  if (a.items <= kBlocks) {   // a block of the grid for each item
    p.b = blockIdx.x / (a.Hk * a.mts);
    if (rows.total > 0 && p.b >= rows.r0 && p.b < rows.r1) {
      p.hk = blockIdx.x / a.mts % a.Hk;
      p.mt = blockIdx.x % a.mts;
      unit = rows.before;
      for (int b = rows.r0; b < p.b; ++b) {
        row_of(a, b, p.n, p.ctx);
        unit += units_of<KT>(a, p.n, p.ctx) * a.Hk;
      }
      row_of(a, p.b, p.n, p.ctx);
      if (p.mt * a.npi < p.n) {
        unit += units_of<KT>(a, p.n, p.ctx) * p.hk;
        for (int mt = 0; mt < p.mt; ++mt) unit += tiles_of<KT>(a, p.n, p.ctx, mt) + kPad;
        p.tiles = tiles_of<KT>(a, p.n, p.ctx, p.mt);
        mine = true;
      }
    }
  } else {                    // for each block of the first kernel: the item that its share's last unit lies in
    const long long x0 = first_unit(rows.total, blockIdx.x), x1 = first_unit(rows.total, blockIdx.x + 1);
    if (x1 > x0 && locate<KT>(a, rows, x1 - 1, p)) {
      unit = x1 - 1 - p.unit;
      mine = unit >= x0 && p.unit < p.tiles;
    }
  }
  if (mine) {
    s_item = p;
    s_unit = unit;
    s_first = block_of(rows.total, unit);
    s_last = block_of(rows.total, unit + p.tiles - 1);
  }
  __syncthreads();
  p = s_item;
  unit = s_unit;
  const int first = s_first, last = s_last;
  const int b = p.b, hk = p.hk, mt = p.mt, n = p.n;
  const int node0 = mt * a.npi, nodes = min(a.npi, n - node0);
  // the parts' places, block by block (-1: a block without units). A block's first segment is its part 0:
  // the first block's only where the item begins its share
  const int parts = last - first + 1;
  if (tid < parts) {
    const int c = first + tid;
    const long long at = first_unit(rows.total, c);
    s_part[tid] = at < first_unit(rows.total, c + 1) ? (2 * c + (at < unit)) * kRows : -1;
  }
  __syncthreads();
  if constexpr (A::kShared) launch_dependents();
  wait_prerequisite();         // (in every block: this grid must not end before the first one)
  if (last == first) return;   // whole
  const bool share = parts >= kJoinWarps;
  const int step = share ? kJoinWarps : 1;   // a warp's parts
  for (int rr = share ? blockIdx.y : blockIdx.y * kJoinWarps + warp; rr < nodes * a.G; rr += gridDim.y * (share ? 1 : kJoinWarps)) {
    const int nl = rr / a.G, hg = rr - nl * a.G, m = nl / a.npt;
    const int row = m * kM + (nl - m * a.npt) * a.G + hg;
    size_t orow = ((size_t)b * a.N + node0 + nl) * a.Hq + hk * a.G + hg;
    if constexpr (A::kShared) orow = ((size_t)__ldg(a.first + b) * a.N_row + node0 + nl) * a.Hq + hk * a.G + hg;
    float acc[kVec], top = -INFINITY, sum = 0.f;
    bool nan = false, faint = false;   // a part's lse is nan; a part's weight is below the smallest float
#pragma unroll
    for (int e = 0; e < kVec; ++e) acc[e] = 0.f;
    // four parts at once, the first of them while their greatest lse is found
    const int c0 = share ? warp : 0;
    float w[4], x[4][kVec];
    auto load = [&](int cc) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int c = cc + u * step, at = c < parts ? s_part[c] : -1;
        w[u] = -INFINITY;
        if (at < 0) continue;   // (the same in the whole warp)
        const size_t p = (size_t)at + row;
        w[u] = a.part_lse[p];
        const float* po = a.part_o + p * D + lane * kVec;
        if constexpr (kVec == 2) {
          const float2 y = *reinterpret_cast<const float2*>(po);
          x[u][0] = y.x;
          x[u][1] = y.y;
        } else {
#pragma unroll
          for (int e = 0; e < kVec; e += 4) {
            const float4 y = *reinterpret_cast<const float4*>(po + e);
            x[u][e] = y.x;
            x[u][e + 1] = y.y;
            x[u][e + 2] = y.z;
            x[u][e + 3] = y.w;
          }
        }
      }
    };
    load(c0);
    if (parts <= 4) {   // every lane has them
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        nan |= w[u] != w[u];
        top = fmaxf(top, w[u]);
      }
    } else {
      for (int c = lane; c < parts; c += 32) {
        const float lse = s_part[c] >= 0 ? a.part_lse[s_part[c] + row] : -INFINITY;
        nan |= lse != lse;
        top = fmaxf(top, lse);
      }
#pragma unroll
      for (int d = 16; d >= 1; d >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      nan = __any_sync(0xffffffffu, nan);
    }
    const float ref = top == -INFINITY ? 0.f : top;
    for (int cc = c0; cc < parts;) {
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const float f = ex2_approx((w[u] - ref) * kLog2e);
        sum += f;
        if (f != 0.f) {   // a part that saw nothing may hold anything
#pragma unroll
          for (int e = 0; e < kVec; ++e) acc[e] = fmaf(f, x[u][e], acc[e]);
        } else {
          faint |= w[u] != -INFINITY;
        }
      }
      cc += 4 * step;
      if (cc < parts) load(cc);
    }
    // (by itself, as in the loop above it cost wide trees 0.6 us instead of 0.3)
    if (faint) {   // an infinity that was seen counts, however small its weight
#pragma unroll 1
      for (int c = c0; c < parts; c += step) {
        const size_t p = (size_t)s_part[c] + row;
        const float lse = s_part[c] >= 0 ? a.part_lse[p] : -INFINITY;
        if (lse == -INFINITY || ex2_approx((lse - ref) * kLog2e) != 0.f) continue;
#pragma unroll
        for (int e = 0; e < kVec; ++e) {
          const float y = a.part_o[p * D + lane * kVec + e];
          if (!(fabsf(y) < INFINITY)) acc[e] += y;
        }
      }
    }
    if (share) {   // (the same in every warp, and so is the row)
      __syncthreads();   // the row before has been read
#pragma unroll
      for (int e = 0; e < kVec; ++e) s_acc[warp][lane * kVec + e] = acc[e];
      if (lane == 0) s_sum[warp] = sum;
      __syncthreads();
      if (warp > 0) continue;
      sum = 0.f;
#pragma unroll
      for (int e = 0; e < kVec; ++e) acc[e] = 0.f;
#pragma unroll
      for (int v = 0; v < kJoinWarps; ++v) {
        sum += s_sum[v];
#pragma unroll
        for (int e = 0; e < kVec; ++e) acc[e] += s_acc[v][lane * kVec + e];
      }
    }
    const float inv = sum > 0.f || sum != sum ? 1.f / sum : 0.f;
#pragma unroll
    for (int e = 0; e < kVec; ++e) acc[e] *= inv;
    const float lse = nan ? NAN : sum > 0.f ? ref + logf(sum) : -INFINITY;
    if constexpr (A::kShared) {
      float* out = a.dense_o + orow * D + lane * kVec;
#pragma unroll
      for (int e = 0; e < kVec; e += kVec > 2 ? 4 : 2) {
        if constexpr (kVec > 2) *reinterpret_cast<float4*>(out + e) = make_float4(acc[e], acc[e + 1], acc[e + 2], acc[e + 3]);
        else *reinterpret_cast<float2*>(out + e) = make_float2(acc[e], acc[e + 1]);
      }
      if (lane == 0) a.dense_lse[orow] = lse;
    } else {
      __nv_bfloat16* out = a.o + orow * D + lane * kVec;
#pragma unroll
      for (int e = 0; e < kVec; e += 2) *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(acc[e], acc[e + 1]);
      if (lane == 0 && a.lse) a.lse[orow] = lse;
    }
  }
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

// What the two kinds of arguments share: sizes, maps, the two launches. a holds what differs.
template <int D, int kForm, class A>
cudaError_t launch(const TreeAttnArgs& p, A a, cudaStream_t st) {
  using C = Cfg<D, kForm>;
  const int nodes = A::kShared ? p.B * p.N : p.N;   // along the queries' map, in one row or in each of B
  a.G = p.Hq / p.Hk;
  a.npt = std::min(kM / a.G, nodes);
  a.npi = C::kTiles * a.npt;
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, p.q, D, p.Hq, nodes, A::kShared ? 1 : p.B, a.G, a.npt) ||
      !make_map(&mk, p.k_pages, D, p.Hk, p.page, p.P, 1, std::min(p.page, C::KT)) ||
      !make_map(&mv, p.v_pages, D, p.Hk, p.page, p.P, 1, std::min(p.page, C::KT)))
    return cudaErrorInvalidValue;
  a.q = static_cast<const __nv_bfloat16*>(p.q);
  a.table = p.table; a.ctx = p.ctx; a.lengths = p.lengths; a.mask = A::kShared ? nullptr : p.mask;
  a.v_pages = static_cast<const __nv_bfloat16*>(p.v_pages);
  a.sl2 = p.scale * kLog2e;
  a.o = static_cast<__nv_bfloat16*>(p.o);
  a.lse = p.lse;
  a.part_o = reinterpret_cast<float*>(p.ws);
  a.part_lse = a.part_o + (size_t)2 * kBlocks * C::kRows * D;
  a.N = nodes; a.Hq = p.Hq; a.Hk = p.Hk; a.W = (p.N + 63) / 64; a.P = p.P; a.page = p.page; a.M = p.M;
  a.page_shift = __builtin_ctz((unsigned)p.page);
  a.mts = (nodes + a.npi - 1) / a.npi;
  a.items = (int)std::min<long long>((long long)a.B * p.Hk * a.mts, 0x7fffffff);
  a.budget = wait_budget_cycles();
  a.err = p.err;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(tree_attn_kernel<D, kForm, A>), C::kSmem, done);
  if (e != cudaSuccess) return e;
  int slot = stage_timer_begin(st, A::kShared ? kKernForkAttnShared : kKernTreeAttn);
  tree_attn_kernel<D, kForm, A><<<kBlocks, kThreads, C::kSmem, st>>>(mq, mk, mv, a);
  stage_timer_end(slot, st);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  // shares of an item's rows, one row each at least
  const int x = std::min(a.items, kBlocks);
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(x, std::max(1, std::min(a.npi * a.G, kNumSMs * kJoinPerSM / x)));
  cfg.blockDim = dim3(kJoinThreads);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  slot = stage_timer_begin(st, A::kShared ? kKernForkAttnShared : kKernTreeAttnJoin);
  e = cudaLaunchKernelEx(&cfg, tree_attn_join_kernel<D, C::kRows, C::KT, A>, a);
  stage_timer_end(slot, st);
  return e;
}

// Two parts a block, each of the largest item's rows: 256, or 128 for D = 256.
inline size_t parts_bytes(int D) { return (size_t)2 * kBlocks * (D == 256 ? kM : 2 * kM) * (D + 1) * sizeof(float); }

}  // namespace
}  // namespace gdr
