// Attention of forked rows whose leading positions are the same: group t's rows first[t] .. first[t + 1] - 1 share
// positions [0, shared[t]), and each goes on over positions of its own (and its drafted nodes). With the softmax
// cut at shared[t],
//   o = (e^(lse_s) o_s + e^(lse_o) o_o) / (e^(lse_s) + e^(lse_o)),
// o_s, lse_s over the shared positions, o_o, lse_o over the row's own.
//
// The shared part: all queries of a group's rows are the rows of one tensor-core problem, so that shared keys
// and values are read once for the group, whatever its size (the tcgen05 frame of gdr_attn_frame.cuh with
// groups in the place of rows). From about 280 query rows a key head on it is bound by the products, below by HBM.
//
// The own part: a key head of a row has few queries (nodes times heads a key head) over keys that nobody
// else reads, so it is bound by reading them. An item is a row, a key head and up to 8, 16, 32 or 64 of its query rows; a
// team of warps takes items one after the other. One warp looks the items up and loads (queries, and tiles of
// the row's positions as TMA boxes of its pages, several tiles and up to two items ahead), the others compute with warp-level
// matrix instructions, of which a 128-row tcgen05 tile would fill a sixteenth or less (starting and draining such an item
// takes 4 us of an SM, against 2 us for its reading). Warps that share rows take positions in turn and are joined at the
// end, in order; then the shared part's result is joined.
//   up to 8 query rows: fork_own_few_kernel, which computes the transposed products, an item a team of eight or four warps, or
//   of one or two where there are many;
//   more: fork_own_kernel, 16 query rows a warp, four warps an item.
//
// Measured (floor: bytes at 6795 GB/s or operations at 1880 TFLOP/s): 256 forks of 8 trunks of up to 8192 positions, 32 / 8
// heads of 128, 94 to 98 us (52.6 HBM): shared part 50, join 15 (partly within the others), own part 41 at 4.7 TB/s, the rest of
// that the end, where the last items run alone. 64 forks of 65536 positions, 16 / 2 heads of 256, 80 to 81 (36.6 operations):
// shared part 64, a 128-row tile an item, whose softmax runs between the products. 64 rows of 64 tokens, 4 trunks, 16 / 4 heads
// of 128, 206 to 211 (89.7 operations): shared part 149 at 60% of the matrix rate (softmax; the eighth of the nodes that is
// absent is computed, too), own part 49, bound by the latency of its steps with eight computing warps an SM. 3 forks of 448
// positions 10.3: one kernel, four tiles one after the other.
//
// Weights are rounded to bfloat16 for their product with v, the sum adds them unrounded; scores, sums and parts are
// float32.
#include "gdr_attn_frame.cuh"

namespace gdr {
namespace {

constexpr int kOwnWarps = 4, kOwnThreads = 32 * (kOwnWarps + 1);   // the last warp loads
constexpr int kOwnBar = 1;   // named barrier of the computing warps (and the next)

struct OwnArgs {
  const __nv_bfloat16 *q, *k_pages, *v_pages;
  const int32_t *table, *ctx, *lengths, *first, *shared;
  const uint64_t* mask;
  float sl2;
  __nv_bfloat16* o;
  float* lse;
  const float *dense_o, *dense_lse;
  int B, N, Hq, Hk, G, W, P, page, page_shift, M, T;
  int npt, heads, splits;    // an item's nodes and heads a node; items that a node's heads of a key head take
  int m_tiles;               // items of a row and key head
  int alone;                 // there was no shared part: this one reads the shared positions, too
  long long budget;
  int* err;
};

// Query rows of an item (16 a warp, WR of the four warps), positions of a tile, and tiles on their way.
template <int D, int WR>
struct Own {
  static constexpr int WK = kOwnWarps / WR;                  // warps that share the positions of a tile
  static constexpr int KT = WK * 16 < 32 ? 32 : WK * 16;
  static constexpr int PW = KT / WK;                         // a warp's positions
  static constexpr int kRows = 16 * WR;
  static constexpr int kTile = KT * D * 2;                   // bytes of K or V
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kAcc = kOwnWarps * 16 * D * 4;        // accumulators at the end of an item
  static constexpr int kFit = ((D == 256 ? 216 : 108) * 1024 - 2 * kQ - kAcc) / (2 * kTile);   // one or two blocks an SM
  static constexpr int NS = kFit > 4 ? 4 : kFit;
  static constexpr int kRing = 2 * kQ, kOut = kRing + NS * 2 * kTile;
  static constexpr int kSmem = kOut + kAcc;
  static_assert(NS >= 2, "a tile is loaded while another is computed");
};
// What the loading warp tells the computing ones of an item.
struct Item {
  int b, hk, node0, h0, n, own, shared, tiles;
  int lead, from;   // pages that are looked up in another row's table, and that row
  int rows, used;   // query rows, and those of them whose nodes are there
};
struct OwnBars {
  uint64_t full[4], empty[4], item_full[2], item_empty[2];
  Item item[2];
  template <int NS>
  __device__ void init(int warps) {   // (one thread)
    for (int i = 0; i < NS; ++i) {
      mbar_init(&full[i], 1);
      mbar_init(&empty[i], warps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&item_full[i], 1);
      mbar_init(&item_empty[i], warps);
    }
  }
};

// 16-byte unit ch of row r in tiles of `rows` rows, 64 columns (128 bytes) at a time, swizzled as TMA writes them.
__device__ __forceinline__ uint32_t unit_at(int rows, int r, int ch) {
  return (uint32_t)((ch >> 3) * rows * 128 + r * 128 + (((ch & 7) ^ (r & 7)) << 4));
}
// Zeroes what is not finite; whether there was any.
__device__ __forceinline__ bool finite_only(uint4& v) {
  uint32_t* u = reinterpret_cast<uint32_t*>(&v);
  uint32_t hit = 0;
#pragma unroll
  for (int e = 0; e < 4; ++e) hit |= ((u[e] & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
  if (!hit) return false;
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if ((u[e] & 0x7F80u) == 0x7F80u) u[e] &= 0xFFFF0000u;
    if ((u[e] & 0x7F800000u) == 0x7F800000u) u[e] &= 0xFFFFu;
  }
  return true;
}
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// A row's own and shared parts joined: their weights are own / total and shared / total (own's accumulator still lacks its
// sum l); m: the greatest score in binary orders.
struct Factors {
  float own, shared, total, lse;
  bool sees, rare;   // it sees something of its own; a weight vanished that is not 0
};
__device__ __forceinline__ Factors factors(bool used, bool joins, float m, float l, float lse_s) {
  Factors f;
  f.sees = used && (l > 0.f || l != l);
  const float lse = f.sees ? m * (1.f / kLog2e) + logf(l) : -INFINITY, ref = fmaxf(lse, lse_s);
  f.own = f.sees ? 1.f : 0.f;
  f.shared = 0.f;
  f.total = 1.f;
  f.lse = lse;
  f.rare = false;
  if (lse != lse || lse_s != lse_s) {
    f.own = f.shared = f.total = NAN;
  } else if (joins && ref > -INFINITY) {
    f.own = lse == ref ? 1.f : ex2_approx((lse - ref) * kLog2e);
    f.shared = lse_s == ref ? 1.f : ex2_approx((lse_s - ref) * kLog2e);
    f.rare = (f.own == 0.f && lse != -INFINITY) || (f.shared == 0.f && lse_s != -INFINITY);
    f.total = f.own + f.shared;
  }
  if (joins) f.lse = ref == -INFINITY && f.total == f.total ? -INFINITY : ref + logf(f.total);
  return f;
}

// The row's group and its numbers (a whole warp; every lane gets the item). falls: `first` is not rising.
template <class C>
__device__ __forceinline__ Item item_of(const OwnArgs& a, long long at, bool falls) {
  const int lane = threadIdx.x & 31;
  Item t;
  const int mt = (int)(at % a.m_tiles), row = (int)(at / a.m_tiles);
  t.b = row / a.Hk;
  t.hk = row - t.b * a.Hk;
  t.node0 = mt / a.splits * a.npt;
  t.h0 = mt % a.splits * a.heads;
  t.n = a.lengths ? __ldg(a.lengths + t.b) : a.N;
  const int ctx = __ldg(a.ctx + t.b);
  t.shared = t.from = 0;
  bool valid = !falls;
  // The one group that holds row b among groups g0 .. g0 + 31: of more than these, the last that begins at or before it and
  // those around it, a factor of 32 a step. (Where `first` falls what is found is not used.)
  int g0 = 0;
  for (int left = a.T; left > 32;) {
    const int step = (left + 31) >> 5, g = g0 + lane * step;
    const int before = __popc(__ballot_sync(0xffffffffu, lane * step < left && __ldg(a.first + g) <= t.b));
    const int at = max(before - 1, 0) * step;
    g0 += at;
    left = min(step, left - at);
  }
  {
    const int g = g0 + lane;
    int f0 = 0, f1 = 0, sh = 0;
    if (g < a.T) {
      f0 = __ldg(a.first + g);
      f1 = __ldg(a.first + g + 1);
      sh = __ldg(a.shared + g);
    }
    const unsigned mine = __ballot_sync(0xffffffffu, f0 <= t.b && t.b < f1);
    if (mine) {
      const int who = __ffs(mine) - 1;
      valid = valid && __shfl_sync(0xffffffffu, (int)group_valid(f0, f1, sh, a.B, a.page, a.M), who);
      t.shared = __shfl_sync(0xffffffffu, sh, who);
      t.from = __shfl_sync(0xffffffffu, f0, who);
    }
  }
  valid = valid && t.n >= 0 && t.n <= a.N && ctx >= t.shared && (long long)ctx + t.n <= (long long)a.M * a.page;
  if (!valid) {
    if (lane == 0) atomicCAS(a.err, 0, kErrDeviceIndex);
    t.n = 0;
    t.shared = 0;
  }
  t.lead = a.alone ? t.shared >> a.page_shift : 0;
  t.own = ctx - (a.alone ? 0 : t.shared);
  const int heads = min(a.heads, a.G - t.h0), nodes = max(0, min(a.npt, t.n - t.node0));
  t.rows = min(a.npt, a.N - t.node0) * heads;
  t.used = nodes * heads;
  // positions of the own part, a node from `own` on; a chain's item needs none past its last node
  const int L = nodes == 0 ? 0 : t.own + (a.mask ? t.n : t.node0 + nodes);
  t.tiles = (L + C::KT - 1) / C::KT;
  return t;
}

// The row's pages from its own part's first position on.
__device__ __forceinline__ const int32_t* own_table(const OwnArgs& a, const Item& t) {
  return a.table + (size_t)t.b * a.M + (a.alone ? 0 : t.shared >> a.page_shift);
}

// The loading warp of a team: items at0, at0 + stride, ... , two of them and NS tiles ahead of what is computed.
template <int D, class C>
__device__ __forceinline__ void load_items(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv, const OwnArgs& a, OwnBars& s,
                                           uint8_t* sm, long long at0, long long stride, int lane) {
  constexpr int KT = C::KT, NS = C::NS;
  const long long items = (long long)a.B * a.Hk * a.m_tiles;
  bool falls = false;
  for (int t = lane; t < a.T; t += 32) {
    const int f0 = __ldg(a.first + t), f1 = __ldg(a.first + t + 1);
    falls |= f0 > f1;
    if (a.alone && at0 == 0 && !group_valid(f0, f1, __ldg(a.shared + t), a.B, a.page, a.M)) atomicCAS(a.err, 0, kErrDeviceIndex);
  }
  falls = __any_sync(0xffffffffu, falls);
  const int rows = min(a.page, KT), most = KT / rows;   // positions of one box, boxes of a tile
  const uint32_t box = rows * 128u;                     // its bytes in one 64-column slab
  Ring<NS> ring;
  bool ok = true;
  int loads = 0, q_loads = 0, k = 0;
  for (long long at = at0; ok && at < items; at += stride, ++k) {
    const Item t = item_of<C>(a, at, falls);
    if (k >= 2) ok = warp_wait(&s.item_empty[k & 1], ((k >> 1) & 1) ^ 1, a.budget);
    if (!ok) break;
    // the queries: row (node, head) as the box leaves them; rows behind it hold anything and are not used
    if (lane == 0) {
      s.item[k & 1] = t;
      mbar_arrive_expect_tx(&s.item_full[k & 1], (uint32_t)(D / 64) * a.heads * a.npt * 128u);
      for (int h = 0; h < D / 64; ++h)
        tma_load_4d(sm + (k & 1) * C::kQ + h * C::kRows * 128, &mq, &s.item_full[k & 1], h * 64, t.hk * a.G + t.h0, t.node0, t.b);
    }
    __syncwarp();
    ++q_loads;
    // its positions
    const int end = t.tiles == 0 ? 0 : t.own + t.n;
    const int32_t *table = own_table(a, t), *lead = a.table + (size_t)t.from * a.M;
    auto page_at = [&](int tile) {
      const int pos = tile * KT + lane * rows, i = pos >> a.page_shift;
      return lane < most && pos < end ? __ldg((i < t.lead ? lead : table) + i) : -1;
    };
    int pg = page_at(0);
    for (int tile = 0; tile < t.tiles; ++tile) {
      const int pieces = min(most, (end - tile * KT + rows - 1) / rows), in_page = (tile * KT + lane * rows) & (a.page - 1);
      int src = pg;
      if (tile + 1 < t.tiles) pg = page_at(tile + 1);
      if (lane < pieces && (src < 0 || src >= a.P)) {   // read as zeros (outside the tensor) and reported
        atomicCAS(a.err, 0, kErrDeviceIndex);
        src = -1;
      }
      const int slot = ring.slot;
      if (loads == NS) ok = warp_wait(&s.empty[slot], ring.parity ^ 1, a.budget);
      else ++loads;
      if (!ok) break;
      if (lane == 0) mbar_arrive_expect_tx(&s.full[slot], 2 * pieces * box * (D / 64));
      __syncwarp();
      if (lane < pieces) {
        uint8_t* dst = sm + C::kRing + slot * 2 * C::kTile + lane * box;
#pragma unroll
        for (int h = 0; h < D / 64; ++h) {
          tma_load_4d(dst + h * KT * 128, &mk, &s.full[slot], h * 64, t.hk, in_page, src);
          tma_load_4d(dst + C::kTile + h * KT * 128, &mv, &s.full[slot], h * 64, t.hk, in_page, src);
        }
      }
      __syncwarp();
      ring.step(1);
    }
  }
  // no copy of this block is left in flight
  for (int i = 0; i < loads; ++i) warp_wait(&s.full[i], i < ring.slot ? ring.parity : ring.parity ^ 1, kDrainBudget);
  for (int i = max(0, q_loads - 2); i < q_loads; ++i) warp_wait(&s.item_full[i & 1], (i >> 1) & 1, kDrainBudget);
  if (!ok && lane == 0) atomicCAS(a.err, 0, kErrTimeout);
}

template <int D, int WR>
__global__ void __launch_bounds__(kOwnThreads, D == 256 ? 1 : 2)
    fork_own_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const __grid_constant__ OwnArgs a) {
  using C = Own<D, WR>;
  constexpr int KT = C::KT, PW = C::PW, NS = C::NS, WK = C::WK, kRows = C::kRows;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ OwnBars s;
  __shared__ float s_m[kOwnWarps][16], s_l[kOwnWarps][16];
  __shared__ int s_bad;   // (the last item in which V of a node was cleaned of something)
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31;
  if (smem_u32(sm) & 1023u) {   // the swizzled tiles rely on it
    if (tid == 0) atomicCAS(a.err, 0, kErrTimeout);
    return;
  }
  if (tid == 0) {
    s.template init<NS>(kOwnWarps);
    s_bad = -1;
    fence_mbar_init();
    prefetch_tmap(&mq);
    prefetch_tmap(&mk);
    prefetch_tmap(&mv);
  }
  __syncthreads();
  const long long items = (long long)a.B * a.Hk * a.m_tiles;
  const size_t step = (size_t)a.Hk * D;   // elements of a position
  bool ok = true;

  if (warp == kOwnWarps) {
    // ---------------------------------------------------------------------------------- loads
    load_items<D, C>(mq, mk, mv, a, s, sm, blockIdx.x, gridDim.x, lane);
    return;
  }

  // ------------------------------------------------------------------------------------ products and softmax
  const int wr = warp / WK, wk = warp % WK;
  // this lane's places in the rows that ldmatrix reads: of Q, of K (positions as rows) and of V
  uint32_t q_off[4], k_off[4], v_off[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    q_off[j] = unit_at(kRows, wr * 16 + (lane & 15), 2 * j + (lane >> 4));
    k_off[j] = unit_at(KT, wk * PW + (lane & 7) + ((lane >> 4) << 3), 2 * j + ((lane >> 3) & 1));
    v_off[j] = unit_at(KT, wk * PW + (lane & 15), 2 * j + (lane >> 4));
  }
  // nodes of this thread's two rows within an item, and of the row whose results this lane prepares (the i-th of the
  // warp's: rows that warps share go to them in turn); that row's place in the outputs from the item's first on
  constexpr int kMine = 16 / WK, kVec = D / 32, kAhead = D == 256 || WR == 1 ? 2 : WR == 2 ? 4 : 8;
  const int node_of[2] = {(wr * 16 + (lane >> 2)) / a.heads, (wr * 16 + (lane >> 2) + 8) / a.heads};
  const int my_row = wr * 16 + (lane % kMine) * WK + wk, my_node = my_row / a.heads;
  const int my_place = my_node * (a.Hq - a.heads) + my_row;
  const uint32_t ring_at = smem_u32(sm) + C::kRing;
  float* acc = reinterpret_cast<float*>(sm + C::kOut);
  Ring<NS> ring;
  int k = 0;
  for (long long at = blockIdx.x; at < items; at += gridDim.x, ++k) {
    // (Warps meet at barriers inside an item, so all of them go through all of its tiles, a warp whose wait ran out
    // without touching them; they leave together, here or before the results.)
    ok = named_bar_and(kOwnBar, 32 * kOwnWarps, warp_wait(&s.item_full[k & 1], (k >> 1) & 1, a.budget));
    if (!ok) break;
    const Item t = s.item[k & 1];
    const int n = t.n, own = t.own, used = t.used;
    // The shared part's results for the warp's first rows, asked for as early as they are there (from the second item on
    // before its tiles: 102.8 -> 100.6 us for 256 forks).
    const size_t base = ((size_t)t.b * a.N + t.node0) * a.Hq + t.hk * a.G + t.h0;
    const bool joins = t.shared > 0 && !a.alone;
    float shared_x[kAhead][kVec], lse_s = -INFINITY;
    auto ask = [&](int i0, float (&x)[kAhead][kVec]) {
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const size_t orow = base + __shfl_sync(0xffffffffu, my_place, i0 + u);
#pragma unroll
        for (int e = 0; e < kVec; ++e) x[u][e] = 0.f;
        if (wr * 16 + (i0 + u) * WK + wk >= used || !joins) continue;
#pragma unroll
        for (int e = 0; e < kVec; e += 2) {
          const float2 v = __ldcg(reinterpret_cast<const float2*>(a.dense_o + orow * D + lane * kVec + e));
          x[u][e] = v.x;
          x[u][e + 1] = v.y;
        }
      }
    };
    auto ask_first = [&] {
      if (joins && lane < kMine && my_row < used) lse_s = __ldcg(a.dense_lse + base + my_place);
      ask(0, shared_x);
    };
    constexpr bool kEarly = WR == 1 && D < 256;   // (registers for the rows of more warps are not left)
    if (kEarly && k > 0) ask_first();
    float o[D / 8][4];
#pragma unroll
    for (int d = 0; d < D / 8; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
    float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
    // this thread's two rows: how far a chain's node sees, or its mask
    int sees_to[2];
    const uint64_t* words[2];
    uint64_t word0[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = wr * 16 + (lane >> 2) + 8 * h, node = r < used ? t.node0 + node_of[h] : 0;
      sees_to[h] = own + min(node + 1, n);
      words[h] = a.mask ? a.mask + ((size_t)t.b * a.N + node) * a.W : nullptr;
      word0[h] = words[h] && r < used ? __ldg(words[h]) : 0;
    }
    uint32_t qf[D / 16][4];
    if (t.tiles > 0) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        ldmatrix4(smem_u32(sm) + (k & 1) * C::kQ + (kk >> 2) * kRows * 128 + q_off[kk & 3], qf[kk]);
    }
    for (int tile = 0; tile < t.tiles; ++tile) {
      ok = ok && warp_wait(&s.full[ring.slot], ring.parity, a.budget);
      const uint32_t k_at = ring_at + ring.slot * 2 * C::kTile, v_at = k_at + C::kTile;
      const int first = tile * KT + wk * PW;              // this warp's positions
      const bool masked = first + PW > own;
      if (masked) {
        // V of positions that are not there must not meet a weight of 0, nor what is not finite of nodes that some do not
        // see (a warp's own positions; warps of other rows with the same positions share them out)
        if (ok) {
          constexpr int kClean = PW / WR;
          bool bad = false;
          for (int x = lane; x < kClean * (D / 8); x += 32) {
            const int r = wr * kClean + x / (D / 8), p = first + r;
            if (p < own) continue;
            const uint32_t u_at = v_at + unit_at(KT, wk * PW + r, x % (D / 8));
            uint4 v = make_uint4(0, 0, 0, 0);
            if (p < own + n) {
              if (n == 1 && !a.mask) continue;            // (it sees itself)
              asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(u_at) : "memory");
              if (!finite_only(v)) continue;
              bad = true;
            }
            asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(u_at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
          }
          if (bad) s_bad = k;
        }
        __syncwarp();
        if (WR > 1) ok = named_bar_and(kOwnBar + 2 + wk, 32 * WR, ok);
      }
      if (ok) {
        float x[PW / 8][4];
#pragma unroll
        for (int c = 0; c < PW / 8; ++c)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[c][e] = 0.f;
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
          for (int c = 0; c < PW / 16; ++c) {
            uint32_t f[4];
            ldmatrix4(k_at + (kk >> 2) * KT * 128 + c * 16 * 128 + k_off[kk & 3], f);
            mma16816(x[2 * c], qf[kk], f[0], f[1]);
            mma16816(x[2 * c + 1], qf[kk], f[2], f[3]);
          }
        }
        if (masked) {
          if (a.mask) {
#pragma unroll
            for (int c = 0; c < PW / 8; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e) {
                const int h = e >> 1, j = first + c * 8 + 2 * (lane & 3) + (e & 1) - own;
                const bool see = j < 0 || (j < n && (((j < 64 ? word0[h] : __ldg(words[h] + (j >> 6))) >> (j & 63)) & 1));
                if (!see) x[c][e] = -INFINITY;
              }
          } else {
#pragma unroll
            for (int c = 0; c < PW / 8; ++c)
#pragma unroll
              for (int e = 0; e < 4; ++e)
                if (first + c * 8 + 2 * (lane & 3) + (e & 1) >= sees_to[e >> 1]) x[c][e] = -INFINITY;
          }
        }
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          float mx = -INFINITY;
#pragma unroll
          for (int c = 0; c < PW / 8; ++c) mx = fmaxf(mx, fmaxf(x[c][2 * h], x[c][2 * h + 1]));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
          mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * a.sl2;
          if (__any_sync(0xffffffffu, mx > m[h])) {
            const float m_new = fmaxf(m[h], mx), f = m[h] == m_new ? 1.f : ex2_approx(m[h] - m_new);
            l[h] *= f;
            if (tile > 0) {
#pragma unroll
              for (int d = 0; d < D / 8; ++d) {
                o[d][2 * h] *= f;
                o[d][2 * h + 1] *= f;
              }
            }
            m[h] = m_new;
          }
          const float off = m[h] == -INFINITY ? 0.f : -m[h];
#pragma unroll
          for (int c = 0; c < PW / 8; ++c)
#pragma unroll
            for (int e = 2 * h; e < 2 * h + 2; ++e) {
              x[c][e] = ex2_approx(fmaf(x[c][e], a.sl2, off));
              l[h] += x[c][e];
            }
        }
#pragma unroll
        for (int c = 0; c < PW / 16; ++c) {
          const uint32_t p[4] = {pack_bf16x2(x[2 * c][0], x[2 * c][1]), pack_bf16x2(x[2 * c][2], x[2 * c][3]),
                                 pack_bf16x2(x[2 * c + 1][0], x[2 * c + 1][1]), pack_bf16x2(x[2 * c + 1][2], x[2 * c + 1][3])};
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            uint32_t f[4];
            ldmatrix4_t(v_at + (d >> 2) * KT * 128 + c * 16 * 128 + v_off[d & 3], f);
            mma16816(o[2 * d], p, f[0], f[1]);
            mma16816(o[2 * d + 1], p, f[2], f[3]);
          }
        }
      }
      if (masked) fence_async_smem();   // (what was cleaned is loaded over)
      __syncwarp();
      if (lane == 0 && ok) mbar_arrive(&s.empty[ring.slot]);
      ring.step(1);
    }

    // ---------------------------------------------------------------------------------- the warps' parts
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = (lane >> 2) + 8 * h;
      if ((lane & 3) == 0) {
        s_m[warp][r] = m[h];
        s_l[warp][r] = l[h];
      }
      // (8-byte units crosswise by row: rows lie 512 bytes apart or more)
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
        *reinterpret_cast<float2*>(acc + (warp * 16 + r) * D + ((d * 8 + 2 * (lane & 3)) ^ ((r & 7) << 3))) = make_float2(o[d][2 * h], o[d][2 * h + 1]);
    }
    if (k == 0) wait_prerequisite();   // (in every block: this grid must not end before the ones it follows)
    if (!kEarly || k == 0) ask_first();
    __syncwarp();
    ok = named_bar_and(kOwnBar + 1, 32 * kOwnWarps, ok);
    if (!ok) break;

    // ---------------------------------------------------------------------------------- results: a warp a row
    // Lane i works out the factors of the warp's i-th row: of each warp's part, and of the shared part.
    const int w0 = wr * WK;
    const bool cleaned = s_bad == k;
    float c[WK], c_s = 0.f, lse = -INFINITY;
    bool rare = false;
#pragma unroll
    for (int w = 0; w < WK; ++w) c[w] = 0.f;
    if (lane < kMine && my_row < used) {
      const int rr = lane * WK + wk;
      float top = s_m[w0][rr], sum = 0.f;
#pragma unroll
      for (int w = 1; w < WK; ++w) top = fmaxf(top, s_m[w0 + w][rr]);
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        const float mw = s_m[w0 + w][rr];
        c[w] = mw == top ? 1.f : ex2_approx(mw - top);
        sum += c[w] * s_l[w0 + w][rr];
      }
      const Factors f = factors(true, joins, top, sum, lse_s);
      lse = f.lse;
      rare = f.rare;
      const float inv = f.sees ? f.own / (sum * f.total) : 0.f;
      c_s = f.shared / f.total;
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        c[w] *= inv;   // (two small factors can vanish together)
        rare |= c[w] == 0.f && s_m[w0 + w][rr] != -INFINITY;
      }
    }
    if (a.lse && lane < kMine && my_row < t.rows) a.lse[base + my_place] = lse;
    const unsigned rares = __ballot_sync(0xffffffffu, (rare || cleaned) && lane < kMine && my_row < used);
    for (int i0 = 0; i0 < kMine; i0 += kAhead) {
      if (wr * 16 + i0 * WK + wk >= t.rows) break;
      if (i0 > 0) ask(i0, shared_x);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        const int i = i0 + u, r = wr * 16 + i * WK + wk, rr = i * WK + wk;
        const size_t orow = base + __shfl_sync(0xffffffffu, my_place, i);
        const float cs = __shfl_sync(0xffffffffu, c_s, i);
        float y[kVec];
#pragma unroll
        for (int e = 0; e < kVec; ++e) y[e] = cs != 0.f ? cs * shared_x[u][e] : 0.f;
#pragma unroll
        for (int w = 0; w < WK; ++w) {
          const float cw = __shfl_sync(0xffffffffu, c[w], i);
          if (cw == 0.f) continue;   // (a part without weight may hold anything)
          const float* from = acc + ((w0 + w) * 16 + rr) * D;
#pragma unroll
          for (int e = 0; e < kVec; e += 2) {
            const float2 v = *reinterpret_cast<const float2*>(from + ((lane * kVec + e) ^ ((rr & 7) << 3)));
            y[e] = fmaf(cw, v.x, y[e]);
            y[e + 1] = fmaf(cw, v.y, y[e + 1]);
          }
        }
        if (r < t.rows) {
          __nv_bfloat16* out = a.o + orow * D + lane * kVec;
#pragma unroll
          for (int e = 0; e < kVec; e += 2) *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(y[e], y[e + 1]);
        }
      }
    }
    // What is not finite counts, however small its weight: in parts whose weight vanished, and elements of seen nodes
    // that were cleaned away. Such rows are formed once more.
    for (unsigned left = rares; left; left &= left - 1) {
      const int i = __ffs(left) - 1, rr = i * WK + wk;
      const size_t orow = base + __shfl_sync(0xffffffffu, my_place, i);
      const float cs = __shfl_sync(0xffffffffu, c_s, i);
      const int nd = t.node0 + __shfl_sync(0xffffffffu, my_node, i);
      const uint64_t* wd = a.mask ? a.mask + ((size_t)t.b * a.N + nd) * a.W : nullptr;
      const int32_t* table = own_table(a, t);
      float cw[WK];
#pragma unroll
      for (int w = 0; w < WK; ++w) cw[w] = __shfl_sync(0xffffffffu, c[w], i);
#pragma unroll 1
      for (int d = lane; d < D; d += 32) {
        float y = 0.f;
        auto add = [&](float f, float z, bool seen) {
          if (f != 0.f) y = fmaf(f, z, y);
          else if (seen && !(fabsf(z) < INFINITY)) y += z;
        };
        if (joins) add(cs, __ldcg(a.dense_o + orow * D + d), __ldcg(a.dense_lse + orow) != -INFINITY);
#pragma unroll
        for (int w = 0; w < WK; ++w) add(cw[w], acc[((w0 + w) * 16 + rr) * D + (d ^ ((rr & 7) << 3))], s_m[w0 + w][rr] != -INFINITY);
        for (int j = 0; cleaned && j < n; ++j) {
          if (wd ? !(wd[j >> 6] >> (j & 63) & 1) : j > nd) continue;
          const int p = own + j, pg = __ldg(table + (p >> a.page_shift));
          if ((unsigned)pg < (unsigned)a.P)
            add(0.f, __bfloat162float(a.v_pages[((size_t)pg * a.page + (p & (a.page - 1))) * step + (size_t)t.hk * D + d]), true);
        }
        a.o[orow * D + d] = __float2bfloat16(y);
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.item_empty[k & 1]);
  }
  if (k == 0) wait_prerequisite();   // (left before the first item's results)
  if (!ok && lane == 0) atomicCAS(a.err, 0, kErrTimeout);
}

// Few query rows (up to 8): the products are turned round, S^T = K Q^T and O^T = V^T P^T: positions and channels are the 16
// rows of the matrix instructions and queries their 8 columns, half as many instructions, exponentials and accumulators as
// with 16 query rows of which 4 or 8 are used. An item's team is WK warps, which share a tile's positions, and one that
// loads; a block is as many teams as fit.
template <int D, int WK>
struct Few {
  // (of two warps, heads of 128: 256 forks by 5, 4 and 3 teams 95.5, 99.6, 99.9 us)
  static constexpr int kTeams = WK >= 4 ? 1 : D == 64 ? 8 : D == 128 ? 5 : 2;
  static constexpr int kBlocks = WK == 4 && D < 256 ? 2 : 1;   // an SM
  static constexpr int kThreads = 32 * kTeams * (WK + 1);
  static constexpr int kRows = 8, PW = WK == 1 ? 32 : 16, KT = PW * WK;   // positions of a warp and of a tile
  static constexpr int kTile = KT * D * 2, kQ = kRows * D * 2, kAcc = WK > 1 ? WK * kRows * D * 4 : 0;
  static constexpr int kFit = ((kBlocks == 2 ? 108 : 224) * 1024 / kTeams - 2 * kQ - kAcc) / (2 * kTile), NS = kFit > 4 ? 4 : kFit;
  static constexpr int kRing = 2 * kQ, kOut = kRing + NS * 2 * kTile, kTeam = kOut + kAcc, kSmem = kTeams * kTeam;
  static_assert(NS >= 2 && kTeam % 1024 == 0 && KT * 128 % 1024 == 0, "a tile is loaded while another is computed; swizzled tiles");
};
__device__ __forceinline__ uint32_t turned(uint32_t x) {   // an 8 x 8 matrix of 16-bit elements, a row's neighbours in a register
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

template <int D, int WK>
__global__ void __launch_bounds__(Few<D, WK>::kThreads, Few<D, WK>::kBlocks)
    fork_own_few_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk, const __grid_constant__ CUtensorMap mv, const __grid_constant__ OwnArgs a) {
  using C = Few<D, WK>;
  constexpr int KT = C::KT, PW = C::PW, NS = C::NS, kTeams = C::kTeams, kBlk = PW / 16;
  extern __shared__ __align__(1024) uint8_t dyn[];
  __shared__ OwnBars bars[kTeams];
  __shared__ float s_m[kTeams][WK][8], s_l[kTeams][WK][8];
  __shared__ int s_bad[kTeams];   // the last item in which V of a node was cleaned of something
  const int tid = threadIdx.x, warp = __shfl_sync(0xffffffffu, tid >> 5, 0), lane = tid & 31, team = warp % kTeams, wk = warp / kTeams;
  if (smem_u32(dyn) & 1023u) {   // the swizzled tiles rely on it
    if (tid == 0) atomicCAS(a.err, 0, kErrTimeout);
    return;
  }
  if (tid == 0) {
    for (int t = 0; t < kTeams; ++t) {
      bars[t].template init<NS>(WK);
      s_bad[t] = -1;
    }
    fence_mbar_init();
    prefetch_tmap(&mq);
    prefetch_tmap(&mk);
    prefetch_tmap(&mv);
  }
  __syncthreads();
  OwnBars& s = bars[team];
  uint8_t* sm = dyn + team * C::kTeam;
  const long long items = (long long)a.B * a.Hk * a.m_tiles, at0 = blockIdx.x + (long long)gridDim.x * team, stride = (long long)gridDim.x * kTeams;
  if (wk == WK) {
    load_items<D, C>(mq, mk, mv, a, s, sm, at0, stride, lane);
    return;
  }
  // this lane's places in the rows that ldmatrix reads: of Q, of K (positions as rows) and of V
  uint32_t q_off[2], k_off[4], v_off[4];
#pragma unroll
  for (int j = 0; j < 2; ++j) q_off[j] = unit_at(8, lane & 7, 4 * j + (lane >> 3));
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    k_off[j] = unit_at(KT, wk * PW + (lane & 15), 2 * j + (lane >> 4));
    v_off[j] = unit_at(KT, wk * PW + (lane & 7) + ((lane >> 4) << 3), 2 * j + ((lane >> 3) & 1));
  }
  const int q0 = 2 * (lane & 3);                       // this thread's two queries, and their nodes within an item
  const int node_of[2] = {q0 / a.heads, (q0 + 1) / a.heads};
  const int out_row = lane >> 2, out_node = out_row / a.heads;   // the query whose results it writes
  const size_t step = (size_t)a.Hk * D;                // elements of a position
  const uint32_t ring_at = smem_u32(sm) + C::kRing;
  float* acc = reinterpret_cast<float*>(sm + C::kOut);
  Ring<NS> ring;
  bool ok = true;
  int k = 0;
  for (long long at = at0; at < items; at += stride, ++k) {
    // (a warp whose wait ran out goes on without touching anything until its team meets, here or before the results)
    ok = warp_wait(&s.item_full[k & 1], (k >> 1) & 1, a.budget);
    if constexpr (WK > 1) ok = named_bar_and(1 + 2 * team, 32 * WK, ok);
    if (!ok) break;
    const Item t = s.item[k & 1];
    const int n = t.n, own = t.own, used = t.used;
    float o[D / 16][4], m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
#pragma unroll
    for (int d = 0; d < D / 16; ++d)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
    // how far a chain's node sees, or its mask
    int sees_to[2];
    const uint64_t* words[2];
    uint64_t word0[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int node = q0 + e < used ? t.node0 + node_of[e] : 0;
      sees_to[e] = own + min(node + 1, n);
      words[e] = a.mask ? a.mask + ((size_t)t.b * a.N + node) * a.W : nullptr;
      word0[e] = words[e] && q0 + e < used ? __ldg(words[e]) : 0;
    }
    uint32_t qf[D / 32][4];
    if (t.tiles > 0) {
#pragma unroll
      for (int kk = 0; kk < D / 32; ++kk) ldmatrix4(smem_u32(sm) + (k & 1) * C::kQ + (kk >> 1) * 1024 + q_off[kk & 1], qf[kk]);
    }
    bool bad = false;
    for (int tile = 0; tile < t.tiles; ++tile) {
      ok = ok && warp_wait(&s.full[ring.slot], ring.parity, a.budget);
      if (!ok) break;
      const uint32_t k_at = ring_at + ring.slot * 2 * C::kTile, v_at = k_at + C::kTile;
      const int first = tile * KT + wk * PW;              // this warp's positions
      const bool masked = first + PW > own;
      if (masked) {
        // V of positions that are not there must not meet a weight of 0, nor what is not finite of nodes that some do not see
        const int r0 = max(0, own - first);
        for (int x = lane; x < (PW - r0) * (D / 8); x += 32) {
          const int r = r0 + x / (D / 8);
          const uint32_t u_at = v_at + unit_at(KT, wk * PW + r, x % (D / 8));
          uint4 v = make_uint4(0, 0, 0, 0);
          if (first + r < own + n) {
            if (n == 1 && !a.mask) continue;            // (it sees itself)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(u_at) : "memory");
            if (!finite_only(v)) continue;
            bad = true;
          }
          asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(u_at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
        }
        __syncwarp();
      }
      float x[kBlk][4];
#pragma unroll
      for (int c = 0; c < kBlk; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) x[c][e] = 0.f;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
#pragma unroll
        for (int c = 0; c < kBlk; ++c) {
          uint32_t f[4];
          ldmatrix4(k_at + (kk >> 2) * KT * 128 + c * 16 * 128 + k_off[kk & 3], f);
          mma16816(x[c], f, qf[kk >> 1][2 * (kk & 1)], qf[kk >> 1][2 * (kk & 1) + 1]);
        }
      if (masked) {
#pragma unroll
        for (int c = 0; c < kBlk; ++c)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int e = i & 1, p = first + c * 16 + 8 * (i >> 1) + (lane >> 2), j = p - own;
            bool see = p < sees_to[e];
            if (a.mask) see = j < 0 || (j < n && (((j < 64 ? word0[e] : __ldg(words[e] + (j >> 6))) >> (j & 63)) & 1));
            if (!see) x[c][i] = -INFINITY;
          }
      }
      float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
      for (int e = 0; e < 2; ++e)
#pragma unroll
        for (int c = 0; c < kBlk; ++c) mx[e] = fmaxf(mx[e], fmaxf(x[c][e], x[c][e + 2]));
#pragma unroll
      for (int z = 4; z < 32; z <<= 1)
#pragma unroll
        for (int e = 0; e < 2; ++e) mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], z));
      if (__any_sync(0xffffffffu, mx[0] * a.sl2 > m[0] || mx[1] * a.sl2 > m[1])) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const float m_new = fmaxf(m[e], mx[e] * a.sl2), f = m[e] == m_new ? 1.f : ex2_approx(m[e] - m_new);
          l[e] *= f;
#pragma unroll
          for (int d = 0; d < D / 16; ++d) {
            o[d][e] *= f;
            o[d][e + 2] *= f;
          }
          m[e] = m_new;
        }
      }
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const float off = m[e] == -INFINITY ? 0.f : -m[e];
#pragma unroll
        for (int c = 0; c < kBlk; ++c)
#pragma unroll
          for (int i = e; i < 4; i += 2) x[c][i] = ex2_approx(fmaf(x[c][i], a.sl2, off));
#pragma unroll
        for (int c = 0; c < kBlk; ++c) l[e] += x[c][e] + x[c][e + 2];
      }
      uint32_t p[kBlk][2];
#pragma unroll
      for (int c = 0; c < kBlk; ++c) {
        p[c][0] = turned(pack_bf16x2(x[c][0], x[c][1]));
        p[c][1] = turned(pack_bf16x2(x[c][2], x[c][3]));
      }
#pragma unroll
      for (int d = 0; d < D / 16; ++d)
#pragma unroll
        for (int c = 0; c < kBlk; ++c) {
          uint32_t f[4];
          ldmatrix4_t(v_at + (d >> 2) * KT * 128 + c * 16 * 128 + v_off[d & 3], f);
          mma16816(o[d], f, p[c][0], p[c][1]);
        }
      if (masked) fence_async_smem();   // (what was cleaned is loaded over)
      __syncwarp();
      if (lane == 0) mbar_arrive(&s.empty[ring.slot]);
      ring.step(1);
    }
    if (k == 0) wait_prerequisite();   // (in every warp: this grid must not end before the ones it follows)
#pragma unroll
    for (int w = 4; w < 32; w <<= 1)
#pragma unroll
      for (int e = 0; e < 2; ++e) l[e] += __shfl_xor_sync(0xffffffffu, l[e], w);
    // ---------------------------------------------------------------------------------- results: a part of the channels a warp
    constexpr int kMine = D / 8 / WK;                    // blocks of 8 channels: wk, wk + WK, ..
    const size_t base = ((size_t)t.b * a.N + t.node0) * a.Hq + t.hk * a.G + t.h0;
    const bool joins = t.shared > 0 && !a.alone;
    float lse_s[2], z[2][kMine];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const bool takes = joins && q0 + e < used;
      const size_t orow = base + node_of[e] * (a.Hq - a.heads) + q0 + e;
      lse_s[e] = takes ? __ldcg(a.dense_lse + orow) : -INFINITY;
#pragma unroll
      for (int d = 0; d < kMine; ++d) z[e][d] = takes ? __ldcg(a.dense_o + orow * D + 8 * (d * WK + wk) + (lane >> 2)) : 0.f;
    }
    bool cleaned = __any_sync(0xffffffffu, bad);
    if constexpr (WK > 1) {
#pragma unroll
      for (int d = 0; d < D / 8; ++d)
        *reinterpret_cast<float2*>(acc + (wk * D + 8 * d + (lane >> 2)) * 8 + q0) = make_float2(o[d >> 1][2 * (d & 1)], o[d >> 1][2 * (d & 1) + 1]);
      if (lane < 4) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          s_m[team][wk][q0 + e] = m[e];
          s_l[team][wk][q0 + e] = l[e];
        }
      }
      if (cleaned && lane == 0) s_bad[team] = k;
      __syncwarp();
      ok = named_bar_and(2 + 2 * team, 32 * WK, ok);
      cleaned = s_bad[team] == k;
    }
    if (!ok) break;
    // the weights of the warps' parts and of the shared one
    float c[2][WK], c_s[2];
    uint32_t rare = 0, seen = 0;                         // bit 16 e + w: part w of query e saw something (16 e + 15: the shared one)
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      float top = m[e], sum = l[e];
      c[e][0] = 1.f;
      if constexpr (WK > 1) {
        top = -INFINITY;
        sum = 0.f;
#pragma unroll
        for (int w = 0; w < WK; ++w) top = fmaxf(top, s_m[team][w][q0 + e]);
#pragma unroll
        for (int w = 0; w < WK; ++w) {
          const float mw = s_m[team][w][q0 + e];
          c[e][w] = mw == top ? 1.f : ex2_approx(mw - top);
          sum += c[e][w] * s_l[team][w][q0 + e];
          if (mw != -INFINITY) seen |= 1u << (16 * e + w);
        }
      } else if (top != -INFINITY) {
        seen |= 1u << (16 * e);
      }
      if (lse_s[e] != -INFINITY) seen |= 0x8000u << (16 * e);
      const Factors f = factors(q0 + e < used, joins, top, sum, lse_s[e]);
      const float inv = f.sees ? f.own / (sum * f.total) : 0.f;
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        c[e][w] *= inv;
        if (f.sees && c[e][w] == 0.f) rare |= 1u << (16 * e + w);
      }
      c_s[e] = f.shared / f.total;
      if (c_s[e] == 0.f) rare |= 0x8000u << (16 * e);
      if (a.lse && wk == 0 && lane < 4 && q0 + e < t.rows) a.lse[base + node_of[e] * (a.Hq - a.heads) + q0 + e] = f.lse;
    }
    rare &= seen;                                        // what saw something and has no weight: it counts where it is not finite
    const size_t out_at = (base + out_node * (a.Hq - a.heads) + out_row) * D + 2 * (lane & 3);
#pragma unroll
    for (int i = 0; i < kMine; ++i) {
      const int d = i * WK + wk;
      float y[2] = {0.f, 0.f};
      auto add = [&](int e, int bit, float f, float part) {
        if (f != 0.f) y[e] = fmaf(f, part, y[e]);        // (without weight it may hold anything)
        else if ((rare >> (16 * e + bit) & 1) && !(fabsf(part) < INFINITY)) y[e] += part;
      };
#pragma unroll
      for (int w = 0; w < WK; ++w) {
        float2 part;
        if constexpr (WK > 1) part = *reinterpret_cast<const float2*>(acc + (w * D + 8 * d + (lane >> 2)) * 8 + q0);
        else part = make_float2(o[i >> 1][2 * (i & 1)], o[i >> 1][2 * (i & 1) + 1]);
        add(0, w, c[0][w], part.x);
        add(1, w, c[1][w], part.y);
      }
      add(0, 15, c_s[0], z[0][i]);
      add(1, 15, c_s[1], z[1][i]);
      const uint32_t u = turned(pack_bf16x2(y[0], y[1]));
      if (out_row < t.rows) *reinterpret_cast<uint32_t*>(a.o + out_at + 8 * d) = u;
    }
    // so do elements of seen nodes that were cleaned away
    if (cleaned && out_row < used) {
      const int nd = t.node0 + out_node;
      const uint64_t* wd = a.mask ? a.mask + ((size_t)t.b * a.N + nd) * a.W : nullptr;
      const int32_t* table = own_table(a, t);
#pragma unroll 1
      for (int d = 2 * wk; d < 2 * (D / 8); d += d & 1 ? 2 * WK - 1 : 1) {   // (this warp's blocks)
        __nv_bfloat16* out = a.o + out_at + 8 * (d >> 1) + (d & 1);
        float y = 0.f;
        for (int j = 0; j < n; ++j) {
          if (wd ? !(wd[j >> 6] >> (j & 63) & 1) : j > nd) continue;
          const int p = own + j, pg = __ldg(table + (p >> a.page_shift));
          if ((unsigned)pg >= (unsigned)a.P) continue;
          const float v = __bfloat162float(a.v_pages[((size_t)pg * a.page + (p & (a.page - 1))) * step + (size_t)t.hk * D + 8 * (d >> 1) + 2 * (lane & 3) + (d & 1)]);
          if (!(fabsf(v) < INFINITY)) y += v;
        }
        if (y != 0.f) *out = __float2bfloat16(__bfloat162float(*out) + y);   // (inf or nan)
      }
    }
    __syncwarp();
    if (lane == 0) mbar_arrive(&s.item_empty[k & 1]);
  }
  if (k == 0) wait_prerequisite();   // (left before the first item's results)
  if (!ok && lane == 0) atomicCAS(a.err, 0, kErrTimeout);
}

size_t dense_rows(const TreeAttnArgs& t) { return (size_t)t.B * t.N * t.Hq; }
float* dense_of(const TreeAttnArgs& t) { return reinterpret_cast<float*>(t.ws + parts_bytes(t.D)); }

template <int D, int kForm>
cudaError_t shared_part(const ForkAttnArgs& p, cudaStream_t s) {
  SharedArgs a{};
  a.B = p.T;
  a.first = p.first;
  a.shared = p.shared;
  a.rows = p.t.B;
  a.N_row = p.t.N;
  a.dense_o = dense_of(p.t);
  a.dense_lse = a.dense_o + dense_rows(p.t) * D;
  return launch<D, kForm>(p.t, a, s);
}

using OwnKernel = void (*)(const CUtensorMap, const CUtensorMap, const CUtensorMap, const OwnArgs);
template <class C, int D, OwnKernel kKernel, int kThreads, int kBlocks>
cudaError_t own_part(const ForkAttnArgs& p, bool alone, cudaStream_t s) {
  const TreeAttnArgs& t = p.t;
  OwnArgs a{};
  a.q = static_cast<const __nv_bfloat16*>(t.q);
  a.k_pages = static_cast<const __nv_bfloat16*>(t.k_pages);
  a.v_pages = static_cast<const __nv_bfloat16*>(t.v_pages);
  a.table = t.table; a.ctx = t.ctx; a.lengths = t.lengths; a.first = p.first; a.shared = p.shared; a.mask = t.mask;
  a.sl2 = t.scale * kLog2e;
  a.o = static_cast<__nv_bfloat16*>(t.o);
  a.lse = t.lse;
  a.dense_o = dense_of(t);
  a.dense_lse = a.dense_o + dense_rows(t) * D;
  a.B = t.B; a.N = t.N; a.Hq = t.Hq; a.Hk = t.Hk; a.G = t.Hq / t.Hk; a.W = (t.N + 63) / 64; a.P = t.P; a.page = t.page;
  a.page_shift = __builtin_ctz((unsigned)t.page);
  a.M = t.M; a.T = p.T;
  a.err = t.err;
  a.heads = std::min(a.G, C::kRows);
  a.splits = (a.G + C::kRows - 1) / C::kRows;
  a.npt = std::min(C::kRows / a.heads, t.N);
  a.m_tiles = (t.N + a.npt - 1) / a.npt * a.splits;
  a.alone = alone;
  a.budget = wait_budget_cycles();
  CUtensorMap mq, mk, mv;
  if (!make_map(&mq, t.q, D, t.Hq, t.N, t.B, a.heads, a.npt) ||
      !make_map(&mk, t.k_pages, D, t.Hk, t.page, t.P, 1, std::min(t.page, C::KT)) ||
      !make_map(&mv, t.v_pages, D, t.Hk, t.page, t.P, 1, std::min(t.page, C::KT)))
    return cudaErrorInvalidValue;
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(kKernel), C::kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)std::min((long long)t.B * t.Hk * a.m_tiles, (long long)kNumSMs * kBlocks));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = alone ? 0 : 1;   // (only behind the shared part's kernels: what others have written is read at once)
  const int slot = stage_timer_begin(s, kKernForkAttnOwn);
  e = cudaLaunchKernelEx(&cfg, kKernel, mq, mk, mv, a);
  stage_timer_end(slot, s);
  return e;
}

template <int D, int WK>
cudaError_t own_few(const ForkAttnArgs& p, bool alone, cudaStream_t s) {
  using C = Few<D, WK>;
  return own_part<C, D, fork_own_few_kernel<D, WK>, C::kThreads, C::kBlocks>(p, alone, s);
}
template <int D, int WR>
cudaError_t own_by_teams(const ForkAttnArgs& p, bool alone, cudaStream_t s) {
  return own_part<Own<D, WR>, D, fork_own_kernel<D, WR>, kOwnThreads, D == 256 ? 1 : 2>(p, alone, s);
}

// Few items: by four warps each, by eight where every item has an SM to itself (16 rows of 250, 1000 and 4000 positions of their
// own, 32 items: 24, 30 and 63 us by four, 26, 26 and 49 by eight; 3 forks of 448 positions 12.3 and 10.3).
template <int D>
cudaError_t own_of_few(const ForkAttnArgs& p, bool alone, cudaStream_t s) {
  if constexpr (D < 256)
    if ((long long)p.t.B * p.t.Hk <= kNumSMs) return own_few<D, 8>(p, alone, s);
  return own_few<D, 4>(p, alone, s);
}

template <int D>
cudaError_t both_parts(const ForkAttnArgs& p, cudaStream_t s) {
  const int G = p.t.Hq / p.t.Hk;
  // two M tiles an item where a group of the average size has more rows a key head than one holds
  const long long rows = ((long long)p.t.B + p.T - 1) / p.T * p.t.N * G;
  // Short rows, all of whose items are resident at once: each reads its shared positions itself, one kernel in the place of
  // three (us by three and by one, 3 rows, 12 items: of 250 positions 25 and 13, 500 26 and 15, 1000 26 and 17, 2000 28 and 23;
  // 64 rows, 256 items: 35 and 15, 35 and 17, 34 and 21, 35 and 31; D = 256, 3 rows: 22 and 15, 22 and 17, 22 and 23, 25 and 36;
  // of 16 query rows a key head, 12 items: 26 and 15, 26 and 17, 26 and 23, 28 and 36; of 64, 6 items: 28 and 19, 28 and 25, 30 and 38).
  // The table's width is all that the host knows of the lengths.
  const int r = p.t.N * G;
  const bool alone = r <= 64 && (long long)p.t.B * p.t.Hk <= kNumSMs * Few<D, 4>::kBlocks &&
                     (long long)p.t.M * p.t.page <= (D == 256 || r > 16 ? 512 : r > 8 ? 1024 : 2048);
  cudaError_t e;
  if (alone) e = cudaSuccess;
  else if constexpr (D == 256) e = shared_part<D, kSplit>(p, s);
  else e = rows > kM ? shared_part<D, kWide>(p, s) : shared_part<D, kNarrow>(p, s);
  if (e != cudaSuccess) return e;
  if (r <= 8) {
    // Few items end sooner when four warps share each, many when more of them are under way (us by four and by one or two,
    // all parts together, own parts of 64 and of 1000 positions; D = 128: 256 items 33 and 31, 55 and 61, 512 items 38 and 34,
    // 80 and 80, 2048 items 61 and 53, 192 and 198; D = 256: 256 items 37 and 34, 79 and 79, 2048 items 104 and 80, 352 and 343).
    const bool many = (long long)p.t.B * p.t.Hk >= 3 * kNumSMs;
    return many ? own_few<D, D == 64 ? 1 : 2>(p, false, s) : own_of_few<D>(p, alone, s);
  }
  return r <= 16 ? own_by_teams<D, 1>(p, alone, s) : r <= 32 ? own_by_teams<D, 2>(p, alone, s) : own_by_teams<D, 4>(p, alone, s);
}

}  // namespace

size_t fork_attn_workspace_bytes(int B, int N, int Hq, int D) {
  return parts_bytes(D) + (size_t)B * N * Hq * (D + 1) * sizeof(float);
}

cudaError_t launch_fork_attn(const ForkAttnArgs& a, cudaStream_t s) {
  return a.t.D == 64 ? both_parts<64>(a, s) : a.t.D == 128 ? both_parts<128>(a, s) : both_parts<256>(a, s);
}

}  // namespace gdr
