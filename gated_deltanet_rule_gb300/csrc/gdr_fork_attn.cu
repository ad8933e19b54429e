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
// else reads, so it is bound by reading them. A block of four warps takes up to 16, 32 or 64 query rows and the
// row's positions tile by tile (asynchronous copies, several tiles ahead); each warp multiplies 16 rows by 16 or
// 32 positions with warp-level matrix instructions, which a 128-row tcgen05 tile would fill to a sixteenth or
// less: starting and draining such an item takes 4 us of an SM, against 2 us for its reading. Warps that share rows
// take positions in turn and are joined at the end, in order; then the block joins the shared part's result.
//
// Weights are rounded to bfloat16 for their product with v, the sum adds them unrounded; scores, sums and parts are
// float32.
#include "gdr_attn_frame.cuh"

namespace gdr {
namespace {

constexpr int kOwnThreads = 128, kOwnWarps = 4;
constexpr int kOwnPages = 128;   // a row's first own pages, looked up ahead

struct OwnArgs {
  const __nv_bfloat16 *q, *k_pages, *v_pages;
  const int32_t *table, *ctx, *lengths, *first, *shared;
  const uint64_t* mask;
  float sl2;
  __nv_bfloat16* o;
  float* lse;
  const float *dense_o, *dense_lse;
  int B, N, Hq, Hk, G, W, P, page, page_shift, M, T;
  int* err;
};

// Query rows of a block (16 a warp, WR of the four warps), positions of a tile, and tiles on their way.
template <int D, int WR>
struct Own {
  static constexpr int WK = kOwnWarps / WR;                  // warps that share the positions of a tile
  static constexpr int KT = WK * 16 < 32 ? 32 : WK * 16;
  static constexpr int PW = KT / WK;                         // a warp's positions
  static constexpr int kRows = 16 * WR;
  static constexpr int kTile = KT * D * 2;                   // bytes of K or V
  static constexpr int NS = D == 256 && WR == 1 ? 2 : D == 64 ? 4 : 3;
  static constexpr int kQ = kRows * D * 2;
  static constexpr int kRing = kQ;
  static constexpr int kStages = NS * 2 * kTile;
  static constexpr int kOut = kOwnWarps * 16 * D * 4;        // accumulators, in the ring's place at the end
  static constexpr int kSmem = kRing + (kStages > kOut ? kStages : kOut);
};

// 16-byte unit ch of row r in rows of D bfloat16, swizzled so that eight rows' units lie in all banks.
template <int D>
__device__ __forceinline__ uint32_t unit_at(int r, int ch) { return (uint32_t)(r * (D * 2) + ((ch ^ (r & 7)) << 4)); }
__device__ __forceinline__ void ldmatrix4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix4_t(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
               : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3]) : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

template <int D, int WR>
__global__ void __launch_bounds__(kOwnThreads) fork_own_kernel(const __grid_constant__ OwnArgs a) {
  using C = Own<D, WR>;
  constexpr int KT = C::KT, PW = C::PW, NS = C::NS, WK = C::WK, kRows = C::kRows;
  extern __shared__ __align__(1024) uint8_t sm[];
  __shared__ int s_group, s_shared, s_bad, s_page[kOwnPages];
  __shared__ float s_m[kOwnWarps][16], s_l[kOwnWarps][16];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int b = blockIdx.x / a.Hk, hk = blockIdx.x - b * a.Hk, r0 = blockIdx.y * kRows;

  // the row's group and its numbers: everything asked for at once
  if (tid == 0) {
    s_group = -1;
    s_bad = 0;
  }
  int n = a.lengths ? __ldg(a.lengths + b) : a.N;
  const int ctx = __ldg(a.ctx + b);
  __syncthreads();
  bool falls = false;
  for (int t = tid; t < a.T; t += kOwnThreads) {
    const int f0 = __ldg(a.first + t), f1 = __ldg(a.first + t + 1), sh = __ldg(a.shared + t);
    falls |= f0 > f1;
    if (f0 <= b && b < f1) {
      s_group = group_valid(f0, f1, sh, a.B, a.page, a.M) ? t : -2;
      s_shared = sh;
    }
  }
  const bool any_falls = __syncthreads_or(falls);
  const int shared = s_group >= 0 ? s_shared : 0;
  const bool valid = !any_falls && s_group != -2 && n >= 0 && n <= a.N && ctx >= shared && (long long)ctx + n <= (long long)a.M * a.page;
  if (!valid) {
    if (tid == 0) atomicCAS(a.err, 0, kErrDeviceIndex);
    n = 0;
  }
  const int own = ctx - shared, rows = min(kRows, a.N * a.G - r0);
  const int used = min(rows, n * a.G - r0);      // rows of nodes that are there
  // position p >= 0 of the row's own part, a node from `own` on; a chain's block needs none past its last node
  const int L = used <= 0 ? 0 : own + (a.mask ? n : min(n, (r0 + used - 1) / a.G + 1));
  const int tiles = (L + KT - 1) / KT;
  const int32_t* table = a.table + (size_t)b * a.M + (shared >> a.page_shift);

  // ------------------------------------------------------------------------------------ loads
  const size_t step = (size_t)a.Hk * D;          // elements of a position
  auto lookup = [&](int m) {                     // page m of the own part (-1: read as zeros, and reported)
    const int pg = __ldg(table + m);
    if ((unsigned)pg < (unsigned)a.P) return pg;
    atomicCAS(a.err, 0, kErrDeviceIndex);
    return -1;
  };
  for (int m = tid; m < kOwnPages; m += kOwnThreads)
    if ((long long)m << a.page_shift < L) s_page[m] = lookup(m);
  constexpr int kChunks = D / 8, kLoads = KT * kChunks / kOwnThreads;   // 16-byte units of a position; a thread's of a tile
  const int ch = tid % kChunks, row0 = tid / kChunks;
  const size_t mine = (size_t)hk * D + ch * 8;
  auto load = [&](int tile) {
    uint8_t* to = sm + C::kRing + (tile % NS) * 2 * C::kTile;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      const int r = row0 + i * (kOwnThreads / kChunks), p = tile * KT + r, m = p >> a.page_shift;
      const int pg = p >= L ? -1 : m < kOwnPages ? s_page[m] : lookup(m);
      const size_t at = pg < 0 ? 0 : ((size_t)pg * a.page + (p & (a.page - 1))) * step + mine;
      const uint32_t bytes = pg < 0 ? 0u : 16u, off = unit_at<D>(r, ch);
      cp_async16_zfill(to + off, a.k_pages + at, bytes);
      cp_async16_zfill(to + C::kTile + off, a.v_pages + at, bytes);
    }
  };
  for (int x = tid; x < kRows * (D / 8); x += kOwnThreads) {
    const int r = x / (D / 8), ch = x % (D / 8), node = (r0 + r) / a.G, g = (r0 + r) - node * a.G;
    const bool there = r < used;
    const size_t at = there ? (((size_t)b * a.N + node) * a.Hq + hk * a.G + g) * D + ch * 8 : 0;
    cp_async16_zfill(sm + unit_at<D>(r, ch), a.q + at, there ? 16u : 0u);
  }
  __syncthreads();
#pragma unroll
  for (int s = 0; s < NS - 1; ++s) {
    if (s < tiles) load(s);
    cp_async_commit();
  }

  // ------------------------------------------------------------------------------------ tiles
  const int wr = warp / WK, wk = warp % WK;
  const uint32_t q_at = smem_u32(sm);
  uint32_t qf[D / 16][4];
  float o[D / 8][4];
#pragma unroll
  for (int d = 0; d < D / 8; ++d)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[d][e] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  // this thread's two rows: their nodes and first mask words
  int node[2];
  const uint64_t* words[2];
  uint64_t word0[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = wr * 16 + (lane >> 2) + 8 * h;
    node[h] = r < used ? (r0 + r) / a.G : 0;
    words[h] = a.mask ? a.mask + ((size_t)b * a.N + node[h]) * a.W : nullptr;
    word0[h] = words[h] && r < used ? __ldg(words[h]) : 0;
  }
  for (int tile = 0; tile < tiles; ++tile) {
    cp_async_wait<NS - 2>();
    __syncthreads();
    uint8_t* kt = sm + C::kRing + (tile % NS) * 2 * C::kTile;
    const bool masked = (tile + 1) * KT > own;
    if (masked) {   // V of nodes: what is not finite must not meet a weight of 0
      bool bad = false;
      for (int x = tid; x < KT * (D / 8); x += kOwnThreads) {
        const int r = x / (D / 8), p = tile * KT + r;
        if (p < own || p >= L) continue;
        uint4* v = reinterpret_cast<uint4*>(kt + C::kTile + unit_at<D>(r, x % (D / 8)));
        uint32_t* u = reinterpret_cast<uint32_t*>(v);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          if ((u[e] & 0x7F80u) == 0x7F80u) { u[e] &= 0xFFFF0000u; bad = true; }
          if ((u[e] & 0x7F800000u) == 0x7F800000u) { u[e] &= 0xFFFFu; bad = true; }
        }
      }
      if (bad) s_bad = 1;
      __syncthreads();
    }
    if (tile == 0) {
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk)
        ldmatrix4(q_at + unit_at<D>(wr * 16 + (lane & 15), kk * 2 + (lane >> 4)), qf[kk]);
    }
    if (tile + NS - 1 < tiles) load(tile + NS - 1);
    cp_async_commit();
    const uint32_t k_at = smem_u32(kt), v_at = k_at + C::kTile;
    float s[PW / 8][4];
#pragma unroll
    for (int c = 0; c < PW / 8; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) s[c][e] = 0.f;
#pragma unroll
    for (int kk = 0; kk < D / 16; ++kk) {
#pragma unroll
      for (int c = 0; c < PW / 16; ++c) {
        uint32_t f[4];
        ldmatrix4(k_at + unit_at<D>(wk * PW + c * 16 + (lane & 7) + ((lane >> 4) << 3), kk * 2 + ((lane >> 3) & 1)), f);
        mma16816(s[2 * c], qf[kk], f[0], f[1]);
        mma16816(s[2 * c + 1], qf[kk], f[2], f[3]);
      }
    }
    if (masked) {
#pragma unroll
      for (int c = 0; c < PW / 8; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int h = e >> 1, j = tile * KT + wk * PW + c * 8 + 2 * (lane & 3) + (e & 1) - own;
          bool see = j < 0;
          if (j >= 0 && j < n) {
            if (a.mask) see = ((j < 64 ? word0[h] : __ldg(words[h] + (j >> 6))) >> (j & 63)) & 1;
            else see = j <= node[h];
          }
          if (!see) s[c][e] = -INFINITY;
        }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float mx = -INFINITY;
#pragma unroll
      for (int c = 0; c < PW / 8; ++c) mx = fmaxf(mx, fmaxf(s[c][2 * h], s[c][2 * h + 1]));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
      mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2)) * a.sl2;
      if (__any_sync(0xffffffffu, mx > m[h])) {
        const float m_new = fmaxf(m[h], mx), f = m[h] == m_new ? 1.f : ex2_approx(m[h] - m_new);
        l[h] *= f;
#pragma unroll
        for (int d = 0; d < D / 8; ++d) {
          o[d][2 * h] *= f;
          o[d][2 * h + 1] *= f;
        }
        m[h] = m_new;
      }
      const float off = m[h] == -INFINITY ? 0.f : -m[h];
#pragma unroll
      for (int c = 0; c < PW / 8; ++c)
#pragma unroll
        for (int e = 2 * h; e < 2 * h + 2; ++e) {
          s[c][e] = ex2_approx(fmaf(s[c][e], a.sl2, off));
          l[h] += s[c][e];
        }
    }
#pragma unroll
    for (int c = 0; c < PW / 16; ++c) {
      const uint32_t p[4] = {pack_bf16x2(s[2 * c][0], s[2 * c][1]), pack_bf16x2(s[2 * c][2], s[2 * c][3]),
                             pack_bf16x2(s[2 * c + 1][0], s[2 * c + 1][1]), pack_bf16x2(s[2 * c + 1][2], s[2 * c + 1][3])};
#pragma unroll
      for (int d = 0; d < D / 16; ++d) {
        uint32_t f[4];
        ldmatrix4_t(v_at + unit_at<D>(wk * PW + c * 16 + (lane & 15), d * 2 + (lane >> 4)), f);
        mma16816(o[2 * d], p, f[0], f[1]);
        mma16816(o[2 * d + 1], p, f[2], f[3]);
      }
    }
  }

  // ------------------------------------------------------------------------------------ the warps' parts
  cp_async_wait<0>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
    l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    if ((lane & 3) == 0) {
      s_m[warp][(lane >> 2) + 8 * h] = m[h];
      s_l[warp][(lane >> 2) + 8 * h] = l[h];
    }
  }
  __syncthreads();   // (and the tiles have been read)
  float* acc = reinterpret_cast<float*>(sm + C::kRing);
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int d = 0; d < D / 8; ++d)
      *reinterpret_cast<float2*>(acc + (warp * 16 + (lane >> 2) + 8 * h) * D + d * 8 + 2 * (lane & 3)) =
          make_float2(o[d][2 * h], o[d][2 * h + 1]);
  wait_prerequisite();   // (in every block: this grid must not end before the ones it follows)
  __syncthreads();

  // ------------------------------------------------------------------------------------ results: a warp a row
  // (the shared part's results are asked for four rows at a time)
  constexpr int kVec = D / 32, kAhead = WR == 1 ? 2 : 4;
  const bool joins = shared > 0;
  for (int rb = warp; rb < rows; rb += kAhead * kOwnWarps) {
    float x[kAhead][kVec], lse_s[kAhead];
    auto orow_of = [&](int r) {
      const int nd = (r0 + r) / a.G, g = (r0 + r) - nd * a.G;
      return ((size_t)b * a.N + nd) * a.Hq + hk * a.G + g;
    };
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int r = rb + u * kOwnWarps;
      lse_s[u] = -INFINITY;
#pragma unroll
      for (int e = 0; e < kVec; ++e) x[u][e] = 0.f;
      if (r >= used || !joins) continue;
      const size_t orow = orow_of(r);
      lse_s[u] = __ldcg(a.dense_lse + orow);
#pragma unroll
      for (int e = 0; e < kVec; e += 2) {
        const float2 v = __ldcg(reinterpret_cast<const float2*>(a.dense_o + orow * D + lane * kVec + e));
        x[u][e] = v.x;
        x[u][e + 1] = v.y;
      }
    }
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      const int r = rb + u * kOwnWarps;
      if (r >= rows) break;
      const size_t orow = orow_of(r);
      float y[kVec], lse = -INFINITY;
#pragma unroll
      for (int e = 0; e < kVec; ++e) y[e] = 0.f;
      if (r < used) {
        const int w0 = (r >> 4) * WK, rr = r & 15;
        float top = s_m[w0][rr];
#pragma unroll
        for (int w = 1; w < WK; ++w) top = fmaxf(top, s_m[w0 + w][rr]);
        float sum = 0.f;
#pragma unroll
        for (int w = 0; w < WK; ++w) {
          const float mw = s_m[w0 + w][rr], f = mw == top ? 1.f : ex2_approx(mw - top);
          sum += f * s_l[w0 + w][rr];
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            const float z = acc[((w0 + w) * 16 + rr) * D + lane * kVec + e];
            if (f != 0.f) y[e] = fmaf(f, z, y[e]);
            else if (mw != -INFINITY && !(fabsf(z) < INFINITY)) y[e] += z;   // an infinity that was seen counts
          }
        }
        const bool sees = sum > 0.f || sum != sum;
        lse = sees ? top * (1.f / kLog2e) + logf(sum) : -INFINITY;
        const float inv = sees ? 1.f / sum : 0.f;
#pragma unroll
        for (int e = 0; e < kVec; ++e) y[e] = sees ? y[e] * inv : 0.f;
        if (s_bad) {   // elements that were cleaned away, of the nodes that this one sees
          const int nd = (r0 + r) / a.G;
          const uint64_t* wd = a.mask ? a.mask + ((size_t)b * a.N + nd) * a.W : nullptr;
          for (int j = 0; j < n; ++j) {
            if (wd ? !(wd[j >> 6] >> (j & 63) & 1) : j > nd) continue;
            const int p = own + j, pg = __ldg(table + (p >> a.page_shift));
            if ((unsigned)pg >= (unsigned)a.P) continue;
            const __nv_bfloat16* v = a.v_pages + ((size_t)pg * a.page + (p & (a.page - 1))) * step + (size_t)hk * D + lane * kVec;
            for (int e = 0; e < kVec; ++e) {
              const float z = __bfloat162float(v[e]);
              if (!(fabsf(z) < INFINITY)) y[e] += z;
            }
          }
        }
        if (joins) {
          const float ref = fmaxf(lse, lse_s[u]);
          float f[2] = {1.f, 0.f};   // the own part's weight, the shared part's
          if (lse != lse || lse_s[u] != lse_s[u]) {
            f[0] = f[1] = NAN;
          } else if (ref > -INFINITY) {
            f[0] = lse == ref ? 1.f : ex2_approx((lse - ref) * kLog2e);
            f[1] = lse_s[u] == ref ? 1.f : ex2_approx((lse_s[u] - ref) * kLog2e);
          }
          const float total = f[0] + f[1], inv2 = 1.f / total;
#pragma unroll
          for (int e = 0; e < kVec; ++e) {
            float z = f[0] != 0.f ? f[0] * y[e] : lse != -INFINITY && !(fabsf(y[e]) < INFINITY) ? y[e] : 0.f;
            if (f[1] != 0.f) z = fmaf(f[1], x[u][e], z);
            else if (lse_s[u] != -INFINITY && !(fabsf(x[u][e]) < INFINITY)) z += x[u][e];
            y[e] = z * inv2;
          }
          lse = ref == -INFINITY && total == total ? -INFINITY : ref + logf(total);
        }
      }
      __nv_bfloat16* out = a.o + orow * D + lane * kVec;
#pragma unroll
      for (int e = 0; e < kVec; e += 2) *reinterpret_cast<uint32_t*>(out + e) = pack_bf16x2(y[e], y[e + 1]);
      if (lane == 0 && a.lse) a.lse[orow] = lse;
    }
  }
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

template <int D, int WR>
cudaError_t own_part(const ForkAttnArgs& p, cudaStream_t s) {
  using C = Own<D, WR>;
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
  static std::atomic<uint64_t> done{0};
  cudaError_t e = allow_smem(reinterpret_cast<const void*>(fork_own_kernel<D, WR>), C::kSmem, done);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)t.B * t.Hk, (t.N * a.G + C::kRows - 1) / C::kRows);
  cfg.blockDim = dim3(kOwnThreads);
  cfg.dynamicSmemBytes = C::kSmem;
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  const int slot = stage_timer_begin(s, kKernForkAttnOwn);
  e = cudaLaunchKernelEx(&cfg, fork_own_kernel<D, WR>, a);
  stage_timer_end(slot, s);
  return e;
}

template <int D>
cudaError_t both_parts(const ForkAttnArgs& p, cudaStream_t s) {
  const int G = p.t.Hq / p.t.Hk;
  // two M tiles an item where a group of the average size has more rows a key head than one holds
  const long long rows = ((long long)p.t.B + p.T - 1) / p.T * p.t.N * G;
  cudaError_t e;
  if constexpr (D == 256) e = shared_part<D, kSplit>(p, s);
  else e = rows > kM ? shared_part<D, kWide>(p, s) : shared_part<D, kNarrow>(p, s);
  if (e != cudaSuccess) return e;
  const int r = p.t.N * G;
  return r <= 16 ? own_part<D, 1>(p, s) : r <= 32 ? own_part<D, 2>(p, s) : own_part<D, 4>(p, s);
}

}  // namespace

size_t fork_attn_workspace_bytes(int B, int N, int Hq, int D) {
  return parts_bytes(D) + (size_t)B * N * Hq * (D + 1) * sizeof(float);
}

cudaError_t launch_fork_attn(const ForkAttnArgs& a, cudaStream_t s) {
  return a.t.D == 64 ? both_parts<64>(a, s) : a.t.D == 128 ? both_parts<128>(a, s) : both_parts<256>(a, s);
}

}  // namespace gdr
