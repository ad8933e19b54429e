// Internal declarations of the attention-layer operators of a speculative step (not part of the
// ABI): q/k norm + rotation, tree attention over pages, draft verification, cache pages.
#pragma once

#include <atomic>
#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "gdr_backward.h"
#include "gdr_epilogue.h"
#include "gdr_internal.h"

namespace gdr {

// Stage-timer ids, after the existing kernels'.
constexpr int kKernQkNormRope = 9;
constexpr int kKernQkNormRopeBwd = 10;
constexpr int kKernTreeAttn = 11;
constexpr int kKernTreeAttnJoin = 12;
constexpr int kKernVerifyDraft = 13;
constexpr int kKernCacheAlloc = 14;
constexpr int kKernCacheCopy = 15;
constexpr int kKernBlockNorm = 16;
constexpr int kKernBlockNormBwd = 17;
constexpr int kKernSample = 18;
constexpr int kKernForkAttnShared = 19;
constexpr int kKernForkAttnOwn = 20;

constexpr int kNumSMs = 152;   // GB300
constexpr int kErrNoPages = 6;   // device error code (gdr_status): a cache had too few free pages

// RMS norm of every query and key head and the rotation by position. The three entry points share
// these arguments: dense outputs (k_out set), keys and values into pages (k_pages set), gradient
// (dq set; q_out, k_out unused).
struct RopeArgs {
  const void* q;
  const void* k;
  const void* v;
  const float* q_w;
  const float* k_w;
  const double* inv_freq;
  const int32_t* pos;
  float eps;
  int interleaved;
  void* q_out;
  void* k_out;
  long long q_tok, q_head, k_tok, k_head, v_tok, v_head;   // strides in elements
  int B, N, Hq, Hk, D, R;
  bool bf16;
  // pages
  void* k_pages;
  void* v_pages;
  const int32_t* table;
  const int32_t* ctx;
  const int32_t* lengths;
  int P, page, M;
  // gradient
  const void* dq_out;
  const void* dk_out;
  float* dq;
  float* dk;
  float* dq_w;
  float* dk_w;
  float* partial;
  int* err;
  // set by the launch: blocks of queries and of keys (values as keys), and tokens of each one's block
  int blocks[2], tokens[2];
};
cudaError_t launch_qk_norm_rope(RopeArgs a, cudaStream_t s);
cudaError_t launch_qk_norm_rope_backward(RopeArgs a, cudaStream_t s);
size_t qk_norm_rope_backward_workspace_bytes(int D);

// Attention of a tree or chain of drafted nodes over the cache's pages (bf16).
struct TreeAttnArgs {
  const void* q;             // [B, N, Hq, D]
  const void* k_pages;       // [P, page, Hk, D]
  const void* v_pages;
  const int32_t* table;      // [B, M]
  const int32_t* ctx;        // [B]
  const int32_t* lengths;    // [B] or NULL
  const uint64_t* mask;      // [B, N, W] or NULL (node i sees nodes <= i)
  float scale;
  void* o;                   // [B, N, Hq, D]
  float* lse;                // [B, N, Hq] or NULL
  int B, N, Hq, Hk, D, P, page, M;
  uint8_t* ws;
  int* err;
};
size_t tree_attn_workspace_bytes(int D);
cudaError_t launch_tree_attn(const TreeAttnArgs& a, cudaStream_t s);

// Attention of forked rows over the positions that groups of them share and over their own.
struct ForkAttnArgs {
  TreeAttnArgs t;            // (t.ws: parts, then dense results)
  const int32_t* first;      // [T + 1]
  const int32_t* shared;     // [T]
  int T;
};
size_t fork_attn_workspace_bytes(int B, int N, int Hq, int D);
cudaError_t launch_fork_attn(const ForkAttnArgs& a, cudaStream_t s);

// Verification of drafted tokens: one cluster of blocks per row walks the row's tree.
struct VerifyArgs {
  const int32_t* tokens;
  const int32_t* parents;
  const int32_t* lengths;
  const void* p;
  const void* q;        // NULL: given drafts
  const float* u;
  const float* u_next;
  int32_t* path;
  int32_t* n_path;
  int32_t* next_token;
  int B, N, V;
  bool bf16;
  int* err;
};
constexpr int kVerifyMaxNodes = 1024;   // nodes of a row whose scalars fit the kernel's shared memory
cudaError_t launch_verify_draft(const VerifyArgs& a, cudaStream_t s);

// Cache pages with reference counts (a page is free when its count is 0).
struct CacheArgs {
  uint8_t* k_cache;          // [layers, P, page, row_bytes]
  uint8_t* v_cache;
  int32_t* table;            // [rows, M]
  int32_t* ctx;              // [rows]
  int32_t* refs;             // [P]
  const int32_t* src;        // [F] (fork only)
  const int32_t* dst;        // [F]
  int layers, P, page, rows, M, F;
  int page_shift;            // log2(page)
  long long row_bytes;
  int extra;                 // reserve: positions past ctx that must have pages
  int32_t* ws;               // need [F], first [F], count; free list
  int* err;
};
size_t cache_workspace_bytes(int F, int M);
cudaError_t launch_cache_fork(const CacheArgs& a, cudaStream_t s);
cudaError_t launch_cache_reserve(const CacheArgs& a, cudaStream_t s);
cudaError_t launch_cache_free(const CacheArgs& a, cudaStream_t s);

struct CompactArgs {
  uint8_t* k_cache;
  uint8_t* v_cache;
  const int32_t* table;
  const int32_t* ctx;
  const int32_t* path;       // [B, W]
  const int32_t* n_path;     // [B]
  int32_t* new_ctx;          // [B]
  int layers, P, page, B, M, W;
  long long row_bytes;
  int* err;
};
constexpr int kCompactMaxPath = 2048;   // path entries whose slots fit the kernel's shared memory
cudaError_t launch_cache_compact(const CompactArgs& a, cudaStream_t s);

// Tokens drawn from filtered logits, and the probabilities that are left.
struct SampleArgs {
  const void* logits;        // [R, V], rows `stride` elements apart
  const float* temperature;  // [R]
  const float* u;            // [R] (with token)
  const int32_t* top_k;      // [R] or NULL
  const float* top_p;        // [R] or NULL
  const float* min_p;        // [R] or NULL
  int32_t* token;            // [R] or NULL
  float* probs;              // [R, V] or NULL
  int R, V;
  long long stride;
  bool bf16;
  int* err;
  int cluster;               // set by the launch: blocks of a row
};
constexpr int kSampleMaxV = 1 << 18;   // entries of a row that a cluster's shared memory holds
cudaError_t launch_sample(const SampleArgs& a, cudaStream_t s);

// The norms around a block with its gate and residual scale: x = h + scale sigmoid(gate) norm(y), norm(x).
struct BlockNormArgs {
  const void* h;             // [rows, C]
  const void* y;             // [rows, C], rows y_row elements apart
  const void* gate;          // [rows, C] or NULL, rows gate_row elements apart
  const float* post_w;       // [C] or NULL (y is not normed)
  const float* scale;        // [C] or NULL (ones)
  const float* pre_w;        // [C]
  float eps;
  void* h_out;
  void* n_out;
  long long rows, y_row, gate_row;
  int C;
  bool bf16;
  // gradient
  const float* dh_out;       // [rows, C] or NULL (zeros)
  const void* dn;
  float* dh;
  void* dy;
  void* dgate;               // (where there is a gate, a post norm, a scale)
  float* dpre_w;
  float* dpost_w;
  float* dscale;
  float* partial;
  int stages;                // set by the launch: rows on their way to a block
};
constexpr int kBlockNormMaxC = 16384;
size_t block_norm_backward_workspace_bytes(int C);
cudaError_t launch_block_norm(const BlockNormArgs& a, cudaStream_t s);
cudaError_t launch_block_norm_backward(const BlockNormArgs& a, cudaStream_t s);

// Lets a kernel use `bytes` of dynamic shared memory: set once on each device (`done`, a bit a device), as
// setting it costs a call 0.8 us.
inline cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);
  if (dev < 64 && (done.load(std::memory_order_relaxed) & bit)) return cudaSuccess;
  e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess && dev < 64) done.fetch_or(bit, std::memory_order_relaxed);
  return e;
}

}  // namespace gdr
