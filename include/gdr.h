/*
 * gdr.h -- C ABI of libgdr, the gated delta rule forward on GB300 (sm_103a).
 *
 * The operation (Kev-4B-LiteRT page "r15_kernel_test.py", function truth_f64; DEG page
 * "model.py", function delta_rule_reference): per row and value head h, with key head
 * hk = h / (Hv/Hk) (adjacent value heads share a key head, repeat_interleave order),
 *
 *   k^ = k / sqrt(sum k^2 + 1e-6),  q~ = q / sqrt(sum q^2 + 1e-6) * D^-0.5
 *   S = S0 (zeros if absent); for each token t:
 *     S = exp(g_t) S;  delta = beta_t (v_t - S^T k^);  S = S + k^ delta^T;  o_t = S^T q~
 *
 * Pads are data: a position with beta = g = 0 neither decays nor writes the state.
 *
 * Conventions shared by every call:
 *  - All array pointers are DEVICE pointers owned by the caller, row-major and contiguous,
 *    16-byte aligned. The library never allocates device memory; scratch memory, where a path
 *    needs it, is a caller-provided workspace.
 *  - D = Dk = Dv must be 128 (GDR_ERR_UNSUPPORTED otherwise). Hv must be a multiple of Hk.
 *  - q, k, v and o share one element type (gdr_dtype); g, beta and every state are float32.
 *  - Calls are asynchronous on `stream` (NULL = the legacy default stream). Host-side argument
 *    checks happen before anything is launched and return an error without touching the GPU.
 *    Errors found on the device (a fork index out of range, a wait that ran out) are recorded
 *    in a sticky device error word that gdr_sync_status() reads and clears.
 *  - No exception crosses the ABI; every call returns a gdr_status. gdr_last_error_message()
 *    gives a one-line reason for the last non-OK status returned on the calling host thread.
 */
#ifndef GDR_H
#define GDR_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  GDR_OK = 0,
  GDR_ERR_INVALID_ARG = 1,   /* null pointer, bad size, misalignment, workspace too small  */
  GDR_ERR_UNSUPPORTED = 2,   /* a size the kernels do not implement (D != 128)            */
  GDR_ERR_CUDA = 3,          /* a CUDA runtime call failed (launch, sync, encode)          */
  GDR_ERR_DEVICE_INDEX = 4,  /* an index, length or page read on the device was out of range */
  GDR_ERR_TIMEOUT = 5,       /* a kernel wait ran past its limit; the kernel stopped early */
  GDR_ERR_NO_PAGES = 6       /* a cache had fewer free pages than its rows needed          */
} gdr_status;

typedef enum { GDR_F32 = 0, GDR_BF16 = 1 } gdr_dtype;

/* Same type as cudaStream_t, declared here so that C callers need no CUDA header. */
typedef struct CUstream_st* gdr_stream_t;

/*
 * Workspace bytes gdr_chunk_fwd needs for these sizes (0 when the path needs none: float32, and
 * rows of one chunk, L <= 64, which the bfloat16 path finishes in a single kernel). For longer
 * rows the bfloat16 tensor-core path keeps per-chunk intermediates there (the factors M', N, Q',
 * P U of each 64-token chunk). Returns 0 for invalid sizes.
 */
size_t gdr_chunk_workspace_bytes(int B, int L, int Hk, int Hv, int D, gdr_dtype dt);

/*
 * Prefill: B rows of L tokens each, every row continuing its own initial state.
 * (Kev-4B-LiteRT "r15_kernel_test.py": kernel(q, k, v, g, beta, initial_state,
 *  output_final_state=True, use_qk_l2norm_in_kernel=True) -> (o, S_T);
 *  DEG "model.py", _delta_rule.)
 *   q, k   [B, L, Hk, D]  dt          raw (not yet normalised) queries and keys
 *   v      [B, L, Hv, D]  dt
 *   g      [B, L, Hv]     float32     natural-log decay per token and value head (<= 0)
 *   beta   [B, L, Hv]     float32     write strength
 *   S0     [B, Hv, D, D]  float32     initial state, S[i][j] = key i, value j; NULL = zeros
 *   o      [B, L, Hv, D]  dt          output, every position (pads included)
 *   S_T    [B, Hv, D, D]  float32     final state; NULL = not written. May alias S0.
 *   ws     workspace of at least gdr_chunk_workspace_bytes(...) bytes (may be NULL if that is 0)
 * L need not be a multiple of 64; nothing is written beyond position L-1.
 */
gdr_status gdr_chunk_fwd(const void* q, const void* k, const void* v, const float* g,
                         const float* beta, const float* S0, void* o, float* S_T, int B, int L,
                         int Hk, int Hv, int D, gdr_dtype dt, void* ws, size_t ws_bytes,
                         gdr_stream_t stream);

/*
 * Prefill of B right-padded rows of different lengths (DEG "model.py": Backbone.forward over a batch
 * whose State.lengths give each row's real tokens; _dn_gates makes the padding exact no-ops).
 * Same arguments, layouts, workspace and results as gdr_chunk_fwd, plus
 *   lengths [B] int32 (device)   valid tokens of each row, in [0, L]
 * Row b runs only its first lengths[b] tokens: positions at or past lengths[b] are pads whatever
 * their g and beta hold, the 64-token chunks wholly past it are skipped (no work), o is not written
 * there (it keeps what the caller left), and S_T[b] is the state after the row's last valid token
 * (S0[b] when the length is 0). A length outside [0, L] leaves that row's o and S_T untouched and
 * records GDR_ERR_DEVICE_INDEX in the device error word.
 */
gdr_status gdr_chunk_fwd_varlen(const void* q, const void* k, const void* v, const float* g,
                                const float* beta, const float* S0, const int32_t* lengths, void* o,
                                float* S_T, int B, int L, int Hk, int Hv, int D, gdr_dtype dt, void* ws,
                                size_t ws_bytes, gdr_stream_t stream);

/*
 * Prefill followed by the layer's gated RMSNorm, fused into the output of the recurrence (DEG
 * "model.py": _linear_layer applies _gated_rms with the in_proj_z gate to _delta_rule's output). Same
 * arguments, workspace and final state as gdr_chunk_fwd, but instead of o it writes
 *   out[b, t, h, :] = w * o / sqrt(mean(o^2) + eps) * silu(z[b, t, h, :]),  silu(x) = x / (1 + exp(-x))
 * over the 128 values of each position and value head, from the float32 o (o itself is not stored):
 *   z    [B, L, Hv, D] bfloat16   the gate; 16-byte aligned
 *   w    [D] float32              the norm weight; 16-byte aligned
 *   eps  >= 0
 *   out  [B, L, Hv, D] bfloat16   must not overlap z
 * bfloat16 only (GDR_ERR_UNSUPPORTED for float32). Rows of several chunks reduce over the four
 * column blocks of a head in the state kernel (a cluster of four CTAs); rows of one chunk (L <= 64)
 * run gdr_gated_rmsnorm over the bf16 o in place.
 */
gdr_status gdr_chunk_fwd_gated(const void* q, const void* k, const void* v, const float* g,
                               const float* beta, const float* S0, const void* z, const float* w, float eps,
                               void* out, float* S_T, int B, int L, int Hk, int Hv, int D, gdr_dtype dt, void* ws,
                               size_t ws_bytes, gdr_stream_t stream);

/* Bytes of caller workspace gdr_fork_fwd needs for these sizes (0 for float32, and 0 for
 * single-chunk forks, L_pad <= 64, which the tensor-core path finishes in one kernel). */
size_t gdr_fork_workspace_bytes(int F, int L_pad, int Hk, int Hv, int D, gdr_dtype dt);

/*
 * Fork batch: F forks, fork f continuing its own copy of trunk[trunk_idx[f]] over its L_pad
 * tokens (right-padded with beta = g = 0). The trunk states are read in place, never copied.
 * bf16 forks run on the same tensor-core kernels as gdr_chunk_fwd (one row per fork, the row's
 * initial state taken from the trunk by index), so fork f equals gdr_chunk_fwd on that row from
 * trunk[trunk_idx[f]] bit for bit; float32 forks run the token loop.
 * (DEG "model.py": fork_delta_rule(q, k, v, g, beta, h0, h0_idx, store) in _fork_linear_layer;
 *  Backbone.fork reads the prefixes by reference through the row index prow.)
 *   q, k        [F, L_pad, Hk, D] dt;  v [F, L_pad, Hv, D] dt;  g, beta [F, L_pad, Hv] float32
 *   trunk       [N, Hv, D, D] float32   shared prefix states
 *   trunk_idx   [F] int64 (device)      fork f starts from trunk[trunk_idx[f]]
 *   o           [F, L_pad, Hv, D] dt
 *   states_out  [F, Hv, D, D] float32   each fork's final state (the `store` of the pages);
 *                                       NULL = not kept. Must not overlap trunk.
 *   ws          workspace of at least gdr_fork_workspace_bytes(...) bytes (NULL if that is 0),
 *               owned by the caller and free for reuse once the call's stream work is done
 * An index outside [0, N) leaves that fork's outputs untouched and records
 * GDR_ERR_DEVICE_INDEX in the device error word.
 */
gdr_status gdr_fork_fwd(const void* q, const void* k, const void* v, const float* g,
                        const float* beta, const float* trunk, const int64_t* trunk_idx, int N,
                        void* o, float* states_out, int F, int L_pad, int Hk, int Hv, int D,
                        gdr_dtype dt, void* ws, size_t ws_bytes, gdr_stream_t stream);

/*
 * One decode step (L = 1) for F rows, each row's state updated in place.
 * (DEG "model.py": DecodeGraph.step -> fork_forward(keep=True, decode=True); an idle row has
 *  lens 0, hence beta = g = 0, and its state stays bit-identical.)
 *   q, k [F, 1, Hk, D] dt;  v [F, 1, Hv, D] dt;  g, beta [F, 1, Hv] float32
 *   states [F, Hv, D, D] float32, read and written in place;  o [F, 1, Hv, D] dt
 */
gdr_status gdr_decode_step(const void* q, const void* k, const void* v, const float* g,
                           const float* beta, float* states, void* o, int F, int Hk, int Hv,
                           int D, gdr_dtype dt, gdr_stream_t stream);

/*
 * Prefill without a caller workspace and without any device allocation. The pages have no
 * counterpart to this call; it is for callers that cannot allocate GPU memory: a host program
 * that owns the whole device memory budget (a serving process or engine that reserves the GPU at
 * start-up, or a plugin loaded into one), or a latency-critical loop where a cudaMalloc, which may
 * synchronise the device and can fail under memory pressure, is not allowed once running.
 *
 * Same arguments (minus ws and ws_bytes), computation, results and errors as gdr_chunk_fwd. The
 * scratch is a fixed array of GDR_NOALLOC_SCRATCH_BYTES in device memory, held by every GPU on which
 * the library's code is loaded until the process exits. Sizes whose workspace
 * (gdr_chunk_workspace_bytes) exceeds it are rejected with GDR_ERR_UNSUPPORTED and a message, before
 * any CUDA call; float32 q/k/v need no scratch.
 * The first call on a device looks up the scratch's device address (with that device current);
 * make that first call before any stream capture. The address belongs to the device's CUDA
 * context: after that context is destroyed (cudaDeviceReset) the next call looks it up again in
 * the new one, so that call too belongs before any capture.
 * Every call uses the same scratch, which keeps the previous call's contents (nothing in it needs
 * to start at zero: each call writes all the scratch it reads). Calls whose GPU work overlaps
 * (other streams, other host threads) race on the scratch: serialise them.
 */
#define GDR_NOALLOC_SCRATCH_BYTES ((size_t)64 * 1024 * 1024)
gdr_status gdr_chunk_fwd_noalloc(const void* q, const void* k, const void* v, const float* g,
                                 const float* beta, const float* S0, void* o, float* S_T, int B,
                                 int L, int Hk, int Hv, int D, gdr_dtype dt, gdr_stream_t stream);

/*
 * GDN prologue: from the layer's q|k|v projection to the path's inputs.
 * (DEG "model.py": _linear_layer with _conv_silu and _dn_gates.) Per row b, with
 * ext = [tail; mixed] along positions (K-1 carried inputs, then the L new ones) and
 * C = (2 Hk + Hv) D channels,
 *   y[t][c] = silu( sum_{j < K} conv_w[c][j] ext[t + j][c] ),  silu(x) = x / (1 + exp(-x))
 * split by channel into q (channels [0, Hk D)), k ([Hk D, 2 Hk D)) and v (the rest), and
 *   beta = sigmoid(b),  g = -exp(A_log[h]) softplus(a + dt_bias[h])   at valid positions t < len_b,
 *   beta = g = 0 at pads (positions >= len_b), so that pads are exact no-ops of the recurrence;
 *   new_tail[b][j] = ext[len_b + j] for j < K-1 (the inputs ending at the last valid token).
 * q, k and v are computed at every position, pads included (their values there do not matter).
 *   mixed    [B, L, C] bfloat16           the projection
 *   tail     [B, K-1, C] bfloat16         the previous call's carry; NULL = zeros (a new sequence)
 *   conv_w   [C, K] float32               depthwise causal weights; tap K-1 meets the current token
 *                                         (16-byte aligned, like mixed, tail, q, k, v and new_tail)
 *   a, b     [B, L, Hv] float32           decay and write-strength projections
 *   A_log, dt_bias [Hv] float32
 *   lengths  [B] int32 (device)           valid tokens per row, in [0, L]; NULL = L for every row.
 *                                         A length outside [0, L] leaves that row's g, beta and
 *                                         new_tail untouched and records GDR_ERR_DEVICE_INDEX.
 *   q, k     [B, L, Hk, D] bfloat16;  v [B, L, Hv, D] bfloat16
 *   g, beta  [B, L, Hv] float32
 *   new_tail [B, K-1, C] bfloat16         NULL = not written; must not overlap tail or mixed
 * K is the convolution width, 1 <= K <= 8 (the pages use 4); B <= 65535 and L <= 1048560
 * (GDR_ERR_UNSUPPORTED otherwise). Arithmetic is float32 from the
 * bfloat16 inputs, with one rounding of q, k, v to bfloat16.
 */
gdr_status gdr_prologue(const void* mixed, const void* tail, const float* conv_w, const float* a,
                        const float* b, const float* A_log, const float* dt_bias, const int32_t* lengths,
                        void* q, void* k, void* v, float* g, float* beta, void* new_tail, int B, int L,
                        int Hk, int Hv, int D, int K, gdr_stream_t stream);

/*
 * The GDN prologue fused into the bfloat16 prefill: gdr_prologue (K = 4, lengths NULL) followed by
 * gdr_chunk_fwd on its q, k, v, g and beta, without q, k, v, g and beta ever reaching memory
 * (DEG "model.py": _linear_layer, where _conv_silu and _dn_gates feed _delta_rule). The chunk
 * kernel forms each 64-token tile of q, k and v as the conv + SiLU of the projection rows (and the
 * carry) in gdr_prologue's own order of operations, one rounding to bfloat16, and each chunk's g and
 * beta from a and b the same way: for rows longer than one chunk (L > 64) o, S_T and new_tail equal
 * those of the two separate calls bit for bit; rows of one chunk take the two-kernel path (which
 * gdr_chunk_fwd replaces by one kernel), equal within the bf16 tolerance, new_tail bit for bit.
 *   mixed, tail, conv_w, a, b, A_log, dt_bias, new_tail   as for gdr_prologue (conv_w [C, 4]; tail
 *                                   NULL = zeros, new_tail NULL = not written)
 *   S0, o, S_T                      as for gdr_chunk_fwd with dt = GDR_BF16 (o [B, L, Hv, D] bf16)
 *   ws    workspace of at least gdr_chunk_fwd_prologue_workspace_bytes(...) bytes (never NULL,
 *         every L included), owned by the caller: the per-chunk factors
 * o and new_tail must overlap neither mixed, tail nor each other. K must be 4 and D 128
 * (GDR_ERR_UNSUPPORTED otherwise); B, Hv <= 65535. Every row has L valid tokens (for rows with their
 * own lengths, call gdr_prologue with lengths and then gdr_chunk_fwd_varlen).
 */
size_t gdr_chunk_fwd_prologue_workspace_bytes(int B, int L, int Hk, int Hv, int D, int K);
gdr_status gdr_chunk_fwd_prologue(const void* mixed, const void* tail, const float* conv_w, const float* a,
                                  const float* b, const float* A_log, const float* dt_bias, const float* S0,
                                  void* o, float* S_T, void* new_tail, int B, int L, int Hk, int Hv, int D,
                                  int K, void* ws, size_t ws_bytes, gdr_stream_t stream);

/*
 * Gated RMSNorm epilogue: per row of D values (a position and value head of the recurrence
 * output o [B, L, Hv, D], so rows = B L Hv), with the gate z of the same shape,
 *   out = w * (x / sqrt(mean(x^2) + eps)) * silu(z),   silu(z) = z / (1 + exp(-z))
 * (DEG "model.py": _gated_rms, applied to the output of _delta_rule with the in_proj_z gate.)
 *   x, z, out  [rows, D] bfloat16   out may be x or z itself, but may not partly overlap them
 *   w          [D] float32          the norm weight (16-byte aligned, like x, z and out)
 * D must be 128; eps >= 0; rows <= 2^34. Arithmetic is float32 from the bfloat16 inputs, one
 * rounding of out.
 */
gdr_status gdr_gated_rmsnorm(const void* x, const void* z, const float* w, float eps, void* out,
                             long long rows, int D, gdr_stream_t stream);

/*
 * Backward of gdr_chunk_fwd: the gradients of a loss with respect to every input, given its
 * gradients dO of the outputs o and dS_T of the final state. The pages train through the
 * recurrence (DEG "model.py", delta_rule_reference inside the training loss; Kev-4B-LiteRT
 * "r15_kernel_test.py", truth_f64) but print no backward; this is the plain reverse of the
 * forward stated at the top of this header, token by token:
 *   dq~ = S_t dO_t;  dS += q~ dO_t^T;  dk^ = dS delta;  ddelta = dS^T k^;  dbeta = ddelta . (v - kv);
 *   dv = beta ddelta;  dkv = -beta ddelta;  dS_a = dS + k^ dkv^T;  dk^ += S_a dkv;
 *   dg = <S_a, dS_a>;  dS = exp(g_t) dS_a
 * (S_a = exp(g_t) S_{t-1}, kv = S_a^T k^), from dS = dS_T at the last token; dS0 is the last dS;
 * dq and dk are taken back through the normalisations and summed over the value heads of a key
 * head. Pads are tokens like any other (their dv is 0 because beta = 0).
 *   q, k, v, g, beta, S0     as for gdr_chunk_fwd (S0 NULL = zeros)
 *   dO     [B, L, Hv, D]  dt        gradient of o
 *   dS_T   [B, Hv, D, D]  float32   gradient of the final state; NULL = zeros
 *   dq, dk [B, L, Hk, D]  float32;  dv [B, L, Hv, D] float32;  dg, dbeta [B, L, Hv] float32
 *   dS0    [B, Hv, D, D]  float32   gradient of S0; NULL = not written
 *   ws     workspace of at least gdr_backward_workspace_bytes(...) bytes (never NULL), owned by
 *          the caller: state checkpoints every 32 tokens, one 32-token segment of states per
 *          (row, value head, 16-column block), and the per-column-block partial sums
 * The outputs must not overlap the inputs or one another. Arithmetic is float32 throughout (the
 * states are recomputed from checkpoints by the forward's own float32 recurrence), and the sums
 * over column blocks and value heads run in a fixed order: the result is deterministic.
 * B <= 65535 and B L < 2^31 (GDR_ERR_UNSUPPORTED otherwise).
 */
size_t gdr_backward_workspace_bytes(int B, int L, int Hk, int Hv, int D);
gdr_status gdr_backward(const void* q, const void* k, const void* v, const float* g, const float* beta,
                        const float* S0, const void* dO, const float* dS_T, float* dq, float* dk,
                        float* dv, float* dg, float* dbeta, float* dS0, int B, int L, int Hk, int Hv,
                        int D, gdr_dtype dt, void* ws, size_t ws_bytes, gdr_stream_t stream);

/*
 * gdr_backward_chunked: the same gradients as gdr_backward for bf16 q, k, v, dO, computed chunk by
 * chunk on the tensor cores. The pages print no backward; this is the reverse of the chunked
 * forward (the chunk algebra of gdr_chunk_fwd, 64-token chunks): the sequential part is the
 * adjoint chain, the forward chain transposed,
 *   dS_c = Gamma_C dS_{c+1} + M'^T dS_{c+1} + Q'^T dO_c    (dS_NC = dS_T, dS0 = dS_0),
 * and the rest is local to each chunk once its entering state S_c and dS_{c+1} are known (the
 * gradients through Delta = U - W S, P, T = (I + A)^-1, the decays and the normalisations).
 * Arguments, shapes, ownership and the no-overlap rule as for gdr_backward; dt must be GDR_BF16
 * (GDR_ERR_UNSUPPORTED otherwise). ws holds at least gdr_backward_chunked_workspace_bytes(...)
 * bytes: the forward's per-chunk factors and the chunk-entry states and adjoints (fp16 with a power
 * of two per 32-column slice, 32 KiB per row, value head and chunk each). The products
 * take fp16 (bf16 for the raw q, k Gram products) operands with float32 accumulation, like the
 * bf16 forward, so the result matches the float64 backward to the bf16 path's tolerance, not
 * gdr_backward's float32 one; the sums run in a fixed order (deterministic).
 */
size_t gdr_backward_chunked_workspace_bytes(int B, int L, int Hk, int Hv, int D);
gdr_status gdr_backward_chunked(const void* q, const void* k, const void* v, const float* g, const float* beta,
                                const float* S0, const void* dO, const float* dS_T, float* dq, float* dk,
                                float* dv, float* dg, float* dbeta, float* dS0, int B, int L, int Hk, int Hv,
                                int D, gdr_dtype dt, void* ws, size_t ws_bytes, gdr_stream_t stream);

/*
 * The chunked backward without its recomputation, for callers that keep the forward's
 * intermediates instead of checkpointing (the DEG model recomputes them; both give the same
 * gradients). gdr_chunk_fwd_save is gdr_chunk_fwd for bf16 rows (o and S_T as gdr_chunk_fwd
 * computes them for rows longer than one chunk, bit for bit; rows of one chunk take the two-kernel
 * path, equal within the bf16 tolerance) that also leaves in `saved` what gdr_backward_chunked's
 * sequential forward passes would recompute: the per-chunk factors, the fp16 chunk-entry states
 * with their powers of two, and v's powers of two. gdr_backward_chunked_saved then runs only the
 * adjoint chain and the chunk-local gradients; its results equal gdr_backward_chunked's bit for bit.
 *   saved  at least gdr_backward_chunked_workspace_bytes(B, L, Hk, Hv, D) bytes, 16-byte aligned,
 *          owned by the caller, overlapping no input or output. Between the two calls it must stay
 *          untouched and the backward must be given the same q, k, v, g, beta and S0 (nothing
 *          checks this: other inputs give wrong gradients, not an error).
 * Arguments, sizes and checks otherwise as gdr_chunk_fwd (dt = GDR_BF16) and gdr_backward_chunked.
 */
gdr_status gdr_chunk_fwd_save(const void* q, const void* k, const void* v, const float* g, const float* beta,
                              const float* S0, void* o, float* S_T, int B, int L, int Hk, int Hv, int D,
                              gdr_dtype dt, void* saved, size_t saved_bytes, gdr_stream_t stream);
gdr_status gdr_backward_chunked_saved(const void* q, const void* k, const void* v, const float* g,
                                      const float* beta, const float* S0, const void* dO, const float* dS_T,
                                      float* dq, float* dk, float* dv, float* dg, float* dbeta, float* dS0, int B,
                                      int L, int Hk, int Hv, int D, gdr_dtype dt, void* saved, size_t saved_bytes,
                                      gdr_stream_t stream);

/*
 * ---------------------------------------------------------------------------------------------
 * Softmax-attention layers beside the gated delta rule layers: the operators of a decoding step
 * that drafts tokens, checks them and keeps what was accepted. Keys and values live in pages that
 * rows (sequences, forks) share:
 *   k_pages, v_pages [P, page, Hk, D] dt   one layer's pages (one layer of [layers, P, page, Hk, D])
 *   table [rows, M] int32                  row b's positions [m page, (m+1) page) live in page
 *                                          table[b][m]; negative (-1 as the calls write it) where the
 *                                          row holds none
 *   ctx   [rows] int32                     committed positions of each row
 * page is 16, 32, 64 or 128 and M page at most 2^31 - 256; D is 64, 128 or 256; Hq is a multiple of Hk
 * (query head h reads key head h / (Hq / Hk)). Drafted nodes 0 .. N-1 of row b (node 0 the last committed
 * token, whose keys are not in the cache yet; every node after its parent) take positions ctx[b] ..
 * ctx[b]+N-1 until the accepted ones are moved to the front; lengths [B] int32 (NULL = N) gives each row's
 * nodes. A length outside [0, N], a context that leaves the table, or a page outside [0, P) is
 * recorded as GDR_ERR_DEVICE_INDEX. No array that a call writes (workspace included) may overlap another
 * of its arrays; overlaps are refused (GDR_ERR_INVALID_ARG).
 * ---------------------------------------------------------------------------------------------
 */

/*
 * RMS norm of every query and key head and the rotation by position, in one pass:
 *   y = w x / sqrt(mean(x^2) + eps);  pair j < R/2 of y turned by the angle pos * inv_freq[j];
 *   elements R .. D-1 pass through.
 * Pairs are (j, j + R/2), or (2j, 2j + 1) with interleaved != 0.
 *   q [B, N, Hq, D], k [B, N, Hk, D] dt   token i of row b starts at (b N + i) *_tok elements, head h
 *                          *_head further (slices of one projection are read in place); strides
 *                          multiples of 16 bytes, of at most 2^22 elements
 *   q_w, k_w [D] float32   norm weights;  eps >= 0
 *   inv_freq [R/2] float64 radians per position;  pos [B, N] int32
 *   q_out [B, N, Hq, D], k_out [B, N, Hk, D] dt   contiguous; may not overlap q or k
 * R is a multiple of 16 in [0, D]. Arithmetic is float32 with one rounding of the outputs; angles are
 * formed modulo a turn in 64-bit integers (to within 2^-31 turn at any position, for |inv_freq| < 2^62; an
 * inv_freq that is larger, infinite or nan makes its pair nan).
 */
gdr_status gdr_qk_norm_rope(const void* q, const void* k, const float* q_w, const float* k_w,
                            const double* inv_freq, const int32_t* pos, float eps, int interleaved, void* q_out,
                            void* k_out, int B, int N, int Hq, int Hk, int D, int R, long long q_tok,
                            long long q_head, long long k_tok, long long k_head, gdr_dtype dt,
                            gdr_stream_t stream);

/*
 * The same, leaving keys and values in the cache: k normed and rotated, v [B, N, Hk, D] (strided like
 * k) as it is, at positions ctx[b] + i of row b for i < lengths[b] (all N if NULL). q_out is computed
 * for every i. A row whose length or context is out of range, or a position whose page is, writes
 * nothing to the pages.
 */
gdr_status gdr_qk_norm_rope_append(const void* q, const void* k, const void* v, const float* q_w,
                                   const float* k_w, const double* inv_freq, const int32_t* pos, float eps,
                                   int interleaved, void* q_out, void* k_pages, void* v_pages,
                                   const int32_t* table, const int32_t* ctx, const int32_t* lengths, int P,
                                   int page, int M, int B, int N, int Hq, int Hk, int D, int R, long long q_tok,
                                   long long q_head, long long k_tok, long long k_head, long long v_tok,
                                   long long v_head, gdr_dtype dt, gdr_stream_t stream);

/*
 * Gradient of gdr_qk_norm_rope: from dq_out, dk_out (contiguous, dt) the gradients dq, dk (contiguous,
 * float32) and dq_w, dk_w [D] float32, with dy = R^T dout and r = 1 / sqrt(mean(x^2) + eps):
 *   dx = r (w dy - x r^2 mean(w dy x)),  dw = sum over tokens and heads of dy x r.
 * ws holds at least gdr_qk_norm_rope_backward_workspace_bytes(D) bytes. The sums run in a fixed order.
 * Outputs and ws overlap nothing.
 */
size_t gdr_qk_norm_rope_backward_workspace_bytes(int D);
gdr_status gdr_qk_norm_rope_backward(const void* q, const void* k, const float* q_w, const float* k_w,
                                     const double* inv_freq, const int32_t* pos, const void* dq_out,
                                     const void* dk_out, float eps, int interleaved, float* dq, float* dk,
                                     float* dq_w, float* dk_w, int B, int N, int Hq, int Hk, int D, int R,
                                     long long q_tok, long long q_head, long long k_tok, long long k_head,
                                     gdr_dtype dt, void* ws, size_t ws_bytes, gdr_stream_t stream);

/*
 * Attention of each row's drafted nodes over its committed positions and the nodes they see:
 *   o[b][i][h] = sum_j p_j v_j,  p = softmax_j(scale q[b][i][h] . k_j),  lse[b][i][h] = log sum_j e^(scale q . k_j)
 *   q, o [B, N, Hq, D] bfloat16;  k_pages, v_pages, table, ctx, lengths as above (the nodes' own keys
 *   and values already in the pages, at ctx[b] + node)
 *   mask [B, N, W] uint64, W = ceil(N / 64): bit j % 64 of word j / 64 says that node i sees node j
 *        (nodes at or past the row's length are never seen); NULL: node i sees nodes 0 .. i (a chain;
 *        N = 1 is the plain decode step, ctx = 0 a prefill)
 *   lse [B, N, Hq] float32, or NULL;  scale > 0
 *   ws at least gdr_tree_attn_workspace_bytes(D) bytes (0 for a D that is not implemented)
 * A node that sees nothing, and every node at or past its row's length, gets o = 0 and lse = -inf.
 * Values of unseen positions do not matter, infinities and NaN included; those of seen nodes reach o however
 * small their weight. A row whose length or context
 * is out of range counts as having no nodes; a page out of range is read as zeros; both record
 * GDR_ERR_DEVICE_INDEX. bfloat16 only (dt other than GDR_BF16: GDR_ERR_UNSUPPORTED), Hq / Hk <= 128.
 * Scores, sums and accumulators are float32; the softmax weights are rounded to bfloat16 for their
 * product with v, o once at the end. The same call gives the same bits every time; where a row's sums are
 * cut follows from all rows' lengths, so a row beside other rows may round differently.
 */
size_t gdr_tree_attn_workspace_bytes(int D);
gdr_status gdr_tree_attn(const void* q, const void* k_pages, const void* v_pages, const int32_t* table,
                         const int32_t* ctx, const int32_t* lengths, const uint64_t* mask, float scale, void* o,
                         float* lse, int B, int N, int Hq, int Hk, int D, int P, int page, int M, gdr_dtype dt,
                         void* ws, size_t ws_bytes, gdr_stream_t stream);

/*
 * gdr_tree_attn for rows whose leading positions are the same, as forks of a trunk have them (gdr_cache_fork shares a
 * source's full pages): keys and values of the shared positions are read once for all rows of a group.
 *   first [T + 1] int32, rising in [0, B]: group t is the rows first[t] .. first[t + 1] - 1 (neighbours; a
 *        group may be empty, rows outside all groups share nothing)
 *   shared [T] int32: positions that the rows of group t share, a multiple of page, at most each row's ctx. They
 *        are read through the table of the group's first row; that of the others is not looked at there.
 * Everything else as for gdr_tree_attn, results too, but for roundings: shared and own positions are attended apart,
 * in float32, and joined by their lse.
 *   ws at least gdr_fork_attn_workspace_bytes(B, N, Hq, D) bytes (0 for sizes that are not implemented)
 * If first falls anywhere, no row is attended (o = 0, lse = -inf); a group whose numbers are out of range, or a row with
 * ctx below shared, counts as having no nodes. Both record GDR_ERR_DEVICE_INDEX. The same call gives the same bits; a row
 * beside other rows may round differently, as for gdr_tree_attn.
 * Few short rows are faster in a table no wider than they need, as M is all that the host knows of their lengths: with
 * B * Hk <= 304 (152 for heads of 256) and N * Hq / Hk <= 64 a call is one kernel where M * page is at most 2048 (1024 where
 * N * Hq / Hk > 8; 512 where it is > 16 and for heads of 256), else three, which take two and a half times as long.
 */
size_t gdr_fork_attn_workspace_bytes(int B, int N, int Hq, int D);
gdr_status gdr_fork_attn(const void* q, const void* k_pages, const void* v_pages, const int32_t* table,
                         const int32_t* ctx, const int32_t* lengths, const uint64_t* mask, const int32_t* first,
                         const int32_t* shared, float scale, void* o, float* lse, int B, int N, int Hq, int Hk, int D,
                         int P, int page, int M, int T, gdr_dtype dt, void* ws, size_t ws_bytes, gdr_stream_t stream);

/*
 * Verification of drafted tokens against the target's probabilities (speculative sampling over a
 * tree; a chain is the tree of one child each). Per row, from the root on: at node `cur` the
 * candidates are its children in index order. With (c, Z) = (0, 1) and rho = max(p[cur] - c q[cur], 0),
 * candidate i of token t is accepted (and becomes cur) if u[i] q[cur][t] Z < rho[t]; a refusal sets
 * c' = c + Z and Z' = sum max(p - c' q, 0), the normalised residual of the refused draft, unless that
 * sum is 0 (then the state stays). With q NULL the drafts are given rather than drawn: a candidate is
 * accepted if u[i] Z < rho[t], and a refusal takes p[t] out (rho[t] = 0, Z loses it). Where no
 * candidate is left, next_token is the smallest t whose running sum of rho passes u_next times the
 * total (the last t with rho > 0 if none does; p itself stands in for an empty rho; -1 for an empty p).
 *   tokens, parents [B, N] int32   node i > 0 has parent parents[i] in [0, i); node 0 is the root.
 *                                  A node with a parent or token out of range is no candidate
 *                                  (GDR_ERR_DEVICE_INDEX)
 *   lengths [B] int32              nodes of each row (not NULL), in [0, N]; 0: path -1, n_path 0, next_token -1;
 *                                  outside: the row's outputs untouched, GDR_ERR_DEVICE_INDEX
 *   p [B, N, V], q [B, N, V] or NULL, dt   target and draft probabilities at each node (entries that
 *                                  are not > 0 count as 0); q's row of a node is what its children
 *                                  were drawn from
 *   u [B, N], u_next [B] float32   uniform numbers in [0, 1)
 *   path [B, N] int32              accepted nodes, the root first, then -1
 *   n_path, next_token [B] int32
 * Sums are carried to about 2^-46. N <= 1024, V < 2^30.
 */
gdr_status gdr_verify_draft(const int32_t* tokens, const int32_t* parents, const int32_t* lengths, const void* p,
                            const void* q, const float* u, const float* u_next, int32_t* path, int32_t* n_path,
                            int32_t* next_token, int B, int N, int V, gdr_dtype dt, gdr_stream_t stream);

/*
 * Pages. refs [P] int32 counts the rows that hold each page; a page is free when its count is 0, and
 * pages are handed out lowest first to the listed rows in order, so results do not depend on timing.
 * k_cache, v_cache [layers, P, page, row_bytes] hold every layer's entries, row_bytes the bytes of one
 * position (Hk D times the element size; a multiple of 16). ws holds at least
 * gdr_cache_workspace_bytes(F, M) bytes (F listed rows). Row lists are int32 [F].
 *
 * gdr_cache_reserve: rows[f] gets pages so that its ctx + extra positions fit.
 * gdr_cache_fork: row dst[f] gives back what it holds and becomes a copy of row src[f]: the full pages
 *   of src's ctx positions are shared, the partly filled last one is copied (its valid positions) to a
 *   new page.
 * gdr_cache_free: rows[f] gives back its pages (table -1, ctx 0).
 * gdr_cache_compact: the entries at ctx + path[b][i] move to ctx + i for i < n_path[b] in every layer
 *   (path rising, as gdr_verify_draft leaves it), and new_ctx[b] = ctx[b] + n_path[b]. new_ctx may
 *   not overlap ctx.
 * A row is refused, untouched, with GDR_ERR_DEVICE_INDEX, if its index is out of range, an earlier
 * entry lists it too, a fork's source is itself listed as dst, its context (a fork's source's; free does
 * not look at it) or any page that it or its source's context holds is out of range (reserve: or it has
 * fewer pages than its context needs, or one behind an empty entry), or its path does not rise
 * inside the table. Where pages run out (GDR_ERR_NO_PAGES) a row to be reserved stays as it was and a row
 * to be forked is left empty.
 */
size_t gdr_cache_workspace_bytes(int F, int M);
gdr_status gdr_cache_reserve(int32_t* table, const int32_t* ctx, int32_t* refs, const int32_t* rows, int extra,
                             int F, int R, int M, int P, int page, void* ws, size_t ws_bytes,
                             gdr_stream_t stream);
gdr_status gdr_cache_fork(void* k_cache, void* v_cache, int32_t* table, int32_t* ctx, int32_t* refs,
                          const int32_t* src, const int32_t* dst, int F, int R, int M, int layers, int P, int page,
                          long long row_bytes, void* ws, size_t ws_bytes, gdr_stream_t stream);
gdr_status gdr_cache_free(int32_t* table, int32_t* ctx, int32_t* refs, const int32_t* rows, int F, int R, int M,
                          int P, gdr_stream_t stream);
gdr_status gdr_cache_compact(void* k_cache, void* v_cache, const int32_t* table, const int32_t* ctx,
                             const int32_t* path, const int32_t* n_path, int32_t* new_ctx, int B, int W, int M,
                             int layers, int P, int page, long long row_bytes, gdr_stream_t stream);

/*
 * Tokens drawn from logits, and the probabilities that the filters leave (what gdr_verify_draft takes as p and
 * q). Per row, with w_i = e^((l_i - max l) / temperature) and tokens in the order of falling logits (equal ones
 * by rising index):
 *   top_k   keeps the first top_k of them (0: all);
 *   top_p   of these the tokens with less than top_p times their mass before them, at least the first (1: all);
 *   min_p   of these the tokens with w_i >= min_p (0: all).
 * The token is the smallest index whose running sum (in index order) of the kept w passes u times their total;
 * probabilities are w_i / total, 0 for tokens that are not kept. temperature 0 keeps the largest logit alone
 * (the first by index).
 *   logits [R, V] dt      row r starts at r * stride elements (any alignment of an element)
 *   temperature [R] float32, >= 0 (but for 0, below 1.5e-30 and above 1e36 it counts as that)
 *   top_k [R] int32, >= 0;  top_p, min_p [R] float32 in [0, 1]   NULL for no such filter
 *   u [R] float32         uniform numbers in [0, 1) (larger ones count as 1: the last kept token); with token
 *   token [R] int32, probs [R, V] float32   either may be NULL, not both
 * A logit that is -inf or nan is never kept; logits of +inf share all the weight. A row without any other logit
 * gets token -1 and probabilities 0. A row whose temperature, top_k, top_p or min_p is out of range keeps its
 * outputs untouched and records GDR_ERR_DEVICE_INDEX. Weights are formed to about 2^-38 of their size and summed in
 * units of 2^-40 of the largest (a weight below half a unit is not drawn). The same call gives the same bits; a bfloat16
 * row has them in any call, a float32 row beside other rows may be off by the sums' last units (2^-37). V <= 2^18, less 8 where rows do not
 * begin on 16 bytes; R <= 2^24.
 */
gdr_status gdr_sample(const void* logits, long long stride, const float* temperature, const float* u,
                      const int32_t* top_k, const float* top_p, const float* min_p, int32_t* token, float* probs,
                      int R, int V, gdr_dtype dt, gdr_stream_t stream);

/*
 * What stands between two blocks of a layer, in one pass over each token's C channels: the norm after the one
 * block, its gate and residual scale, the sum into the residual, and the norm before the other:
 *   z = post_w y / sqrt(mean(y^2) + eps),   x = h + scale sigmoid(gate) z,
 *   h_out = x,   n_out = pre_w x / sqrt(mean(x^2) + eps)
 *   h [rows, C] dt            the residual;  y, gate [rows, C] dt  the block's output and its gate, rows y_row and
 *                             gate_row elements apart (multiples of 16 bytes; slices of one projection)
 *   post_w, gate, scale       NULL: z = y, no gate (1), no scale (1)
 *   post_w, scale, pre_w [C] float32;  eps >= 0
 *   h_out, n_out [rows, C] dt   h_out may be h itself; otherwise outputs overlap nothing
 * C is a multiple of 8, at most 16384. Arithmetic is float32 with one rounding of each output (the second norm
 * is of the unrounded sum).
 */
gdr_status gdr_block_norm(const void* h, const void* y, const void* gate, const float* post_w, const float* scale,
                          const float* pre_w, float eps, void* h_out, void* n_out, long long rows, int C,
                          long long y_row, long long gate_row, gdr_dtype dt, gdr_stream_t stream);

/*
 * Gradient of gdr_block_norm, from dh_out [rows, C] float32 (NULL: zeros), the gradient of the residual that the
 * layers behind it left, and dn [rows, C] dt: with s = 1 / sqrt(mean(x^2) + eps), r = 1 / sqrt(mean(y^2) + eps), g = sigmoid(gate),
 *   dx = dh_out + s (pre_w dn - x s^2 mean(pre_w dn x)),   dh = dx,   dz = dx scale g,
 *   dy = r (post_w dz - y r^2 mean(post_w dz y)) (dz without post_w),   dgate = dx scale z g (1 - g),
 *   dpre_w = sum dn x s,   dpost_w = sum dz y r,   dscale = sum dx g z   (over the rows)
 *   dh [rows, C] float32 (the residual's gradient is summed over the layers);  dy, dgate [rows, C] dt
 *   dpre_w, dpost_w, dscale [C] float32;  dgate, dpost_w, dscale non-NULL exactly where gate, post_w, scale are
 *   ws at least gdr_block_norm_backward_workspace_bytes(C) bytes (0 for a C that is not implemented)
 * The inputs are the forward's (h as it was before). dh may be dh_out itself; otherwise outputs and ws overlap nothing.
 * The sums run in a fixed order: the same bits every time.
 */
size_t gdr_block_norm_backward_workspace_bytes(int C);
gdr_status gdr_block_norm_backward(const void* h, const void* y, const void* gate, const float* post_w,
                                   const float* scale, const float* pre_w, const float* dh_out, const void* dn,
                                   float eps, float* dh, void* dy, void* dgate, float* dpre_w, float* dpost_w,
                                   float* dscale, long long rows, int C, long long y_row, long long gate_row,
                                   gdr_dtype dt, void* ws, size_t ws_bytes, gdr_stream_t stream);

/* Synchronise `stream`, then read and clear the sticky device error word of the current device. */
gdr_status gdr_sync_status(gdr_stream_t stream);

/*
 * Testing aid (failure detection): the SM clock cycles a kernel wait may take before the kernel
 * gives up, records GDR_ERR_TIMEOUT in the device error word, waits (again bounded) for its own
 * copies and products still in flight, frees its tensor memory and exits. Default about 2e9
 * cycles (roughly 1 s); 0 makes every wait that is not already satisfied give up at once; a
 * negative value restores the default. Applies to launches made after the call; results of a call
 * that timed out are undefined, and the next call runs normally.
 */
gdr_status gdr_debug_set_wait_budget(long long cycles);

/* Static strings; never NULL. */
const char* gdr_status_string(gdr_status status);
const char* gdr_last_error_message(void);

/*
 * Stage timer (measurement aid). When enabled, every kernel the library launches is bracketed
 * by a pair of CUDA events recorded on its launch stream (up to `capacity` launches).
 * gdr_stage_timer_collect() synchronises those events and, for each kernel id k < max_ids,
 * writes the summed milliseconds to total_ms[k] and the launch count to launches[k], then
 * clears the record. gdr_kernel_name(k) names kernel id k (NULL past the last id).
 */
gdr_status gdr_stage_timer_enable(int on, int capacity);
gdr_status gdr_stage_timer_collect(double* total_ms, int* launches, int max_ids);
const char* gdr_kernel_name(int id);

#ifdef __cplusplus
}
#endif

#endif /* GDR_H */
