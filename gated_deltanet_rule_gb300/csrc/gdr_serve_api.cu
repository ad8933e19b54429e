// C ABI of the attention-layer operators: host-side argument checks (before any CUDA call) and dispatch.
#include <cuda_runtime.h>

#include <cstdarg>
#include <cstdio>
#include <initializer_list>

#include "gdr.h"
#include "gdr_serve.h"

using namespace gdr;

namespace {

gdr_status fail(gdr_status st, const char* fmt, ...) {
  char buf[512];
  va_list ap;
  va_start(ap, fmt);
  vsnprintf(buf, sizeof(buf), fmt, ap);
  va_end(ap);
  return static_cast<gdr_status>(record_error(st, buf));
}

gdr_status launched(cudaError_t e, const char* who) {
  if (e != cudaSuccess) return fail(GDR_ERR_CUDA, "%s: launch failed: %s", who, cudaGetErrorString(e));
  return static_cast<gdr_status>(record_error(GDR_OK, ""));
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Range {
  const void* p;
  unsigned long long bytes;
  const char* name;
};
bool overlap(const Range& a, const Range& b) {
  if (!a.p || !b.p) return false;
  const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
  return a0 < b0 + b.bytes && b0 < a0 + a.bytes;
}
// No output may overlap an input or another output.
gdr_status apart(std::initializer_list<Range> outs, std::initializer_list<Range> ins, const char* who) {
  for (const Range* o = outs.begin(); o != outs.end(); ++o) {
    for (const Range* p = o + 1; p != outs.end(); ++p)
      if (overlap(*o, *p)) return fail(GDR_ERR_INVALID_ARG, "%s: %s overlaps %s", who, o->name, p->name);
    for (const Range& in : ins)
      if (overlap(*o, in)) return fail(GDR_ERR_INVALID_ARG, "%s: %s overlaps %s", who, o->name, in.name);
  }
  return GDR_OK;
}

gdr_status check_heads(int B, int N, int Hq, int Hk, int D, gdr_dtype dt, const char* who) {
  if (B < 1 || N < 1 || Hq < 1 || Hk < 1)
    return fail(GDR_ERR_INVALID_ARG, "%s: sizes must be >= 1 (B=%d N=%d Hq=%d Hk=%d)", who, B, N, Hq, Hk);
  if (Hq % Hk != 0) return fail(GDR_ERR_INVALID_ARG, "%s: Hq=%d is not a multiple of Hk=%d", who, Hq, Hk);
  if (dt != GDR_F32 && dt != GDR_BF16) return fail(GDR_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dt);
  if (D != 64 && D != 128 && D != 256)
    return fail(GDR_ERR_UNSUPPORTED, "%s: head dimension D=%d is not implemented (64, 128 or 256)", who, D);
  if (Hq > 65535) return fail(GDR_ERR_UNSUPPORTED, "%s: Hq=%d exceeds 65535", who, Hq);
  if ((long long)B * N > (1ll << 24)) return fail(GDR_ERR_UNSUPPORTED, "%s: B*N=%lld exceeds 2^24", who, (long long)B * N);
  return GDR_OK;
}

gdr_status check_pages(int P, int page, int M, const char* who) {
  if (P < 1 || M < 1) return fail(GDR_ERR_INVALID_ARG, "%s: sizes must be >= 1 (P=%d M=%d)", who, P, M);
  if (page != 16 && page != 32 && page != 64 && page != 128)
    return fail(GDR_ERR_UNSUPPORTED, "%s: pages of %d positions are not implemented (16, 32, 64 or 128)", who, page);
  if ((long long)M * page > 0x7fffff00ll)   // (kernels count positions in whole tiles of up to 128)
    return fail(GDR_ERR_UNSUPPORTED, "%s: M*page=%lld positions exceed 2^31 - 256", who, (long long)M * page);
  return GDR_OK;
}

// What the three norm + rotation calls share; es is the element size.
gdr_status check_rope(const RopeArgs& a, gdr_dtype dt, const char* who) {
  if (!a.q || !a.k || !a.q_w || !a.k_w || !a.pos || (!a.inv_freq && a.R > 0))
    return fail(GDR_ERR_INVALID_ARG, "%s: q, k, q_w, k_w, inv_freq and pos must be non-NULL", who);
  gdr_status st = check_heads(a.B, a.N, a.Hq, a.Hk, a.D, dt, who);
  if (st != GDR_OK) return st;
  if (a.R < 0 || a.R > a.D || a.R % 16 != 0)
    return fail(GDR_ERR_INVALID_ARG, "%s: R=%d is not a multiple of 16 in [0, D]", who, a.R);
  if (!(a.eps >= 0.f)) return fail(GDR_ERR_INVALID_ARG, "%s: eps must be >= 0", who);
  const int es = dt == GDR_BF16 ? 2 : 4;
  const long long strides[] = {a.q_tok, a.q_head, a.k_tok, a.k_head, a.v_tok, a.v_head};
  for (long long s : strides)
    if (s < 0 || s * es % 16 != 0 || s > (1ll << 22))
      return fail(GDR_ERR_INVALID_ARG, "%s: strides must be multiples of 16 bytes, of at most 2^22 elements", who);
  if (a.Hq * a.q_head > (1ll << 30) || a.Hk * a.k_head > (1ll << 30) || a.Hk * a.v_head > (1ll << 30))
    return fail(GDR_ERR_UNSUPPORTED, "%s: a token's heads span more than 2^30 elements", who);
  for (const void* p : {a.q, a.k, a.v, (const void*)a.q_w, (const void*)a.k_w})
    if (p && !aligned(p, 16)) return fail(GDR_ERR_INVALID_ARG, "%s: q, k, v, q_w and k_w must be 16-byte aligned", who);
  if (!aligned(a.inv_freq, 8) || !aligned(a.pos, 4))
    return fail(GDR_ERR_INVALID_ARG, "%s: inv_freq must be 8-byte and pos 4-byte aligned", who);
  return GDR_OK;
}

// Bytes spanned by B N tokens of H heads at these strides.
unsigned long long span(const RopeArgs& a, int H, long long tok, long long head, int es) {
  return ((unsigned long long)((long long)a.B * a.N - 1) * tok + (unsigned long long)(H - 1) * head + a.D) * es;
}

// The same for the three norm + rotation calls, whose weights, frequencies and positions are inputs besides `ins`.
gdr_status apart_rope(const RopeArgs& a, std::initializer_list<Range> outs, std::initializer_list<Range> ins, const char* who) {
  const gdr_status st = apart(outs, ins, who);
  if (st != GDR_OK) return st;
  return apart(outs, {{a.q_w, a.D * 4ull, "q_w"}, {a.k_w, a.D * 4ull, "k_w"}, {a.inv_freq, a.R * 4ull, "inv_freq"},
                      {a.pos, (unsigned long long)a.B * a.N * 4, "pos"}}, who);
}

gdr_status check_cache(const void* k_cache, const void* v_cache, int layers, int P, int page, long long row_bytes,
                       const char* who) {
  if (!k_cache || !v_cache) return fail(GDR_ERR_INVALID_ARG, "%s: k_cache and v_cache must be non-NULL", who);
  if (!aligned(k_cache, 16) || !aligned(v_cache, 16))
    return fail(GDR_ERR_INVALID_ARG, "%s: k_cache and v_cache must be 16-byte aligned", who);
  if (layers < 1 || row_bytes < 16 || row_bytes % 16 != 0)
    return fail(GDR_ERR_INVALID_ARG, "%s: layers=%d must be >= 1 and row_bytes=%lld a multiple of 16", who, layers, row_bytes);
  if (layers > 16383 || row_bytes > (1ll << 30))
    return fail(GDR_ERR_UNSUPPORTED, "%s: layers=%d or row_bytes=%lld too large", who, layers, row_bytes);
  return GDR_OK;
}
unsigned long long cache_bytes(int layers, int P, int page, long long row_bytes) {
  return (unsigned long long)layers * P * page * row_bytes;
}

gdr_status check_rows(const void* table, const void* ctx, const void* refs, const void* rows, int F, int R, int M, int P,
                      const char* who) {
  if (!table || !ctx || !refs || !rows)
    return fail(GDR_ERR_INVALID_ARG, "%s: table, ctx, refs and the row list must be non-NULL", who);
  if (F < 1 || R < 1) return fail(GDR_ERR_INVALID_ARG, "%s: sizes must be >= 1 (F=%d rows=%d)", who, F, R);
  for (const void* p : {table, ctx, refs, rows})
    if (!aligned(p, 4)) return fail(GDR_ERR_INVALID_ARG, "%s: table, ctx, refs and row lists must be 4-byte aligned", who);
  if (M < 1 || P < 1) return fail(GDR_ERR_INVALID_ARG, "%s: sizes must be >= 1 (P=%d M=%d)", who, P, M);
  if ((long long)F * M > 0x3fffffffll || F > 1 << 20)
    return fail(GDR_ERR_UNSUPPORTED, "%s: F=%d rows of M=%d pages are too many", who, F, M);
  return GDR_OK;
}

gdr_status check_ws(const void* ws, size_t given, size_t need, const char* who) {
  if (!ws || given < need)
    return fail(GDR_ERR_INVALID_ARG, "%s: workspace of %zu bytes needed, %zu given", who, need, ws ? given : (size_t)0);
  if (!aligned(ws, 16)) return fail(GDR_ERR_INVALID_ARG, "%s: the workspace must be 16-byte aligned", who);
  return GDR_OK;
}

gdr_status no_device(const char* who) { return fail(GDR_ERR_CUDA, "%s: no CUDA device available", who); }

}  // namespace

extern "C" {

gdr_status gdr_qk_norm_rope(const void* q, const void* k, const float* q_w, const float* k_w,
                            const double* inv_freq, const int32_t* pos, float eps, int interleaved, void* q_out,
                            void* k_out, int B, int N, int Hq, int Hk, int D, int R, long long q_tok,
                            long long q_head, long long k_tok, long long k_head, gdr_dtype dt,
                            gdr_stream_t stream) {
  const char* who = "gdr_qk_norm_rope";
  RopeArgs a{};
  a.q = q; a.k = k; a.q_w = q_w; a.k_w = k_w; a.inv_freq = inv_freq; a.pos = pos; a.eps = eps;
  a.interleaved = interleaved != 0; a.q_out = q_out; a.k_out = k_out;
  a.q_tok = q_tok; a.q_head = q_head; a.k_tok = k_tok; a.k_head = k_head;
  a.B = B; a.N = N; a.Hq = Hq; a.Hk = Hk; a.D = D; a.R = R; a.bf16 = dt == GDR_BF16;
  gdr_status st = check_rope(a, dt, who);
  if (st != GDR_OK) return st;
  if (!q_out || !k_out) return fail(GDR_ERR_INVALID_ARG, "%s: q_out and k_out must be non-NULL", who);
  if (!aligned(q_out, 16) || !aligned(k_out, 16))
    return fail(GDR_ERR_INVALID_ARG, "%s: q_out and k_out must be 16-byte aligned", who);
  const int es = dt == GDR_BF16 ? 2 : 4;
  const unsigned long long T = (unsigned long long)B * N * D * es;
  st = apart_rope(a, {{q_out, T * Hq, "q_out"}, {k_out, T * Hk, "k_out"}},
                  {{q, span(a, Hq, q_tok, q_head, es), "q"}, {k, span(a, Hk, k_tok, k_head, es), "k"}}, who);
  if (st != GDR_OK) return st;
  return launched(launch_qk_norm_rope(a, reinterpret_cast<cudaStream_t>(stream)), who);
}

gdr_status gdr_qk_norm_rope_append(const void* q, const void* k, const void* v, const float* q_w,
                                   const float* k_w, const double* inv_freq, const int32_t* pos, float eps,
                                   int interleaved, void* q_out, void* k_pages, void* v_pages,
                                   const int32_t* table, const int32_t* ctx, const int32_t* lengths, int P,
                                   int page, int M, int B, int N, int Hq, int Hk, int D, int R, long long q_tok,
                                   long long q_head, long long k_tok, long long k_head, long long v_tok,
                                   long long v_head, gdr_dtype dt, gdr_stream_t stream) {
  const char* who = "gdr_qk_norm_rope_append";
  RopeArgs a{};
  a.q = q; a.k = k; a.v = v; a.q_w = q_w; a.k_w = k_w; a.inv_freq = inv_freq; a.pos = pos; a.eps = eps;
  a.interleaved = interleaved != 0; a.q_out = q_out; a.k_pages = k_pages; a.v_pages = v_pages;
  a.table = table; a.ctx = ctx; a.lengths = lengths; a.P = P; a.page = page; a.M = M;
  a.q_tok = q_tok; a.q_head = q_head; a.k_tok = k_tok; a.k_head = k_head; a.v_tok = v_tok; a.v_head = v_head;
  a.B = B; a.N = N; a.Hq = Hq; a.Hk = Hk; a.D = D; a.R = R; a.bf16 = dt == GDR_BF16;
  gdr_status st = check_rope(a, dt, who);
  if (st != GDR_OK) return st;
  if (!v || !q_out || !k_pages || !v_pages || !table || !ctx)
    return fail(GDR_ERR_INVALID_ARG, "%s: v, q_out, k_pages, v_pages, table and ctx must be non-NULL", who);
  st = check_pages(P, page, M, who);
  if (st != GDR_OK) return st;
  for (const void* p : {(const void*)q_out, (const void*)k_pages, (const void*)v_pages})
    if (!aligned(p, 16)) return fail(GDR_ERR_INVALID_ARG, "%s: q_out, k_pages and v_pages must be 16-byte aligned", who);
  for (const void* p : {(const void*)table, (const void*)ctx, (const void*)lengths})
    if (!aligned(p, 4)) return fail(GDR_ERR_INVALID_ARG, "%s: table, ctx and lengths must be 4-byte aligned", who);
  const int es = dt == GDR_BF16 ? 2 : 4;
  const unsigned long long pages = (unsigned long long)P * page * Hk * D * es;
  st = apart_rope(a, {{q_out, (unsigned long long)B * N * Hq * D * es, "q_out"}, {k_pages, pages, "k_pages"}, {v_pages, pages, "v_pages"}},
                  {{q, span(a, Hq, q_tok, q_head, es), "q"}, {k, span(a, Hk, k_tok, k_head, es), "k"},
                   {v, span(a, Hk, v_tok, v_head, es), "v"}, {table, (unsigned long long)B * M * 4, "table"},
                   {ctx, B * 4ull, "ctx"}, {lengths, B * 4ull, "lengths"}}, who);
  if (st != GDR_OK) return st;
  a.err = device_error_word();
  if (!a.err) return no_device(who);
  return launched(launch_qk_norm_rope(a, reinterpret_cast<cudaStream_t>(stream)), who);
}

size_t gdr_qk_norm_rope_backward_workspace_bytes(int D) {
  return D == 64 || D == 128 || D == 256 ? qk_norm_rope_backward_workspace_bytes(D) : 0;
}

gdr_status gdr_qk_norm_rope_backward(const void* q, const void* k, const float* q_w, const float* k_w,
                                     const double* inv_freq, const int32_t* pos, const void* dq_out,
                                     const void* dk_out, float eps, int interleaved, float* dq, float* dk,
                                     float* dq_w, float* dk_w, int B, int N, int Hq, int Hk, int D, int R,
                                     long long q_tok, long long q_head, long long k_tok, long long k_head,
                                     gdr_dtype dt, void* ws, size_t ws_bytes, gdr_stream_t stream) {
  const char* who = "gdr_qk_norm_rope_backward";
  RopeArgs a{};
  a.q = q; a.k = k; a.q_w = q_w; a.k_w = k_w; a.inv_freq = inv_freq; a.pos = pos; a.eps = eps;
  a.interleaved = interleaved != 0; a.dq_out = dq_out; a.dk_out = dk_out; a.dq = dq; a.dk = dk; a.dq_w = dq_w; a.dk_w = dk_w;
  a.q_tok = q_tok; a.q_head = q_head; a.k_tok = k_tok; a.k_head = k_head; a.partial = static_cast<float*>(ws);
  a.B = B; a.N = N; a.Hq = Hq; a.Hk = Hk; a.D = D; a.R = R; a.bf16 = dt == GDR_BF16;
  gdr_status st = check_rope(a, dt, who);
  if (st != GDR_OK) return st;
  if (!dq_out || !dk_out || !dq || !dk || !dq_w || !dk_w)
    return fail(GDR_ERR_INVALID_ARG, "%s: dq_out, dk_out, dq, dk, dq_w and dk_w must be non-NULL", who);
  for (const void* p : {dq_out, dk_out, (const void*)dq, (const void*)dk, (const void*)dq_w, (const void*)dk_w})
    if (!aligned(p, 16)) return fail(GDR_ERR_INVALID_ARG, "%s: every gradient must be 16-byte aligned", who);
  const size_t need = qk_norm_rope_backward_workspace_bytes(D);
  st = check_ws(ws, ws_bytes, need, who);
  if (st != GDR_OK) return st;
  const int es = dt == GDR_BF16 ? 2 : 4;
  const unsigned long long T = (unsigned long long)B * N * D;
  st = apart_rope(a, {{dq, T * Hq * 4, "dq"}, {dk, T * Hk * 4, "dk"}, {dq_w, D * 4ull, "dq_w"}, {dk_w, D * 4ull, "dk_w"}, {ws, need, "ws"}},
                  {{q, span(a, Hq, q_tok, q_head, es), "q"}, {k, span(a, Hk, k_tok, k_head, es), "k"},
                   {dq_out, T * Hq * es, "dq_out"}, {dk_out, T * Hk * es, "dk_out"}}, who);
  if (st != GDR_OK) return st;
  return launched(launch_qk_norm_rope_backward(a, reinterpret_cast<cudaStream_t>(stream)), who);
}

size_t gdr_tree_attn_workspace_bytes(int D) {
  return D == 64 || D == 128 || D == 256 ? tree_attn_workspace_bytes(D) : 0;
}

gdr_status gdr_tree_attn(const void* q, const void* k_pages, const void* v_pages, const int32_t* table,
                         const int32_t* ctx, const int32_t* lengths, const uint64_t* mask, float scale, void* o,
                         float* lse, int B, int N, int Hq, int Hk, int D, int P, int page, int M, gdr_dtype dt,
                         void* ws, size_t ws_bytes, gdr_stream_t stream) {
  const char* who = "gdr_tree_attn";
  if (!q || !k_pages || !v_pages || !table || !ctx || !o)
    return fail(GDR_ERR_INVALID_ARG, "%s: q, k_pages, v_pages, table, ctx and o must be non-NULL", who);
  gdr_status st = check_heads(B, N, Hq, Hk, D, dt, who);
  if (st == GDR_OK && dt != GDR_BF16) st = fail(GDR_ERR_UNSUPPORTED, "%s: bfloat16 only (dt=%d)", who, (int)dt);
  if (st == GDR_OK) st = check_pages(P, page, M, who);
  if (st != GDR_OK) return st;
  if (Hq / Hk > 128) return fail(GDR_ERR_UNSUPPORTED, "%s: Hq/Hk=%d exceeds 128 heads a group", who, Hq / Hk);
  if (B > 65535 || (long long)N * Hq > 1 << 28 || (long long)B * N * Hk > 0x7fffffffll) return fail(GDR_ERR_UNSUPPORTED, "%s: B=%d or N*Hq too large", who, B);
  if (!(scale > 0.f) || scale > 1e30f) return fail(GDR_ERR_INVALID_ARG, "%s: scale must be positive and finite", who);
  for (const void* p : {q, k_pages, v_pages, (const void*)o})
    if (!aligned(p, 16)) return fail(GDR_ERR_INVALID_ARG, "%s: q, k_pages, v_pages and o must be 16-byte aligned", who);
  for (const void* p : {(const void*)table, (const void*)ctx, (const void*)lengths, (const void*)lse})
    if (!aligned(p, 4)) return fail(GDR_ERR_INVALID_ARG, "%s: table, ctx, lengths and lse must be 4-byte aligned", who);
  if (!aligned(mask, 8)) return fail(GDR_ERR_INVALID_ARG, "%s: mask must be 8-byte aligned", who);
  const size_t need = tree_attn_workspace_bytes(D);
  st = check_ws(ws, ws_bytes, need, who);
  if (st != GDR_OK) return st;
  const unsigned long long rows = (unsigned long long)B * N * Hq, pages = (unsigned long long)P * page * Hk * D * 2;
  st = apart({{o, rows * D * 2, "o"}, {lse, rows * 4, "lse"}, {ws, need, "ws"}},
             {{q, rows * D * 2, "q"}, {k_pages, pages, "k_pages"}, {v_pages, pages, "v_pages"},
              {table, (unsigned long long)B * M * 4, "table"}, {ctx, B * 4ull, "ctx"}, {lengths, B * 4ull, "lengths"},
              {mask, (unsigned long long)B * N * ((N + 63) / 64) * 8, "mask"}}, who);
  if (st != GDR_OK) return st;
  int* err = device_error_word();
  if (!err) return no_device(who);
  const TreeAttnArgs a{q, k_pages, v_pages, table, ctx, lengths, mask, scale, o, lse, B, N, Hq, Hk, D, P, page, M,
                       static_cast<uint8_t*>(ws), err};
  return launched(launch_tree_attn(a, reinterpret_cast<cudaStream_t>(stream)), who);
}

gdr_status gdr_verify_draft(const int32_t* tokens, const int32_t* parents, const int32_t* lengths, const void* p,
                            const void* q, const float* u, const float* u_next, int32_t* path, int32_t* n_path,
                            int32_t* next_token, int B, int N, int V, gdr_dtype dt, gdr_stream_t stream) {
  const char* who = "gdr_verify_draft";
  if (!tokens || !parents || !lengths || !p || !u || !u_next || !path || !n_path || !next_token)
    return fail(GDR_ERR_INVALID_ARG, "%s: tokens, parents, lengths, p, u, u_next, path, n_path and next_token must be non-NULL", who);
  if (B < 1 || N < 1 || V < 1) return fail(GDR_ERR_INVALID_ARG, "%s: sizes must be >= 1 (B=%d N=%d V=%d)", who, B, N, V);
  if (dt != GDR_F32 && dt != GDR_BF16) return fail(GDR_ERR_INVALID_ARG, "%s: unknown dtype %d", who, (int)dt);
  if (N > kVerifyMaxNodes) return fail(GDR_ERR_UNSUPPORTED, "%s: N=%d exceeds %d nodes", who, N, kVerifyMaxNodes);
  if (V >= 1 << 30 || B > 1 << 24) return fail(GDR_ERR_UNSUPPORTED, "%s: B=%d or V=%d too large", who, B, V);
  const uintptr_t es = dt == GDR_BF16 ? 2 : 4;
  for (const void* x : {(const void*)tokens, (const void*)parents, (const void*)lengths, (const void*)u, (const void*)u_next,
                        (const void*)path, (const void*)n_path, (const void*)next_token})
    if (!aligned(x, 4)) return fail(GDR_ERR_INVALID_ARG, "%s: int32 and float32 arrays must be 4-byte aligned", who);
  if (!aligned(p, es) || !aligned(q, es))
    return fail(GDR_ERR_INVALID_ARG, "%s: p and q must be aligned to their elements", who);
  const unsigned long long bn = (unsigned long long)B * N;
  gdr_status st = apart({{path, bn * 4, "path"}, {n_path, B * 4ull, "n_path"}, {next_token, B * 4ull, "next_token"}},
                        {{tokens, bn * 4, "tokens"}, {parents, bn * 4, "parents"}, {lengths, B * 4ull, "lengths"},
                         {p, bn * V * es, "p"}, {q, bn * V * es, "q"}, {u, bn * 4, "u"}, {u_next, B * 4ull, "u_next"}}, who);
  if (st != GDR_OK) return st;
  int* err = device_error_word();
  if (!err) return no_device(who);
  const VerifyArgs a{tokens, parents, lengths, p, q, u, u_next, path, n_path, next_token, B, N, V, dt == GDR_BF16, err};
  return launched(launch_verify_draft(a, reinterpret_cast<cudaStream_t>(stream)), who);
}

size_t gdr_cache_workspace_bytes(int F, int M) {
  if (F < 1 || M < 1 || (long long)F * M > 0x3fffffffll) return 0;
  return cache_workspace_bytes(F, M);
}

gdr_status gdr_cache_reserve(int32_t* table, const int32_t* ctx, int32_t* refs, const int32_t* rows, int extra,
                             int F, int R, int M, int P, int page, void* ws, size_t ws_bytes,
                             gdr_stream_t stream) {
  const char* who = "gdr_cache_reserve";
  gdr_status st = check_rows(table, ctx, refs, rows, F, R, M, P, who);
  if (st == GDR_OK) st = check_pages(P, page, M, who);
  if (st == GDR_OK && extra < 0) st = fail(GDR_ERR_INVALID_ARG, "%s: extra=%d must be >= 0", who, extra);
  if (st == GDR_OK) st = check_ws(ws, ws_bytes, cache_workspace_bytes(F, M), who);
  if (st == GDR_OK)
    st = apart({{table, (unsigned long long)R * M * 4, "table"}, {refs, P * 4ull, "refs"}, {ws, cache_workspace_bytes(F, M), "ws"}},
               {{ctx, R * 4ull, "ctx"}, {rows, F * 4ull, "rows"}}, who);
  if (st != GDR_OK) return st;
  CacheArgs a{};
  a.table = table; a.ctx = const_cast<int32_t*>(ctx); a.refs = refs; a.dst = rows; a.extra = extra;
  a.F = F; a.rows = R; a.M = M; a.P = P; a.page = page; a.ws = static_cast<int32_t*>(ws);
  a.err = device_error_word();
  if (!a.err) return no_device(who);
  return launched(launch_cache_reserve(a, reinterpret_cast<cudaStream_t>(stream)), who);
}

gdr_status gdr_cache_fork(void* k_cache, void* v_cache, int32_t* table, int32_t* ctx, int32_t* refs,
                          const int32_t* src, const int32_t* dst, int F, int R, int M, int layers, int P, int page,
                          long long row_bytes, void* ws, size_t ws_bytes, gdr_stream_t stream) {
  const char* who = "gdr_cache_fork";
  gdr_status st = check_rows(table, ctx, refs, dst, F, R, M, P, who);
  if (st == GDR_OK) st = check_pages(P, page, M, who);
  if (st == GDR_OK && (!src || !aligned(src, 4)))
    st = fail(GDR_ERR_INVALID_ARG, "%s: src must be non-NULL and 4-byte aligned", who);
  if (st == GDR_OK) st = check_cache(k_cache, v_cache, layers, P, page, row_bytes, who);
  if (st == GDR_OK) st = check_ws(ws, ws_bytes, cache_workspace_bytes(F, M), who);
  if (st == GDR_OK) {
    const unsigned long long bytes = cache_bytes(layers, P, page, row_bytes);
    st = apart({{k_cache, bytes, "k_cache"}, {v_cache, bytes, "v_cache"}, {table, (unsigned long long)R * M * 4, "table"},
                {ctx, R * 4ull, "ctx"}, {refs, P * 4ull, "refs"}, {ws, cache_workspace_bytes(F, M), "ws"}},
               {{src, F * 4ull, "src"}, {dst, F * 4ull, "dst"}}, who);
  }
  if (st != GDR_OK) return st;
  CacheArgs a{};
  a.k_cache = static_cast<uint8_t*>(k_cache); a.v_cache = static_cast<uint8_t*>(v_cache);
  a.table = table; a.ctx = ctx; a.refs = refs; a.src = src; a.dst = dst;
  a.layers = layers; a.P = P; a.page = page; a.page_shift = __builtin_ctz((unsigned)page); a.rows = R; a.M = M; a.F = F; a.row_bytes = row_bytes;
  a.ws = static_cast<int32_t*>(ws);
  a.err = device_error_word();
  if (!a.err) return no_device(who);
  return launched(launch_cache_fork(a, reinterpret_cast<cudaStream_t>(stream)), who);
}

gdr_status gdr_cache_free(int32_t* table, int32_t* ctx, int32_t* refs, const int32_t* rows, int F, int R, int M,
                          int P, gdr_stream_t stream) {
  const char* who = "gdr_cache_free";
  gdr_status st = check_rows(table, ctx, refs, rows, F, R, M, P, who);
  if (st == GDR_OK)
    st = apart({{table, (unsigned long long)R * M * 4, "table"}, {ctx, R * 4ull, "ctx"}, {refs, P * 4ull, "refs"}},
               {{rows, F * 4ull, "rows"}}, who);
  if (st != GDR_OK) return st;
  CacheArgs a{};
  a.table = table; a.ctx = ctx; a.refs = refs; a.dst = rows; a.F = F; a.rows = R; a.M = M; a.P = P;
  a.err = device_error_word();
  if (!a.err) return no_device(who);
  return launched(launch_cache_free(a, reinterpret_cast<cudaStream_t>(stream)), who);
}

gdr_status gdr_cache_compact(void* k_cache, void* v_cache, const int32_t* table, const int32_t* ctx,
                             const int32_t* path, const int32_t* n_path, int32_t* new_ctx, int B, int W, int M,
                             int layers, int P, int page, long long row_bytes, gdr_stream_t stream) {
  const char* who = "gdr_cache_compact";
  if (!table || !ctx || !path || !n_path || !new_ctx)
    return fail(GDR_ERR_INVALID_ARG, "%s: table, ctx, path, n_path and new_ctx must be non-NULL", who);
  if (B < 1 || W < 1) return fail(GDR_ERR_INVALID_ARG, "%s: sizes must be >= 1 (B=%d W=%d)", who, B, W);
  if (W > kCompactMaxPath || B > 1 << 24)
    return fail(GDR_ERR_UNSUPPORTED, "%s: W=%d exceeds %d path entries, or B=%d is too large", who, W, kCompactMaxPath, B);
  gdr_status st = check_pages(P, page, M, who);
  if (st == GDR_OK) st = check_cache(k_cache, v_cache, layers, P, page, row_bytes, who);
  if (st != GDR_OK) return st;
  for (const void* x : {(const void*)table, (const void*)ctx, (const void*)path, (const void*)n_path, (const void*)new_ctx})
    if (!aligned(x, 4)) return fail(GDR_ERR_INVALID_ARG, "%s: int32 arrays must be 4-byte aligned", who);
  const unsigned long long bytes = cache_bytes(layers, P, page, row_bytes);
  st = apart({{k_cache, bytes, "k_cache"}, {v_cache, bytes, "v_cache"}, {new_ctx, B * 4ull, "new_ctx"}},
             {{ctx, B * 4ull, "ctx"}, {n_path, B * 4ull, "n_path"}, {path, (unsigned long long)B * W * 4, "path"}, {table, (unsigned long long)B * M * 4, "table"}}, who);
  if (st != GDR_OK) return st;
  int* err = device_error_word();
  if (!err) return no_device(who);
  const CompactArgs a{static_cast<uint8_t*>(k_cache), static_cast<uint8_t*>(v_cache), table, ctx, path, n_path, new_ctx,
                      layers, P, page, B, M, W, row_bytes, err};
  return launched(launch_cache_compact(a, reinterpret_cast<cudaStream_t>(stream)), who);
}

}  // extern "C"
