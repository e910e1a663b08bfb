// C-ABI entry points of the decoder's operators (molora_decoder.h): argument validation on the
// host, launches.
#include <hip/hip_runtime.h>

#include <algorithm>
#include <cmath>
#include <memory>
#include <new>

#include "capi_internal.h"
#include "decoder_launch.h"
#include "molora_decoder.h"

using molora::aligned;
using molora::fail;
using molora::hip_fail;
using molora::ok;

static_assert(MOLORA_SCORE_SOFTMAX == molora::kScoreSoftmax && MOLORA_SCORE_SIGMOID == molora::kScoreSigmoid, "scores");

namespace {

constexpr long long kMaxRows = 1ll << 24;      // tokens, sequences
constexpr long long kMaxGroups = 1ll << 24;    // workgroups of a launch: 2^32 threads of 256 each
constexpr long long kMaxStride = 1ll << 23;    // elements between tokens: 64 rows fit 32-bit byte offsets
constexpr int kMaxWindow = 1 << 25;            // wider than any sequence

hipStream_t stream_of(void* s) { return reinterpret_cast<hipStream_t>(s); }

molora::Rows rows_of(const molora_rows* r) {
  return {static_cast<uint16_t*>(r->p), r->token, r->head};
}

// One packed tensor of T rows of H heads; written ones must not overlap themselves.
int check_rows(const molora_rows* r, const char* name, long long T, int H, int D, bool written) {
  if (r == nullptr) return fail(MOLORA_EINVAL, "%s is NULL", name);
  if (T == 0) return MOLORA_OK;
  if (r->p == nullptr || !aligned(r->p, 16)) return fail(MOLORA_EINVAL, "%s: NULL or not 16-byte aligned", name);
  if (r->token < 0 || r->head < 0 || r->token % 8 != 0 || r->head % 8 != 0)
    return fail(MOLORA_EINVAL, "%s: strides %lld, %lld must be non-negative multiples of 8", name, r->token, r->head);
  if (r->token >= kMaxStride || r->head >= (1ll << 40))
    return fail(MOLORA_ENOTSUP, "%s: strides %lld, %lld too large", name, r->token, r->head);
  if (written) {
    const bool by_token = (H == 1 || r->head >= D) && (T == 1 || r->token >= (H - 1) * r->head + D);
    const bool by_head = (T == 1 || r->token >= D) && (H == 1 || r->head >= (T - 1) * r->token + D);
    if (!by_token && !by_head) return fail(MOLORA_EINVAL, "%s: its rows overlap", name);
  }
  return MOLORA_OK;
}

int check_score(int N, int K, int k, int score, float factor) {
  if (N < 0) return fail(MOLORA_EINVAL, "N=%d < 0", N);
  if (K < 1 || K > MOLORA_MAX_ADAPTERS) return fail(MOLORA_ENOTSUP, "K=%d outside [1, %d]", K, MOLORA_MAX_ADAPTERS);
  if (k < 1 || k > K || k > MOLORA_MAX_TOPK)
    return fail(MOLORA_ENOTSUP, "k=%d outside [1, min(K=%d, %d)]", k, K, MOLORA_MAX_TOPK);
  if ((long long)N * K >= (1ll << 31) || N >= (1 << 29))
    return fail(MOLORA_ENOTSUP, "N=%d tokens of K=%d logits: too many", N, K);
  if (score != MOLORA_SCORE_SOFTMAX && score != MOLORA_SCORE_SIGMOID) return fail(MOLORA_EINVAL, "score=%d", score);
  if (!std::isfinite(factor)) return fail(MOLORA_EINVAL, "factor is not finite");
  return MOLORA_OK;
}

int check_heads(int n_heads, int n_kv_heads, int head_dim) {
  if (head_dim != 64 && head_dim != 128) return fail(MOLORA_ENOTSUP, "head_dim=%d is neither 64 nor 128", head_dim);
  if (n_kv_heads < 1 || n_heads < 1 || n_heads > 1024 || n_heads % n_kv_heads != 0)
    return fail(MOLORA_ENOTSUP, "n_heads=%d, n_kv_heads=%d", n_heads, n_kv_heads);
  return MOLORA_OK;
}

int check_mask(int window, int sinks, float scale) {
  if (window < 0 || sinks < 0) return fail(MOLORA_EINVAL, "window=%d, sinks=%d: negative", window, sinks);
  if (sinks > kMaxRows) return fail(MOLORA_ENOTSUP, "sinks=%d too large", sinks);
  if (!(scale > 0.f) || !std::isfinite(scale)) return fail(MOLORA_EINVAL, "scale must be positive and finite");
  return MOLORA_OK;
}

int check_shape(const molora_attn_shape* s) {
  if (s == nullptr) return fail(MOLORA_EINVAL, "shape is NULL");
  int rc = check_heads(s->n_heads, s->n_kv_heads, s->head_dim);
  if (rc != MOLORA_OK) return rc;
  if (s->n_seq < 0 || s->Tq < 0 || s->Tkv < 0) return fail(MOLORA_EINVAL, "negative n_seq, Tq or Tkv");
  if (s->n_seq >= kMaxRows || s->Tq >= kMaxRows || s->Tkv >= kMaxRows)
    return fail(MOLORA_ENOTSUP, "n_seq=%d, Tq=%d, Tkv=%d too large", s->n_seq, s->Tq, s->Tkv);
  if (std::max(molora::attn_slots(s->Tq, s->n_seq, molora::kAttnQ) * s->n_heads,
               molora::attn_slots(s->Tkv, s->n_seq, molora::kAttnK) * s->n_kv_heads) >= kMaxGroups)
    return fail(MOLORA_ENOTSUP, "too many (tile, head) pairs");
  if ((rc = check_mask(s->window, s->sinks, s->scale)) != MOLORA_OK) return rc;
  if (s->n_seq > 0 && (s->q_off == nullptr || !aligned(s->q_off, 4) || !aligned(s->kv_off, 4)))
    return fail(MOLORA_EINVAL, "q_off NULL, or offsets misaligned");
  return MOLORA_OK;
}

molora::AttnArgs attn_args(const molora_attn_shape* s, const molora_rows* q, const molora_rows* k,
                           const molora_rows* v, const molora_rows* o) {
  molora::AttnArgs a{};
  a.q = rows_of(q);
  a.k = rows_of(k);
  a.v = rows_of(v);
  a.o = rows_of(o);
  a.q_off = s->q_off;
  a.kv_off = s->kv_off != nullptr ? s->kv_off : s->q_off;
  a.n_seq = s->n_seq;
  a.Hq = s->n_heads;
  a.Hkv = s->n_kv_heads;
  a.D = s->head_dim;
  a.Tq = s->Tq;
  a.Tkv = s->Tkv;
  a.window = std::min(s->window, kMaxWindow);
  a.sinks = s->sinks;
  a.scale = s->scale;
  return a;
}

size_t fwd_bytes_of(const molora_attn_shape* s) {
  return molora::attn_fwd_ws_bytes(s->Tq, s->Tkv, s->n_seq, s->n_heads, s->head_dim, s->window, s->sinks);
}

molora::AttnBwdPlan bwd_plan_of(const molora_attn_shape* s) {
  return molora::attn_bwd_plan(s->Tq, s->Tkv, s->n_seq, s->n_heads, s->n_kv_heads, s->head_dim, s->window,
                               s->sinks);
}

int check_cache(const molora_kv_cache* c) {
  if (c == nullptr) return fail(MOLORA_EINVAL, "cache is NULL");
  if (c->head_dim != 64 && c->head_dim != 128)
    return fail(MOLORA_ENOTSUP, "head_dim=%d is neither 64 nor 128", c->head_dim);
  if (c->n_pages < 1 || c->n_kv_heads < 1 || c->n_kv_heads > 1024)
    return fail(MOLORA_ENOTSUP, "n_pages=%d, n_kv_heads=%d", c->n_pages, c->n_kv_heads);
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0)
    return fail(MOLORA_ENOTSUP, "page_size=%d is not 16, 32, 64, 128 or 256", c->page_size);
  if (c->dtype != MOLORA_BF16 && c->dtype != MOLORA_E4M3) return fail(MOLORA_EINVAL, "cache dtype %d", c->dtype);
  return MOLORA_OK;
}

int check_cache_ptrs(const molora_kv_cache* c) {
  if (c->k == nullptr || c->v == nullptr || !aligned(c->k, 16) || !aligned(c->v, 16))
    return fail(MOLORA_EINVAL, "cache k or v NULL or not 16-byte aligned");
  if (c->dtype == MOLORA_E4M3 && (c->k_scale == nullptr || c->v_scale == nullptr || !aligned(c->k_scale, 16) ||
                                  !aligned(c->v_scale, 16)))
    return fail(MOLORA_EINVAL, "e4m3 cache: k_scale or v_scale NULL or not 16-byte aligned");
  return MOLORA_OK;
}

int check_table(const molora_kv_cache* c, int n_seq, int width) {
  if (n_seq < 0 || width < 0) return fail(MOLORA_EINVAL, "n_seq=%d, table_width=%d", n_seq, width);
  if (n_seq >= kMaxRows || (long long)width * c->page_size >= (1ll << 30))
    return fail(MOLORA_ENOTSUP, "n_seq=%d, table_width=%d too large", n_seq, width);
  return MOLORA_OK;
}

molora::KvCacheDev cache_dev(const molora_kv_cache* c) {
  molora::KvCacheDev d{};
  d.k = c->k;
  d.v = c->v;
  d.k_scale = c->k_scale;
  d.v_scale = c->v_scale;
  d.n_pages = c->n_pages;
  d.Hkv = c->n_kv_heads;
  while ((1 << d.page_shift) < c->page_size) ++d.page_shift;
  d.D = c->head_dim;
  d.e4m3 = c->dtype == MOLORA_E4M3;
  return d;
}

}  // namespace

extern "C" {

int molora_route_scores(const float* logits, const float* bias, int N, int K, int k, int score, int n_group,
                        int topk_group, int renorm, float factor, int32_t* idx, float* w, void* stream) {
  const int rc = check_score(N, K, k, score, factor);
  if (rc != MOLORA_OK) return rc;
  if (n_group < 1 || K % n_group != 0 || topk_group < 1 || topk_group > n_group || k > topk_group * (K / n_group))
    return fail(MOLORA_ENOTSUP, "n_group=%d, topk_group=%d with K=%d, k=%d", n_group, topk_group, K, k);
  if (N == 0) return ok();
  if (logits == nullptr || idx == nullptr || w == nullptr) return fail(MOLORA_EINVAL, "a required pointer is NULL");
  if (!aligned(logits, 16) || !aligned(bias, 4) || !aligned(idx, 4) || !aligned(w, 4))
    return fail(MOLORA_EINVAL, "misaligned pointer");
  molora::RouteScoresArgs a{logits, bias, N, K, k, score, n_group, topk_group, renorm != 0, factor, idx, w};
  const hipError_t e = molora::launch_route_scores(a, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "route_scores launch");
}

int molora_route_scores_backward(const float* logits, const int32_t* idx, const float* dw, int N, int K, int k,
                                 int score, int renorm, float factor, float* dlogits, void* stream) {
  const int rc = check_score(N, K, k, score, factor);
  if (rc != MOLORA_OK) return rc;
  if (N == 0) return ok();
  if (logits == nullptr || idx == nullptr || dw == nullptr || dlogits == nullptr)
    return fail(MOLORA_EINVAL, "a required pointer is NULL");
  if (!aligned(logits, 16) || !aligned(dlogits, 16) || !aligned(idx, 4) || !aligned(dw, 4))
    return fail(MOLORA_EINVAL, "misaligned pointer");
  molora::RouteScoresArgs a{logits, nullptr, N, K, k, score, 1, 1, renorm != 0, factor, const_cast<int32_t*>(idx),
                            nullptr};
  const hipError_t e = molora::launch_route_scores_backward(a, dw, dlogits, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "route_scores_backward launch");
}

int molora_attn_forward_workspace(const molora_attn_shape* shape, size_t* bytes) {
  if (bytes == nullptr) return fail(MOLORA_EINVAL, "bytes is NULL");
  const int rc = check_shape(shape);
  if (rc != MOLORA_OK) return rc;
  *bytes = fwd_bytes_of(shape);
  return ok();
}

int molora_attn_forward(const molora_attn_shape* shape, const molora_rows* q, const molora_rows* k,
                        const molora_rows* v, const molora_rows* o, float* lse, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_shape(shape);
  if (rc != MOLORA_OK) return rc;
  const int D = shape->head_dim;
  if ((rc = check_rows(q, "q", shape->Tq, shape->n_heads, D, false)) != MOLORA_OK) return rc;
  if ((rc = check_rows(k, "k", shape->Tkv, shape->n_kv_heads, D, false)) != MOLORA_OK) return rc;
  if ((rc = check_rows(v, "v", shape->Tkv, shape->n_kv_heads, D, false)) != MOLORA_OK) return rc;
  if ((rc = check_rows(o, "o", shape->Tq, shape->n_heads, D, true)) != MOLORA_OK) return rc;
  if (!aligned(lse, 4)) return fail(MOLORA_EINVAL, "lse misaligned");
  if (shape->Tq == 0 || shape->n_seq == 0) return ok();
  const size_t need = fwd_bytes_of(shape);
  if (need > 0 && (ws == nullptr || ws_bytes < need || !aligned(ws, 256)))
    return fail(MOLORA_ENOSPC, "workspace of %zu bytes (256-byte aligned) needed, %zu given", need, ws_bytes);
  molora::AttnArgs a = attn_args(shape, q, k, v, o);
  a.lse = lse;
  a.splits = molora::attn_q_splits(shape->Tq, shape->Tkv, shape->n_seq, shape->n_heads, shape->window, shape->sinks);
  a.part = static_cast<float*>(ws);
  const hipError_t e = molora::launch_attn_forward(a, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "attn_forward launch");
}

int molora_attn_backward_workspace(const molora_attn_shape* shape, size_t* bytes) {
  if (bytes == nullptr) return fail(MOLORA_EINVAL, "bytes is NULL");
  const int rc = check_shape(shape);
  if (rc != MOLORA_OK) return rc;
  *bytes = bwd_plan_of(shape).total;
  return ok();
}

int molora_attn_backward(const molora_attn_shape* shape, const molora_rows* dout, const molora_rows* q,
                         const molora_rows* k, const molora_rows* v, const molora_rows* o, const float* lse,
                         const molora_rows* dq, const molora_rows* dk, const molora_rows* dv, void* ws,
                         size_t ws_bytes, void* stream) {
  int rc = check_shape(shape);
  if (rc != MOLORA_OK) return rc;
  const int D = shape->head_dim, Hq = shape->n_heads, Hkv = shape->n_kv_heads;
  if ((rc = check_rows(dout, "dout", shape->Tq, Hq, D, false)) != MOLORA_OK) return rc;
  if ((rc = check_rows(q, "q", shape->Tq, Hq, D, false)) != MOLORA_OK) return rc;
  if ((rc = check_rows(k, "k", shape->Tkv, Hkv, D, false)) != MOLORA_OK) return rc;
  if ((rc = check_rows(v, "v", shape->Tkv, Hkv, D, false)) != MOLORA_OK) return rc;
  if ((rc = check_rows(o, "o", shape->Tq, Hq, D, false)) != MOLORA_OK) return rc;
  if ((rc = check_rows(dq, "dq", shape->Tq, Hq, D, true)) != MOLORA_OK) return rc;
  if ((rc = check_rows(dk, "dk", shape->Tkv, Hkv, D, true)) != MOLORA_OK) return rc;
  if ((rc = check_rows(dv, "dv", shape->Tkv, Hkv, D, true)) != MOLORA_OK) return rc;
  if (shape->n_seq == 0 || (shape->Tq == 0 && shape->Tkv == 0)) return ok();
  if (shape->Tq > 0 && (lse == nullptr || !aligned(lse, 4))) return fail(MOLORA_EINVAL, "lse NULL or misaligned");
  const molora::AttnBwdPlan plan = bwd_plan_of(shape);
  if (plan.total > 0 && (ws == nullptr || ws_bytes < plan.total || !aligned(ws, 256)))
    return fail(MOLORA_ENOSPC, "workspace of %zu bytes (256-byte aligned) needed, %zu given", plan.total, ws_bytes);
  molora::AttnBackwardArgs b{};
  b.f = attn_args(shape, q, k, v, o);
  b.f.lse = const_cast<float*>(lse);
  b.dout = rows_of(dout);
  b.dq = rows_of(dq);
  b.dk = rows_of(dk);
  b.dv = rows_of(dv);
  char* base = static_cast<char*>(ws);
  b.lse2 = reinterpret_cast<float*>(base + plan.lse_off);
  b.delta = reinterpret_cast<float*>(base + plan.delta_off);
  b.part = reinterpret_cast<float*>(base + plan.part_off);
  b.q_splits = plan.q_splits;
  b.q_part = reinterpret_cast<float*>(base + plan.q_part_off);
  b.splits = plan.splits;
  b.sink_splits = plan.sink_splits;
  b.sink_tiles = plan.sink_tiles;
  b.most = plan.most;
  b.min_steps = plan.min_steps;
  b.sink_min = plan.sink_min;
  const hipError_t e = molora::launch_attn_backward(b, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "attn_backward launch");
}

int molora_kv_append(const molora_kv_cache* cache, const molora_rows* k, const molora_rows* v, int T, int n_seq,
                     const int32_t* q_off, const int32_t* table, int table_width, const int32_t* lens, void* stream) {
  int rc = check_cache(cache);
  if (rc != MOLORA_OK) return rc;
  if ((rc = check_table(cache, n_seq, table_width)) != MOLORA_OK) return rc;
  if (T < 0) return fail(MOLORA_EINVAL, "T=%d < 0", T);
  if (T >= kMaxRows) return fail(MOLORA_ENOTSUP, "T=%d too large", T);
  if (q_off == nullptr && T > n_seq) return fail(MOLORA_EINVAL, "%d rows for %d sequences without q_off", T, n_seq);
  if ((rc = check_rows(k, "k", T, cache->n_kv_heads, cache->head_dim, false)) != MOLORA_OK) return rc;
  if ((rc = check_rows(v, "v", T, cache->n_kv_heads, cache->head_dim, false)) != MOLORA_OK) return rc;
  if (T == 0 || n_seq == 0 || table_width == 0) return ok();
  if ((rc = check_cache_ptrs(cache)) != MOLORA_OK) return rc;
  if (table == nullptr || lens == nullptr || !aligned(table, 4) || !aligned(lens, 4) || !aligned(q_off, 4))
    return fail(MOLORA_EINVAL, "table or lens NULL, or a pointer misaligned");
  molora::KvAppendArgs a{cache_dev(cache), rows_of(k), rows_of(v), T, n_seq, q_off, table, table_width, lens};
  const hipError_t e = molora::launch_kv_append(a, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "kv_append launch");
}

static int check_decode(const molora_kv_cache* cache, int n_seq, int n_heads, int table_width) {
  int rc = check_cache(cache);
  if (rc != MOLORA_OK) return rc;
  if ((rc = check_heads(n_heads, cache->n_kv_heads, cache->head_dim)) != MOLORA_OK) return rc;
  if ((rc = check_table(cache, n_seq, table_width)) != MOLORA_OK) return rc;
  if ((long long)n_seq * n_heads >= kMaxRows) return fail(MOLORA_ENOTSUP, "n_seq=%d, n_heads=%d", n_seq, n_heads);
  return MOLORA_OK;
}

int molora_attn_decode_workspace(const molora_kv_cache* cache, int n_seq, int n_heads, int table_width, size_t* bytes) {
  if (bytes == nullptr) return fail(MOLORA_EINVAL, "bytes is NULL");
  const int rc = check_decode(cache, n_seq, n_heads, table_width);
  if (rc != MOLORA_OK) return rc;
  *bytes = molora::decode_plan(n_seq, n_heads, cache->n_kv_heads, cache->head_dim, cache->page_size, table_width).total;
  return ok();
}

int molora_attn_decode(const molora_kv_cache* cache, const molora_rows* q, const molora_rows* o, float* lse, int n_seq,
                       int n_heads, const int32_t* table, int table_width, const int32_t* lens, int window, int sinks,
                       float scale, void* ws, size_t ws_bytes, void* stream) {
  int rc = check_decode(cache, n_seq, n_heads, table_width);
  if (rc != MOLORA_OK) return rc;
  if ((rc = check_mask(window, sinks, scale)) != MOLORA_OK) return rc;
  if ((rc = check_rows(q, "q", n_seq, n_heads, cache->head_dim, false)) != MOLORA_OK) return rc;
  if ((rc = check_rows(o, "o", n_seq, n_heads, cache->head_dim, true)) != MOLORA_OK) return rc;
  if (!aligned(lse, 4)) return fail(MOLORA_EINVAL, "lse misaligned");
  if (n_seq == 0) return ok();
  if ((rc = check_cache_ptrs(cache)) != MOLORA_OK) return rc;
  if (lens == nullptr || !aligned(lens, 4) || (table_width > 0 && (table == nullptr || !aligned(table, 4))))
    return fail(MOLORA_EINVAL, "table or lens NULL or misaligned");
  const molora::DecodePlan p =
      molora::decode_plan(n_seq, n_heads, cache->n_kv_heads, cache->head_dim, cache->page_size, table_width);
  if (p.total > 0 && (ws == nullptr || ws_bytes < p.total || !aligned(ws, 256)))
    return fail(MOLORA_ENOSPC, "workspace of %zu bytes (256-byte aligned) needed, %zu given", p.total, ws_bytes);
  molora::DecodeArgs a{};
  a.c = cache_dev(cache);
  a.q = rows_of(q);
  a.o = rows_of(o);
  a.lse = lse;
  a.n_seq = n_seq;
  a.Hq = n_heads;
  a.table = table;
  a.width = table_width;
  a.lens = lens;
  a.window = std::min(window, 1 << 30);
  a.sinks = sinks;
  a.scale = scale;
  a.splits = p.splits;
  a.part = static_cast<float*>(ws);
  const hipError_t e = molora::launch_attn_decode(a, stream_of(stream));
  return e == hipSuccess ? ok() : hip_fail(e, "attn_decode launch");
}

// The serving form's checks; on success *part is the decode attention's plan (single tokens).
static int check_serve(int d, int f, int n_layers, const molora_xf_layer* layers, const molora_kv_cache* caches, int n_seq,
                       int N, int table_width, int k, int* K, size_t* lora_bytes, int* paths, bool single,
                       molora::DecodePlan* part) {
  if (d <= 0 || f <= 0 || d % 128 != 0 || f % 128 != 0)
    return fail(MOLORA_ENOTSUP, "d=%d and f=%d must be positive multiples of 128", d, f);
  if (n_layers < 1 || n_layers > 1024 || layers == nullptr || caches == nullptr)
    return fail(MOLORA_EINVAL, "n_layers=%d, or layers or caches NULL", n_layers);
  if (n_seq < 0 || N < 0) return fail(MOLORA_EINVAL, "n_seq=%d, N=%d", n_seq, N);
  const int heads = d / molora::kXfHeadDim;
  if (N >= kMaxRows || (long long)N * std::max(d, f) >= (1ll << 31) || heads > 1024 ||
      (long long)n_seq * heads >= kMaxRows || molora::attn_slots(N, n_seq, molora::kAttnQ) * heads >= kMaxGroups)
    return fail(MOLORA_ENOTSUP, "batch of %d tokens in %d sequences too large", N, n_seq);
  if (k < 1 || k > MOLORA_MAX_TOPK) return fail(MOLORA_ENOTSUP, "k=%d outside [1, %d]", k, MOLORA_MAX_TOPK);
  for (int l = 0; l < n_layers; ++l) {
    int rc = check_cache(&caches[l]);
    if (rc == MOLORA_OK) rc = check_cache_ptrs(&caches[l]);
    if (rc == MOLORA_OK) rc = check_table(&caches[l], n_seq, table_width);
    if (rc != MOLORA_OK) return rc;
    if (caches[l].head_dim != molora::kXfHeadDim || caches[l].n_kv_heads != heads)
      return fail(MOLORA_EINVAL, "layer %d: the cache holds %d heads of %d, %d of %d needed", l, caches[l].n_kv_heads,
                  caches[l].head_dim, heads, molora::kXfHeadDim);
    if (caches[l].page_size != caches[0].page_size)
      return fail(MOLORA_EINVAL, "layer %d: page_size %d differs from %d", l, caches[l].page_size, caches[0].page_size);
  }
  int first = -1;  // one resolved path per projection serves every layer
  for (int l = 0; l < n_layers; ++l) {
    if (layers[l].lora == nullptr) continue;
    if (first < 0) first = l;
    if (layers[l].lora->r_pad != layers[first].lora->r_pad)
      return fail(MOLORA_ENOTSUP, "layers %d and %d: adapters of different (padded) rank", first, l);
  }
  *part = single ? molora::decode_plan(n_seq, heads, heads, molora::kXfHeadDim, caches[0].page_size, table_width)
                 : molora::DecodePlan{};
  return molora::xf_check_layers(d, f, n_layers, layers, std::max(N, 1), k, K, lora_bytes, paths);
}

int molora_xf_serve_workspace(int d, int f, int n_layers, const molora_xf_layer* layers, const molora_kv_cache* caches,
                              int n_seq, int N, int table_width, int k, size_t* bytes) {
  if (bytes == nullptr) return fail(MOLORA_EINVAL, "bytes is NULL");
  int K = 0;
  size_t lb = 0;
  molora::DecodePlan part{};
  const int rc = check_serve(d, f, n_layers, layers, caches, n_seq, N, table_width, k, &K, &lb, nullptr, true, &part);
  if (rc != MOLORA_OK) return rc;
  *bytes = molora::xf_serve_plan(N, d, f, lb, part.total).total;
  return ok();
}

static int serve(int d, int f, int n_layers, const molora_xf_layer* layers, const molora_kv_cache* caches, int n_seq,
                 int N, const int32_t* q_off, const int32_t* table, int table_width, const int32_t* lens, int window,
                 int sinks, const void* x_in, void* x_out, int k, const int32_t* offsets, const int32_t* perm,
                 const float* perm_w, const int32_t* inv, void* ws, size_t ws_bytes, void* stream, bool single) {
  int K = 0, paths[4] = {0, 0, 0, 0};
  size_t lb = 0;
  molora::DecodePlan part{};
  int rc = check_serve(d, f, n_layers, layers, caches, n_seq, N, table_width, k, &K, &lb, paths, single, &part);
  if (rc != MOLORA_OK) return rc;
  if ((rc = check_mask(window, sinks, 1.f)) != MOLORA_OK) return rc;
  if (N == 0) return ok();
  if (n_seq == 0) return fail(MOLORA_EINVAL, "%d tokens in no sequence", N);
  if (x_in == nullptr || x_out == nullptr || !aligned(x_in, 16) || !aligned(x_out, 16))
    return fail(MOLORA_EINVAL, "x_in or x_out NULL or not 16-byte aligned");
  if (table == nullptr || lens == nullptr || !aligned(table, 4) || !aligned(lens, 4) || !aligned(q_off, 4) ||
      (!single && q_off == nullptr))
    return fail(MOLORA_EINVAL, "table, lens or q_off NULL or misaligned");
  if (table_width == 0) return fail(MOLORA_EINVAL, "table_width is 0");
  if (K > 0 && (offsets == nullptr || perm == nullptr || perm_w == nullptr || inv == nullptr || !aligned(offsets, 4) ||
                !aligned(perm, 4) || !aligned(perm_w, 4) || !aligned(inv, 4)))
    return fail(MOLORA_EINVAL, "offsets, perm, perm_w and inv are required, 4-byte aligned, with LoRA layers");
  const size_t need = molora::xf_serve_plan(N, d, f, lb, part.total).total;
  if (ws == nullptr || ws_bytes < need || !aligned(ws, 256))
    return fail(MOLORA_ENOSPC, "workspace of %zu bytes (256-byte aligned) needed, %zu given", need, ws_bytes);
  std::unique_ptr<molora::XfLayerDev[]> dev(new (std::nothrow) molora::XfLayerDev[n_layers]);
  std::unique_ptr<molora::KvCacheDev[]> cd(new (std::nothrow) molora::KvCacheDev[n_layers]);
  if (dev == nullptr || cd == nullptr) return fail(MOLORA_EHIP, "out of host memory");
  molora::xf_layers_dev(n_layers, layers, dev.get());
  for (int l = 0; l < n_layers; ++l) cd[l] = cache_dev(&caches[l]);
  const char* what = "";
  molora::XfServeLaunch v{};
  molora::XfLaunch& a = v.xf;
  a.d = d; a.f = f; a.n_seq = N; a.seq_len = 1; a.n_layers = n_layers; a.K = K; a.k = k;
  a.eps = 1e-6f;
  a.layers = dev.get();
  a.x_in = static_cast<const uint16_t*>(x_in);
  a.x_out = static_cast<uint16_t*>(x_out);
  a.offsets = offsets; a.perm = perm; a.perm_w = perm_w; a.inv = inv;
  a.path_qkv = paths[0]; a.path_o = paths[1]; a.path_gu = paths[2]; a.path_down = paths[3];
  a.lora_bytes = lb;
  a.ws = static_cast<char*>(ws);
  a.what = &what;
  v.caches = cd.get();
  v.n_seq = n_seq;
  v.q_off = single ? nullptr : q_off;
  v.table = table;
  v.width = table_width;
  v.lens = lens;
  v.window = std::min(window, kMaxWindow);
  v.sinks = sinks;
  v.splits = part.splits;
  v.part_bytes = part.total;
  const hipError_t e = molora::launch_xf_serve(v, stream_of(stream));
  if (e != hipSuccess) return fail(MOLORA_EHIP, "decoder serving (%s): %s", what, hipGetErrorString(e));
  return ok();
}

int molora_xf_prefill(int d, int f, int n_layers, const molora_xf_layer* layers, const molora_kv_cache* caches, int n_seq,
                      int N, const int32_t* q_off, const int32_t* table, int table_width, const int32_t* lens, int window,
                      int sinks, const void* x_in, void* x_out, int k, const int32_t* offsets, const int32_t* perm,
                      const float* perm_w, const int32_t* inv, void* ws, size_t ws_bytes, void* stream) {
  return serve(d, f, n_layers, layers, caches, n_seq, N, q_off, table, table_width, lens, window, sinks, x_in, x_out, k,
               offsets, perm, perm_w, inv, ws, ws_bytes, stream, false);
}

int molora_xf_decode(int d, int f, int n_layers, const molora_xf_layer* layers, const molora_kv_cache* caches, int n_seq,
                     const int32_t* table, int table_width, const int32_t* lens, int window, int sinks, const void* x_in,
                     void* x_out, int k, const int32_t* offsets, const int32_t* perm, const float* perm_w,
                     const int32_t* inv, void* ws, size_t ws_bytes, void* stream) {
  return serve(d, f, n_layers, layers, caches, n_seq, n_seq, nullptr, table, table_width, lens, window, sinks, x_in,
               x_out, k, offsets, perm, perm_w, inv, ws, ws_bytes, stream, true);
}

}  // extern "C"
