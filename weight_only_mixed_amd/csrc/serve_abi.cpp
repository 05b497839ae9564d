// C ABI of the serving operators (slq_serve.h): argument validation on the
// host, then the HIP launchers.  As in slq_abi.cpp every check runs before the
// first HIP call.
#include <cmath>
#include <hip/hip_runtime.h>

#include <stdint.h>

#include "../../include/slq_serve.h"
#include "serve.h"

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 30;     // rows * heads, and cached tokens per sequence
constexpr int64_t kMaxBatch = 65535;
constexpr int64_t kMaxStride = (int64_t)1 << 40;

bool aligned(const void *p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

struct Extent {
  const void *p;
  size_t n;
};
bool overlap(Extent a, Extent b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const char *pa = static_cast<const char *>(a.p), *pb = static_cast<const char *>(b.p);
  return pa < pb + b.n && pb < pa + a.n;
}

slq_status from_hip(hipError_t e) { return e == hipSuccess ? SLQ_OK : SLQ_EHIP; }

size_t elem_bytes(slq_dtype t) { return t == SLQ_F32 ? 4 : 2; }
bool dtype_ok(slq_dtype t) { return t == SLQ_F32 || t == SLQ_BF16 || t == SLQ_F16; }

struct CacheExtents {
  Extent codes[2], scales[2];
  bool hits(Extent e) const {
    return overlap(e, codes[0]) || overlap(e, codes[1]) || overlap(e, scales[0]) ||
           overlap(e, scales[1]);
  }
};

// Bytes from a page's first to behind its last code.
int64_t page_span(const slq_kv_cache *c) {
  return (int64_t)(c->heads - 1) * c->head_stride + (int64_t)(c->page_size - 1) * c->token_stride +
         c->head_dim;
}

slq_status check_cache(const slq_kv_cache *c, slq::KvView *v, CacheExtents *x) {
  if (!c) return SLQ_EINVAL;
  if (c->format != SLQ_KV_INT8 && c->format != SLQ_KV_E4M3) return SLQ_EINVAL;
  if (c->heads < 1 || c->heads > 1024 || c->head_dim < 1 || c->page_size < 1 || c->pages < 0 ||
      c->pages >= ((int64_t)1 << 31))
    return SLQ_EINVAL;
  if (c->head_dim != 64 && c->head_dim != 128 && c->head_dim != 256) return SLQ_ENOTSUP;
  if (c->page_size < 16 || c->page_size > 256 || (c->page_size & (c->page_size - 1)) != 0)
    return SLQ_ENOTSUP;
  const int64_t ps = c->page_stride, hs = c->head_stride, ts = c->token_stride;
  if (ps < 0 || hs < 0 || ts < 0 || ps >= kMaxStride || hs >= kMaxStride || ts >= kMaxStride ||
      ps % 16 || hs % 16 || ts % 16)
    return SLQ_EINVAL;
  const bool heads_outside = ts >= c->head_dim &&
                             (c->heads == 1 || hs >= (c->page_size - 1) * ts + c->head_dim);
  const bool slots_outside = (c->heads == 1 || hs >= c->head_dim) &&
                             ts >= (c->heads - 1) * hs + c->head_dim;
  if (!heads_outside && !slots_outside) return SLQ_EINVAL;
  const int64_t span = page_span(c);
  if (span >= ((int64_t)1 << 31)) return SLQ_EINVAL;   // offsets within a page fit 32 bits
  if (c->pages > 1 && (ps < span || ps > ((int64_t)1 << 60) / c->pages)) return SLQ_EINVAL;
  *x = CacheExtents{};
  if (c->pages > 0) {
    if (!c->k_codes || !c->v_codes || !c->k_scales || !c->v_scales) return SLQ_EINVAL;
    if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->k_scales, 4) ||
        !aligned(c->v_scales, 4))
      return SLQ_EINVAL;
    const size_t all = (size_t)((c->pages - 1) * ps + span);
    const size_t sb = (size_t)(c->pages * c->heads) * sizeof(float);
    x->codes[0] = {c->k_codes, all};
    x->codes[1] = {c->v_codes, all};
    x->scales[0] = {c->k_scales, sb};
    x->scales[1] = {c->v_scales, sb};
    if (overlap(x->codes[0], x->codes[1])) {
      // K and V may alternate within one allocation, page by page
      const uintptr_t k = (uintptr_t)c->k_codes, w = (uintptr_t)c->v_codes;
      const int64_t apart = (int64_t)(k < w ? w - k : k - w);
      if (apart < span || ps < apart + span) return SLQ_EINVAL;
    }
    for (int i = 0; i < 2; ++i)
      for (int j = 0; j < 2; ++j)
        if (overlap(x->codes[i], x->scales[j])) return SLQ_EINVAL;
    if (overlap(x->scales[0], x->scales[1])) return SLQ_EINVAL;
  }
  *v = slq::KvView{{c->k_codes, c->v_codes}, {c->k_scales, c->v_scales}, ps, hs, ts, c->pages,
                   c->heads, c->head_dim, __builtin_ctz((unsigned)c->page_size)};
  return SLQ_OK;
}

struct SeqExtents {
  Extent e[3];
  bool hits(Extent x) const { return overlap(x, e[0]) || overlap(x, e[1]) || overlap(x, e[2]); }
};

slq_status check_seqs(const slq_kv_seqs *s, const slq_kv_cache *c, int64_t rows, int64_t heads,
                      slq::SeqView *v, SeqExtents *x) {
  if (!s || s->batch < 0 || s->batch > kMaxBatch || rows < 0 || rows * heads >= kMaxRows ||
      rows >= kMaxRows)
    return SLQ_EINVAL;
  if (s->max_pages < 1 || (int64_t)s->max_pages * c->page_size > kMaxRows ||
      s->table_stride < s->max_pages || s->table_stride >= kMaxStride)
    return SLQ_EINVAL;
  *x = SeqExtents{};
  if (s->batch > 0) {
    if (!s->table || !s->lens || !s->cu) return SLQ_EINVAL;
    if (!aligned(s->table, 4) || !aligned(s->lens, 4) || !aligned(s->cu, 4)) return SLQ_EINVAL;
    x->e[0] = {s->table, ((size_t)(s->batch - 1) * s->table_stride + s->max_pages) * 4};
    x->e[1] = {s->lens, (size_t)s->batch * 4};
    x->e[2] = {s->cu, (size_t)(s->batch + 1) * 4};
  }
  *v = slq::SeqView{s->table, s->lens, s->cu, s->table_stride, s->batch, s->max_pages,
                    (int32_t)rows};
  return SLQ_OK;
}

// A strided [rows][heads][dim] input.
slq_status check_rows(const void *p, slq_dtype t, int64_t rows, int64_t heads, int64_t dim,
                      int64_t row_stride, int64_t head_stride, Extent *x) {
  const int64_t eb = (int64_t)elem_bytes(t);
  if (row_stride < 0 || head_stride < 0 || row_stride >= kMaxStride / 64 ||
      head_stride >= kMaxStride / 64 || row_stride * eb % 16 || head_stride * eb % 16)
    return SLQ_EINVAL;
  if (rows > 0 && (!p || !aligned(p, 16))) return SLQ_EINVAL;
  *x = {p, rows == 0 ? 0
                     : (size_t)(((rows - 1) * row_stride + (heads - 1) * head_stride + dim) * eb)};
  return SLQ_OK;
}

struct AttnChecked {
  slq::KvView c;
  slq::SeqView s;
  CacheExtents cx;
  SeqExtents sx;
  slq::KvAttnPlan plan;
};
slq_status check_attn(const slq_kv_cache *cache, const slq_kv_seqs *seqs, int64_t rows,
                      int32_t heads_q, int32_t window, int64_t max_q, int64_t max_len,
                      AttnChecked *o) {
  slq_status st = check_cache(cache, &o->c, &o->cx);
  if (st != SLQ_OK) return st;
  if (heads_q < 1 || heads_q > 65536 || heads_q % cache->heads || window < 0 || max_q < 1 ||
      max_len < 1)
    return SLQ_EINVAL;
  st = check_seqs(seqs, cache, rows, heads_q, &o->s, &o->sx);
  if (st != SLQ_OK) return st;
  o->plan = slq::KvAttnPlan{};
  if (seqs->batch > 0 && rows > 0)
    o->plan = slq::kv_attn_plan(seqs->batch, cache->heads, cache->head_dim,
                                (int64_t)seqs->max_pages * cache->page_size, rows, heads_q, window,
                                max_q, max_len);
  return SLQ_OK;
}

}  // namespace

extern "C" {

slq_status slq_kv_write(const slq_kv_cache *cache, const slq_kv_seqs *seqs, const void *k,
                        const void *v, slq_dtype dtype, int64_t rows, int64_t k_row_stride,
                        int64_t k_head_stride, int64_t v_row_stride, int64_t v_head_stride,
                        int64_t max_new, slq_stream stream) {
  slq::KvView c;
  slq::SeqView s;
  CacheExtents cx;
  SeqExtents sx;
  slq_status st = check_cache(cache, &c, &cx);
  if (st != SLQ_OK) return st;
  if (!dtype_ok(dtype) || max_new < 1) return SLQ_EINVAL;
  st = check_seqs(seqs, cache, rows, cache->heads, &s, &sx);
  if (st != SLQ_OK) return st;
  Extent kx, vx;
  st = check_rows(k, dtype, rows, c.heads, c.dim, k_row_stride, k_head_stride, &kx);
  if (st == SLQ_OK) st = check_rows(v, dtype, rows, c.heads, c.dim, v_row_stride, v_head_stride, &vx);
  if (st != SLQ_OK) return st;
  if (cx.hits(kx) || cx.hits(vx)) return SLQ_EINVAL;
  for (const Extent &e : sx.e)
    if (cx.hits(e)) return SLQ_EINVAL;
  if (rows == 0 || s.batch == 0 || c.pages == 0) return SLQ_OK;
  return from_hip(slq::launch_kv_write(c, s, cache->format == SLQ_KV_E4M3, k, v, (int)dtype,
                                       k_row_stride, k_head_stride, v_row_stride, v_head_stride,
                                       max_new, static_cast<hipStream_t>(stream)));
}

slq_status slq_kv_read(const slq_kv_cache *cache, const slq_kv_seqs *seqs, void *k_out, void *v_out,
                       slq_dtype dtype, int64_t rows, int64_t max_rows, slq_stream stream) {
  slq::KvView c;
  slq::SeqView s;
  CacheExtents cx;
  SeqExtents sx;
  slq_status st = check_cache(cache, &c, &cx);
  if (st != SLQ_OK) return st;
  if (!dtype_ok(dtype) || max_rows < 1) return SLQ_EINVAL;
  st = check_seqs(seqs, cache, rows, cache->heads, &s, &sx);
  if (st != SLQ_OK) return st;
  const int64_t row = (int64_t)c.heads * c.dim;
  Extent kx, vx;
  st = check_rows(k_out, dtype, rows, c.heads, c.dim, row, c.dim, &kx);
  if (st == SLQ_OK) st = check_rows(v_out, dtype, rows, c.heads, c.dim, row, c.dim, &vx);
  if (st != SLQ_OK) return st;
  if (cx.hits(kx) || cx.hits(vx) || sx.hits(kx) || sx.hits(vx) || overlap(kx, vx)) return SLQ_EINVAL;
  if (rows == 0 || s.batch == 0) return SLQ_OK;
  return from_hip(slq::launch_kv_read(c, s, cache->format == SLQ_KV_E4M3, k_out, v_out, (int)dtype,
                                      max_rows, static_cast<hipStream_t>(stream)));
}

size_t slq_kv_attention_workspace_bytes(const slq_kv_cache *cache, const slq_kv_seqs *seqs,
                                        int64_t rows, int32_t heads_q, int32_t window,
                                        int64_t max_q, int64_t max_len) {
  AttnChecked a;
  if (check_attn(cache, seqs, rows, heads_q, window, max_q, max_len, &a) != SLQ_OK) return 0;
  return a.plan.ws_bytes;
}

slq_status slq_kv_attention(const slq_kv_cache *cache, const slq_kv_seqs *seqs, const void *q,
                            slq_dtype dtype, int64_t rows, int32_t heads_q, int64_t q_row_stride,
                            int64_t q_head_stride, float scale, int32_t window, int64_t max_q,
                            int64_t max_len, void *out, float *lse, void *workspace,
                            slq_stream stream) {
  AttnChecked a;
  slq_status st = check_attn(cache, seqs, rows, heads_q, window, max_q, max_len, &a);
  if (st != SLQ_OK) return st;
  if (!dtype_ok(dtype) || !std::isfinite(scale)) return SLQ_EINVAL;
  if (dtype == SLQ_F32) return SLQ_ENOTSUP;
  const int64_t dim = a.c.dim;
  Extent qx, ox;
  st = check_rows(q, dtype, rows, heads_q, dim, q_row_stride, q_head_stride, &qx);
  if (st == SLQ_OK) st = check_rows(out, dtype, rows, heads_q, dim, heads_q * dim, dim, &ox);
  if (st != SLQ_OK) return st;
  const Extent lx{lse, (size_t)(rows * heads_q) * sizeof(float)}, wx{workspace, a.plan.ws_bytes};
  if (!aligned(lse, 4)) return SLQ_EINVAL;
  if (wx.n > 0 && (!workspace || !aligned(workspace, 256))) return SLQ_EINVAL;
  const Extent outs[3] = {ox, lx, wx};
  for (int i = 0; i < 3; ++i) {
    if (overlap(outs[i], qx) || a.cx.hits(outs[i]) || a.sx.hits(outs[i])) return SLQ_EINVAL;
    for (int j = i + 1; j < 3; ++j)
      if (overlap(outs[i], outs[j])) return SLQ_EINVAL;
  }
  if (rows == 0 || a.s.batch == 0) return SLQ_OK;
  slq::KvAttnArgs k{};
  k.c = a.c;
  k.s = a.s;
  k.q = static_cast<const uint16_t *>(q);
  k.q_row = q_row_stride;
  k.q_head = q_head_stride;
  k.out = static_cast<uint16_t *>(out);
  k.lse = lse;
  k.scale_log2 = (float)((double)scale * 1.4426950408889634);
  k.window = window;
  k.group = heads_q / a.c.heads;
  k.heads_q = heads_q;
  k.bf16 = dtype == SLQ_BF16;
  return from_hip(slq::launch_kv_attention(k, cache->format == SLQ_KV_E4M3, a.plan, workspace,
                                           static_cast<hipStream_t>(stream)));
}

static bool sample_dims_ok(int64_t rows, int64_t vocab) {
  return rows >= 0 && rows < ((int64_t)1 << 22) && vocab >= 1 && vocab <= ((int64_t)1 << 24);
}

size_t slq_sample_workspace_bytes(int64_t rows, int64_t vocab) {
  if (!sample_dims_ok(rows, vocab) || rows == 0) return 0;
  return slq::sample_workspace(rows, vocab);
}

slq_status slq_sample(const void *logits, slq_dtype dtype, int64_t rows, int64_t vocab,
                      int64_t row_stride, const float *u, const float *temperature,
                      const int32_t *top_k, const float *top_p, const float *min_p,
                      int32_t *tokens, float *logprobs, void *workspace, slq_stream stream) {
  if (!dtype_ok(dtype) || !sample_dims_ok(rows, vocab)) return SLQ_EINVAL;
  const size_t eb = elem_bytes(dtype);
  if (row_stride < 0 || row_stride >= kMaxStride) return SLQ_EINVAL;
  if (rows == 0) return SLQ_OK;
  const size_t wsb = slq_sample_workspace_bytes(rows, vocab);
  if (!logits || !u || !tokens) return SLQ_EINVAL;
  if (!aligned(logits, eb) || !aligned(u, 4) || !aligned(temperature, 4) || !aligned(top_k, 4) ||
      !aligned(top_p, 4) || !aligned(min_p, 4) || !aligned(tokens, 4) || !aligned(logprobs, 4))
    return SLQ_EINVAL;
  if (wsb > 0 && (!workspace || !aligned(workspace, 256))) return SLQ_EINVAL;
  const size_t rb = (size_t)rows * 4;
  const Extent in[6] = {{logits, ((size_t)((rows - 1) * row_stride + vocab)) * eb}, {u, rb},
                        {temperature, rb}, {top_k, rb}, {top_p, rb}, {min_p, rb}};
  const Extent out[3] = {{tokens, rb}, {logprobs, rb}, {workspace, wsb}};
  for (int i = 0; i < 3; ++i) {
    for (const Extent &e : in)
      if (overlap(out[i], e)) return SLQ_EINVAL;
    for (int j = i + 1; j < 3; ++j)
      if (overlap(out[i], out[j])) return SLQ_EINVAL;
  }
  const slq::SampleArgs a{logits, rows, vocab, row_stride, u, temperature, top_k, top_p, min_p,
                          tokens, logprobs};
  return from_hip(slq::launch_sample(a, (int)dtype, workspace, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
