// The paged cache and the ragged batch as the kernels see them, and the index
// arithmetic that keeps every access inside them whatever the device arrays
// (lengths, row offsets, page numbers) hold.  Plain C++, so that it can be
// built and tested on the host.
#pragma once
#include <stdint.h>

#if defined(__HIP__) || defined(__HIPCC__)
#include <hip/hip_runtime.h>
#define SLQ_HD __host__ __device__ __forceinline__
#else
#define SLQ_HD inline
#endif

namespace slq {

struct KvView {
  uint8_t *codes[2];      // K, V
  float *scales[2];       // [pages][heads]
  int64_t page_stride, head_stride, token_stride;
  int64_t pages;
  int32_t heads, dim;
  int32_t shift;          // page_size = 1 << shift
};

struct SeqView {
  const int32_t *table, *lens, *cu;
  int64_t table_stride;
  int32_t batch, max_pages;
  int32_t rows;
};

// A sequence's rows in the caller's arrays and its positions in the cache.
struct KvSpan {
  int32_t row0, n;   // rows row0 .. row0 + n - 1
  int32_t pos0;      // position of row0 (negative: that row does not exist)
  int32_t len;       // tokens that can exist: 0 .. len - 1, len <= capacity
};

SLQ_HD int32_t kv_clamp(int32_t v, int32_t lo, int32_t hi) { return v < lo ? lo : v > hi ? hi : v; }

SLQ_HD KvSpan kv_span(const SeqView &s, int32_t shift, int32_t b) {
  KvSpan r;
  r.row0 = kv_clamp(s.cu[b], 0, s.rows);
  r.n = kv_clamp(s.cu[b + 1], r.row0, s.rows) - r.row0;
  const int32_t len = s.lens[b] < 0 ? 0 : s.lens[b];
  r.pos0 = len - r.n;
  r.len = kv_clamp(len, 0, s.max_pages << shift);
  return r;
}

// The table entry to read for tokens p << shift .. (any p: always inside the
// table), and the page that the entry read there stands for, or -1.
SLQ_HD int64_t kv_entry(const SeqView &s, int32_t b, int32_t p) {
  return (int64_t)b * s.table_stride + kv_clamp(p, 0, s.max_pages - 1);
}
SLQ_HD int32_t kv_page_of(const SeqView &s, int64_t pages, int32_t p, int32_t entry) {
  return p >= 0 && p < s.max_pages && entry >= 0 && entry < pages ? entry : -1;
}
SLQ_HD int32_t kv_page(const SeqView &s, int64_t pages, int32_t b, int32_t p) {
  return kv_page_of(s, pages, p, s.table[kv_entry(s, b, p)]);
}

// The new slots [lo, hi) of page p of a sequence (empty: lo >= hi), and the
// caller's row of slot lo.
struct KvPart {
  int32_t lo, hi, row;
};
SLQ_HD KvPart kv_part(const KvSpan &s, int32_t shift, int32_t p) {
  const int64_t base = (int64_t)p << shift;
  const int64_t first = s.pos0 > 0 ? s.pos0 : 0;
  const int64_t end = (int64_t)s.pos0 + s.n;
  KvPart r;
  r.lo = (int32_t)(first > base ? first - base : 0);
  const int64_t hi = end - base, size = (int64_t)1 << shift;
  r.hi = (int32_t)(hi < 0 ? 0 : hi < size ? hi : size);
  r.row = (int32_t)(s.row0 + (base + r.lo - s.pos0));
  return r;
}

// Pages that hold the existing new rows: first .. last (none: last < first).
SLQ_HD int32_t kv_first_page(const KvSpan &s, int32_t shift) {
  return (s.pos0 > 0 ? s.pos0 : 0) >> shift;
}
SLQ_HD int32_t kv_last_page(const KvSpan &s, int32_t shift) {
  const int32_t end = s.pos0 + s.n;
  return end <= 0 || s.n == 0 ? -1 : (end - 1) >> shift;
}

// Tokens [lo, hi) that at least one of a sequence's query rows i0..i1 can see.
struct KvRange {
  int32_t lo, hi;
};
SLQ_HD KvRange kv_visible(const KvSpan &s, int32_t window, int32_t i0, int32_t i1) {
  const int32_t end = s.pos0 + i1 + 1;
  KvRange r;
  r.hi = end < s.len ? (end > 0 ? end : 0) : s.len;
  const int32_t first = s.pos0 + i0;
  r.lo = window > 0 && first >= window ? first - window + 1 : 0;
  // an empty range lies within the tokens too: positions behind them reach 2^31,
  // where a walk in steps of a block would pass the range of int
  if (r.lo > r.hi) r.lo = r.hi;
  return r;
}

}  // namespace slq
