// Internal launchers of the serving operators (host code; arguments already
// validated) and the element types they share.
#pragma once
#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "kv_view.h"

namespace slq {

enum ElemType { kElemF32 = 0, kElemBf16 = 1, kElemF16 = 2 };

// kv_cache.hip.  Strides in elements.
hipError_t launch_kv_write(const KvView &c, const SeqView &s, bool e4m3, const void *k,
                           const void *v, int type, int64_t k_row, int64_t k_head, int64_t v_row,
                           int64_t v_head, int64_t max_new, hipStream_t st);
hipError_t launch_kv_read(const KvView &c, const SeqView &s, bool e4m3, void *k, void *v, int type,
                          int64_t max_rows, hipStream_t st);

// kv_attention.hip
struct KvAttnPlan {
  int nt;         // 16-query tiles per workgroup of the decode kernel; 0: prompt kernel
  int tiles;      // workgroups along a sequence's query rows
  bool wide;      // 8 waves per workgroup of the decode kernel
  int splits;     // workgroups along the tokens, at most
  int chunk;      // tokens per split, at least
  int grain;      // tokens that splits are multiples of
  int share;      // workgroups that share all tokens evenly (0: not split)
  int rows;       // query rows per kv head and sequence, as expected
  size_t ws_bytes;
};
KvAttnPlan kv_attn_plan(int batch, int heads, int dim, int64_t capacity, int64_t rows, int heads_q,
                        int window, int64_t max_q, int64_t max_len);
struct KvAttnArgs {
  KvView c;
  SeqView s;
  const uint16_t *q;
  int64_t q_row, q_head;   // elements
  uint16_t *out;
  float *lse;
  float *part_o;           // [splits][rows * heads_q][dim]
  float *part_lse;         // [splits][rows * heads_q], base 2
  float scale_log2;        // softmax scale * log2(e)
  int32_t window, group, heads_q;
  int32_t splits, chunk, grain, share, tiles, join_rows;
  int32_t heads_first;     // grid order of the decode kernel
  int32_t bf16;            // else binary16
};
hipError_t launch_kv_attention(KvAttnArgs a, bool e4m3, const KvAttnPlan &plan, void *ws,
                               hipStream_t st);

// sample.hip
struct SampleArgs {
  const void *logits;
  int64_t rows, vocab, row_stride;
  const float *u, *temperature;
  const int32_t *top_k;
  const float *top_p, *min_p;
  int32_t *tokens;
  float *logprobs;
};
size_t sample_workspace(int64_t rows, int64_t vocab);
hipError_t launch_sample(const SampleArgs &a, int type, void *ws, hipStream_t st);

}  // namespace slq
