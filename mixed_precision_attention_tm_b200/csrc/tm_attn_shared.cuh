// tm_attn_shared.cuh -- what the kernels of tm_attn_shared_prefix share: the
// launch's arguments, its split of the work and the form of partial results.
//
// Query heads of one K/V head and consecutive tokens are packed into rows:
// row r of a sequence (or of the whole batch, for the prefix) is token r / g,
// query head kv_head * g + r % g, g = Hq / Hkv, so that every byte of K and V
// is used for all rows that see it.  Keys are cut into ranges ("splits"); a
// split's result for a row is (O, m, l): the running maximum m of its scores
// in powers of two, l = sum 2^(s - m + kPOffset) and O = the same sum of
// weighted values, fp32.  One slot of the workspace holds one split's results
// of all rows, prefix splits first; results join as
//   out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i,  M = max m_i.
#pragma once

#include "tm_paged.cuh"

namespace tmk {

constexpr int kSmsB200 = 148;

// P is rounded to fp16 for the P.V product.  Its largest value is 2^kPOffset
// instead of 1, which keeps weights down to 2^-20 of the largest normal fp16
// numbers, and even with an INT8 cache's V scale (at most 65504 / 127 = 516 for
// values fp16 holds) multiplied in, below fp16's 65504.
constexpr float kPOffset = 6.0f;

struct SharedPlan {
  int group;                  // query heads per K/V head
  int own_rows, pre_rows;     // row blocks (of 16 rows) per sequence, of the batch
  int own_splits, pre_splits;
  int own_chunk, pre_chunk;   // keys per split
  int slots;                  // own_splits + pre_splits
  int64_t ml_bytes, bytes;    // workspace: (m, l) of every slot and row, then O
};

SharedPlan shared_plan(int64_t T, int32_t Hq, int32_t Hkv, int32_t d, int32_t batch, int64_t max_seqlen,
                       int64_t prefix_len, int64_t max_kv_len);

struct SharedArgs {
  const __half* q;
  int64_t q_t, q_h;
  __half* out;
  int64_t o_t, o_h;
  PagedPool pool;
  PageTable pt;
  const int32_t *kv_lens, *cu, *prefix_pages;
  int64_t T, per_seq, prefix_len, max_kv;
  int batch, causal;
  SharedPlan plan;
  float2* ml;     // [slots][T * Hq]
  float* o;       // [slots][T * Hq][d]
  float scale_log2;
};

__device__ __forceinline__ void seq_rows(const SharedArgs& a, int b, int64_t& start, int64_t& n) {
  if (a.cu != nullptr) {
    start = __ldg(a.cu + b);
    n = __ldg(a.cu + b + 1) - start;
  } else {
    start = b * a.per_seq;
    n = a.per_seq;
  }
}

__device__ __forceinline__ int64_t rows_in_use(const SharedArgs& a) {
  const int64_t n = a.cu != nullptr ? static_cast<int64_t>(__ldg(a.cu + a.batch)) : a.T;
  return n < a.T ? n : a.T;
}

}  // namespace tmk
