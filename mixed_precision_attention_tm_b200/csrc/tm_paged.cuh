// tm_paged.cuh -- addressing of the paged K/V cache, shared by the kernels
// that write it, read it back and attend over it, and by the host checks.
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/tm.h"
#include "tm_device.cuh"

namespace tmk {

// What a kernel needs of a tm_paged_kv, page size as a shift.
struct PagedPool {
  uint8_t *k, *v;
  __half *ks, *vs;
  int64_t stride_page, stride_t, stride_h;      // bytes
  int64_t sstride_page, sstride_t, sstride_h;   // elements of the scales
  int32_t num_pages, page_shift, H;
};

struct PageTable {
  const int32_t* table;
  int64_t stride;
  int32_t cols, page_shift, num_pages;
};

// Column of own position j, and whether it and the page there may be used.
__host__ __device__ __forceinline__ bool page_column_ok(int64_t j, int32_t cols, int32_t page_shift) {
  return j >= 0 && (j >> page_shift) < cols;
}
__host__ __device__ __forceinline__ bool page_ok(int32_t page, int32_t num_pages) {
  return page >= 0 && page < num_pages;
}

// Page of own position j of sequence b, or -1 where the table or the page
// number does not allow it.
__host__ __device__ __forceinline__ int32_t page_of(const PageTable& t, int b, int64_t j) {
  if (!page_column_ok(j, t.cols, t.page_shift)) return -1;
  const int32_t page = t.table[b * t.stride + (j >> t.page_shift)];
  return page_ok(page, t.num_pages) ? page : -1;
}

// Number of sequences that end at or before row t of a packed batch: the
// sequence that holds row t, or `batch` behind the last one.  cu is
// non-decreasing (empty sequences count as ended), so each round of 32
// pivots, one per lane, leaves one 32nd of the range; a batch of up to 32
// sequences takes one load.  All lanes of the warp call it with the same t.
__device__ __forceinline__ int sequence_of(const int32_t* __restrict__ cu, int batch, int64_t t) {
  const int lane = threadIdx.x & 31;
  int lo = 0, n = batch;                  // the answer lies in lo .. lo + n
  while (n > 0) {
    const int step = (n + 31) / 32;
    const int i = lo + lane * step + step - 1;            // last sequence of this lane's share
    const bool ended = i < lo + n && __ldg(cu + i + 1) <= t;
    const int full = __popc(__ballot_sync(0xffffffffu, ended));
    const int at = lo + full * step;
    if (step == 1) return at < lo + n ? at : lo + n;
    n = lo + n - at;
    if (n > step - 1) n = step - 1;
    if (n < 0) n = 0;
    lo = at;
  }
  return lo;
}

// Host side (tm_paged.cu): checks a cache descriptor and fills the kernels'
// form of it.
tm_status paged_pool(const tm_paged_kv* c, PagedPool* p, bool* int8);
tm_status page_table(const PagedPool& p, const int32_t* table, int64_t stride, int32_t cols, PageTable* t);
// A THD fp16 operand: pointer, alignment and strides as tm.h asks.
bool thd_ok(const tm_tensor* x, int64_t T, int64_t H, int64_t d);
// The same for an operand that is written: no two of its elements share memory.
bool thd_out_ok(const tm_tensor* x, int64_t T, int64_t H, int64_t d);

}  // namespace tmk
