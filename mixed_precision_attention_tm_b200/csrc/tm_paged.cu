// tm_paged.cu -- host checks of the paged K/V cache and tm_kv_gather, the
// cache's rows back in contiguous fp16 tensors for the prefill attention.
#include "tm_paged.cuh"

#include "tm_host.h"

namespace tmk {

bool thd_ok(const tm_tensor* x, int64_t T, int64_t H, int64_t d) {
  return x != nullptr && x->T == T && x->H == H && x->d == d && x->H > 0 && (x->data != nullptr || T == 0) &&
         (reinterpret_cast<uintptr_t>(x->data) & 15u) == 0 && (T <= 1 || (x->stride_t >= 0 && x->stride_t % 8 == 0)) &&
         (H <= 1 || (x->stride_h >= 0 && x->stride_h % 8 == 0));   // the stride of a lone row is never used
}

bool thd_out_ok(const tm_tensor* x, int64_t T, int64_t H, int64_t d) {
  if (!thd_ok(x, T, H, d)) return false;
  if (H > 1 && (T <= 1 || x->stride_h <= x->stride_t))      // heads within rows
    return x->stride_h >= d && (T <= 1 || x->stride_t >= (H - 1) * x->stride_h + d);
  return T <= 1 || (x->stride_t >= d && (H <= 1 || x->stride_h >= (T - 1) * x->stride_t + d));
}

tm_status paged_pool(const tm_paged_kv* c, PagedPool* p, bool* int8) {
  if (c == nullptr || c->k == nullptr || c->v == nullptr || c->num_pages <= 0 || c->H <= 0) return TM_ERR_INVALID_ARG;
  if ((c->k_scales == nullptr) != (c->v_scales == nullptr)) return TM_ERR_INVALID_ARG;
  *int8 = c->k_scales != nullptr;
  const int64_t e = *int8 ? 1 : 2;
  if ((reinterpret_cast<uintptr_t>(c->k) | reinterpret_cast<uintptr_t>(c->v)) & 15u) return TM_ERR_INVALID_ARG;
  if (c->stride_page <= 0 || c->stride_t <= 0 || c->stride_h <= 0) return TM_ERR_INVALID_ARG;
  if ((c->stride_page * e) % 16 || (c->stride_t * e) % 16 || (c->stride_h * e) % 16) return TM_ERR_INVALID_ARG;
  if (*int8) {
    if ((reinterpret_cast<uintptr_t>(c->k_scales) | reinterpret_cast<uintptr_t>(c->v_scales)) & 1u)
      return TM_ERR_INVALID_ARG;
    if (c->scale_stride_page <= 0 || c->scale_stride_t <= 0 || c->scale_stride_h <= 0) return TM_ERR_INVALID_ARG;
  }
  if (c->d != 64 && c->d != 128) return TM_ERR_UNSUPPORTED;
  int shift = 0;
  while ((1 << shift) < c->page_size && shift < 9) ++shift;
  if (c->page_size != (1 << shift) || shift < 4 || shift > 8) return TM_ERR_UNSUPPORTED;
  p->k = static_cast<uint8_t*>(c->k);
  p->v = static_cast<uint8_t*>(c->v);
  p->ks = static_cast<__half*>(c->k_scales);
  p->vs = static_cast<__half*>(c->v_scales);
  p->stride_page = c->stride_page * e;
  p->stride_t = c->stride_t * e;
  p->stride_h = c->stride_h * e;
  p->sstride_page = c->scale_stride_page;
  p->sstride_t = c->scale_stride_t;
  p->sstride_h = c->scale_stride_h;
  p->num_pages = c->num_pages;
  p->page_shift = shift;
  p->H = c->H;
  return TM_OK;
}

tm_status page_table(const PagedPool& p, const int32_t* table, int64_t stride, int32_t cols, PageTable* t) {
  if (table == nullptr || (reinterpret_cast<uintptr_t>(table) & 3u) || cols <= 0 || stride < 0)
    return TM_ERR_INVALID_ARG;
  t->table = table;
  t->stride = stride;
  t->cols = cols;
  t->page_shift = p.page_shift;
  t->num_pages = p.num_pages;
  return TM_OK;
}

namespace {

constexpr int kGatherWarps = 8;

// 16 codes times their row's scale, each product exact in fp32 and rounded once.
__device__ __forceinline__ void scaled16(uint4 c, float s, uint4& lo, uint4& hi) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
  uint32_t o[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const char4 b = *reinterpret_cast<const char4*>(&w[i]);
    o[2 * i] = pack_half2(b.x * s, b.y * s);
    o[2 * i + 1] = pack_half2(b.z * s, b.w * s);
  }
  lo = make_uint4(o[0], o[1], o[2], o[3]);
  hi = make_uint4(o[4], o[5], o[6], o[7]);
}

// A warp takes R consecutive rows of the packed tensors.  Their sequences,
// places and pages are looked up side by side, one row per lane; then the rows'
// 16-byte pieces of K and V lie across the lanes, several loads in flight before
// the first store.  The kernel moves bytes only: what bounds it is HBM (each byte
// read and written once).  Four rows where a row has at most 64 pieces of K
// and there are rows enough for two blocks per SM (36000 rows, 2 heads of 64: 6.6 us
// against 12.5 with one row; INT8, 4 heads of 128: 19.1 and 25.6), else one (8 heads
// of 128: 86.6 us, 0.98 of the copy bandwidth, against 90.8 with four; 1800
// rows of 8 heads of 64: 2.9 and 4.2).
template <int D, bool INT8, int R>
__global__ void __launch_bounds__(kGatherWarps * 32, 4)
kv_gather_kernel(PagedPool pool, PageTable pt, const int32_t* __restrict__ cu, int batch, int64_t T, int H,
                 __half* __restrict__ ko, int64_t k_st, int64_t k_sh, __half* __restrict__ vo, int64_t v_st,
                 int64_t v_sh, DevErr err) {
  const int64_t t0 = (static_cast<int64_t>(blockIdx.x) * kGatherWarps + (threadIdx.x >> 5)) * R;
  const int lane = threadIdx.x & 31;
  if (t0 >= T) return;
  // lane r (any lane with R = 1): where row t0 + r lies in the pool (-1: nowhere, or not to be written)
  int64_t mine = -1, my_scale = 0;
  {
    int b = sequence_of(cu, batch, t0);
    const int64_t t = t0 + (R == 1 ? 0 : lane);
    if (t < T && (R == 1 || lane < R)) {
      if (R > 1)
        while (b < batch && __ldg(cu + b + 1) <= t) ++b;
      const int64_t j = b < batch ? t - __ldg(cu + b) : -1;      // negative before the first sequence, too
      if (j >= 0) {
        const int32_t page = page_of(pt, b, j);
        if (page < 0) {
          if (R > 1 || lane == 0) dev_error(err, TM_DEVERR_SEQLEN);
        } else {
          const int64_t slot = j & ((1 << pt.page_shift) - 1);
          mine = page * pool.stride_page + slot * pool.stride_t;
          my_scale = page * pool.sstride_page + slot * pool.sstride_t;
        }
      }
    }
    if (R == 1 && mine < 0) return;
  }
  constexpr int CPH = INT8 ? D / 16 : D / 8;   // 16-byte pieces of a head
  const int n = H * CPH;                       // of a row
  constexpr int U = INT8 && R > 1 ? 2 : 4;
  for (int c0 = 0; c0 < R * n; c0 += 32 * U) {
    uint4 a[U], w[U];
    int64_t sat[U];       // INT8: where the scales lie
    bool real[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = c0 + u * 32 + lane;
      const int r = R == 1 ? 0 : static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(n)), c = i - r * n;
      const int64_t row = R == 1 ? mine : __shfl_sync(0xffffffffu, mine, r & 31);
      const int64_t srow = !INT8 || R == 1 ? my_scale : __shfl_sync(0xffffffffu, my_scale, r & 31);
      real[u] = false;
      if (i < R * n && row >= 0) {
        const int h = c / CPH;
        const int64_t src = row + h * pool.stride_h + (c % CPH) * 16;
        a[u] = __ldcs(reinterpret_cast<const uint4*>(pool.k + src));
        w[u] = __ldcs(reinterpret_cast<const uint4*>(pool.v + src));
        if (INT8) {
          sat[u] = srow + h * pool.sstride_h;
        }
        real[u] = true;
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (!real[u]) continue;
      const int i = c0 + u * 32 + lane;
      const int r = R == 1 ? 0 : static_cast<int>(static_cast<uint32_t>(i) / static_cast<uint32_t>(n));
      const int c = i - r * n, h = c / CPH;
      const int e = (c % CPH) * (INT8 ? 16 : 8);
      uint4* kd = reinterpret_cast<uint4*>(ko + (t0 + r) * k_st + h * k_sh + e);
      uint4* vd = reinterpret_cast<uint4*>(vo + (t0 + r) * v_st + h * v_sh + e);
      if (INT8) {
        uint4 lo, hi;
        scaled16(a[u], __half2float(pool.ks[sat[u]]), lo, hi);
        kd[0] = lo;
        kd[1] = hi;
        scaled16(w[u], __half2float(pool.vs[sat[u]]), lo, hi);
        vd[0] = lo;
        vd[1] = hi;
      } else {
        *kd = a[u];
        *vd = w[u];
      }
    }
  }
}

}  // namespace
}  // namespace tmk

extern "C" tm_status tm_block_table_check(const int32_t* table_host, int64_t table_stride, int32_t table_cols,
                                          const int32_t* kv_lens_host, int32_t batch, int32_t num_pages,
                                          int32_t page_size, int32_t* bad) {
  if (table_host == nullptr || kv_lens_host == nullptr || batch < 0 || table_cols <= 0 || num_pages <= 0 ||
      table_stride < 0)
    return TM_ERR_INVALID_ARG;
  int shift = 0;
  while ((1 << shift) < page_size && shift < 9) ++shift;
  if (page_size != (1 << shift) || shift < 4 || shift > 8) return TM_ERR_UNSUPPORTED;
  const tmk::PageTable t{table_host, table_stride, table_cols, shift, num_pages};
  for (int b = 0; b < batch; ++b) {
    for (int64_t j = 0; j < kv_lens_host[b]; j += page_size) {
      if (tmk::page_of(t, b, j) >= 0) continue;
      if (bad != nullptr) {
        bad[0] = b;
        bad[1] = static_cast<int32_t>(j >> shift);
      }
      return TM_ERR_INVALID_ARG;
    }
  }
  return TM_OK;
}

extern "C" tm_status tm_kv_gather(const tm_paged_kv* cache, const int32_t* table, int64_t table_stride,
                                  int32_t table_cols, const int32_t* cu_seqlens_k, int32_t batch, tm_tensor* k_out,
                                  tm_tensor* v_out, void* stream) {
  using namespace tmk;
  PagedPool pool;
  PageTable pt;
  bool int8 = false;
  tm_status st = paged_pool(cache, &pool, &int8);
  if (st != TM_OK) return st;
  st = page_table(pool, table, table_stride, table_cols, &pt);
  if (st != TM_OK) return st;
  if (cu_seqlens_k == nullptr || (reinterpret_cast<uintptr_t>(cu_seqlens_k) & 3u) || batch <= 0 || k_out == nullptr)
    return TM_ERR_INVALID_ARG;
  const int64_t T = k_out->T;
  if (cache->H > 65536) return TM_ERR_UNSUPPORTED;
  if (T < 0 || !thd_out_ok(k_out, T, cache->H, cache->d) || !thd_out_ok(v_out, T, cache->H, cache->d))
    return TM_ERR_INVALID_ARG;
  if (T == 0) return TM_OK;
  const int pieces = cache->H * cache->d / (int8 ? 16 : 8);
  const int rows = pieces <= 64 && T >= 2 * 148 * 4 * kGatherWarps ? 4 : 1;
  const int64_t blocks = (T + kGatherWarps * rows - 1) / (kGatherWarps * rows);
  if (blocks > 0x7fffffff) return TM_ERR_UNSUPPORTED;
  const DevErr err{device_error_word()};
  if (err.word == nullptr) return cuda_fail(static_cast<int>(cudaErrorInvalidSymbol));
  auto kernel = cache->d == 128 ? (int8 ? (rows == 4 ? kv_gather_kernel<128, true, 4> : kv_gather_kernel<128, true, 1>)
                                        : (rows == 4 ? kv_gather_kernel<128, false, 4> : kv_gather_kernel<128, false, 1>))
                                : (int8 ? (rows == 4 ? kv_gather_kernel<64, true, 4> : kv_gather_kernel<64, true, 1>)
                                        : (rows == 4 ? kv_gather_kernel<64, false, 4> : kv_gather_kernel<64, false, 1>));
  kernel<<<static_cast<unsigned>(blocks), kGatherWarps * 32, 0, as_stream(stream)>>>(
      pool, pt, cu_seqlens_k, batch, T, cache->H, static_cast<__half*>(k_out->data), k_out->stride_t, k_out->stride_h,
      static_cast<__half*>(v_out->data), v_out->stride_t, v_out->stride_h, err);
  return check_cuda(cudaGetLastError());
}
