// tm_attn_shared.cuh -- what the kernels of tm_attn_shared_prefix share: the
// launch's arguments, its split of the work and the form of partial results.
//
// Query heads of one K/V head and consecutive tokens are packed into rows:
// row r of a sequence (or of the whole batch, for the prefix) is token r / g,
// query head kv_head * g + r % g, g = Hq / Hkv, so that every byte of K and V
// is used for all rows that see it.  Keys are cut into ranges ("splits"); a
// split's result for a row is (O, m, l): a reference m of its scores in powers
// of two (a maximum of some time, less kPOffset), l = sum 2^(s - m) and O = the same sum
// of weighted values, fp32.  One slot of the workspace holds one split's results
// of all rows, prefix splits first; results join as
//   out = sum_i 2^(m_i - M) O_i / sum_i 2^(m_i - M) l_i,  M = max m_i.
#pragma once

#include <atomic>

#include "tm_host.h"
#include "tm_paged.cuh"

namespace tmk {

constexpr int kSmsB200 = 148;

// P is rounded to fp16 for the P.V product.  A weight is 2^kPOffset, not 1,
// where the score equals the row's reference, so that weights down to 2^-20 of
// that stay normal fp16 numbers; above the reference fp16 leaves 2^9 (2^8 where
// a part of INT8 V's scale is multiplied in), by which scores may pass it before
// it is raised.
constexpr float kPOffset = 6.0f;

// Which kernel takes the prefix, and which the own tokens.  The split-key
// kernel costs about 0.008 us for each 16-row block and key tile of 128; the tile
// kernel starts about 9 us later and costs 0.013 us for each 256-row block and key tile.
// Measured (32 query heads over 8, 32 tokens of single rows, fp16): behind 1024
// shared positions 15.8 us (split) and 19.4 us (tile), behind 8192 42.0 and 24.9 us.
constexpr int64_t kTileStart = 1000;      // in 16-row blocks and key tiles
constexpr bool prefix_on_tiles(int64_t blocks16, int64_t blocks256, int64_t key_tiles) {
  return 2 * blocks16 * key_tiles > 2 * kTileStart + 3 * blocks256 * key_tiles;
}
// A sequence's packed rows: a tile of few rows is mostly empty (60 sequences of
// 64 rows over 600 keys: 104 us split, 95 us on tiles; over 150 keys 67 and 70
// us; of 32 rows 105 and 149 us).
constexpr bool own_on_tiles(int64_t rows, int64_t key_tiles) { return rows > 64 || (rows > 48 && key_tiles > 4); }
// A short prefix is multiplied by every row block of the own tokens instead of
// once for the packed batch, which costs the tiles that packing saves and spares a
// pass, its results and the join (about 20 us, 1200 row blocks and key tiles: measured equal at 1248).
constexpr bool prefix_folded(int64_t own_blocks, int64_t packed_blocks, int64_t key_tiles) {
  return (own_blocks - packed_blocks) * key_tiles < 1200;
}
// Key tiles that an item of own tokens costs besides its own (first copies, way out), and a join.
constexpr int kItemTiles = 4;
constexpr int kMostSplits = 30;
// Key tiles that a row block's start and end cost a CTA of the tile kernel (about 6 us at 1.9 us a tile).
constexpr int kSplitBlockTiles = 3;

struct SharedPlan {
  int group;                  // query heads per K/V head
  int own_tile, pre_tile;     // 1: on the tile kernel (256-row blocks), 0: on the split-key kernel (16- or 8-row blocks)
  int own_rows, pre_rows;     // row blocks per sequence, of the batch
  int narrow;                 // split-key kernel: blocks of 8 rows, not 16
  int own_splits, pre_splits; // most results of a row
  int own_chunk;              // keys per split
  int fold;                   // key tiles of the prefix that the own tokens' row blocks go through first (no prefix results)
  int pre_chunk;              // the same of the prefix; on the tile kernel: key tiles per CTA
  int pre_tiles, pre_ctas;    // tile kernel: key tiles of the prefix, CTAs
  int pre_pieces;             // tile kernel: pieces of a row block, 0: pieces of the whole line
  int slots;                  // own_splits + pre_splits
  int64_t ml_bytes, bytes;    // workspace: (m, l) of every slot and row, then O
};

// Split-key kernel: rows of a block, and CTAs that an SM holds (their rings; INT8 at d = 128 in blocks of 16: registers).
__host__ __device__ constexpr int split_block(bool narrow) { return narrow ? 8 : 16; }
constexpr int split_resident(int d, bool int8, bool narrow) { return d == 64 || (int8 && narrow) ? 4 : int8 ? 3 : 2; }

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

SharedPlan shared_plan(int64_t T, int32_t Hq, int32_t Hkv, int32_t d, bool int8, int32_t batch, int64_t max_seqlen,
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
__device__ __forceinline__ int64_t first_row(const SharedArgs& a) { return a.cu != nullptr ? __ldg(a.cu) : 0; }

// Whether a sequence has rows that the launch was not sized for.
__device__ __forceinline__ bool rows_outside(const SharedArgs& a, int64_t start, int64_t n, int block) {
  return start < 0 || n < 0 || start + n > a.T || n * a.plan.group > static_cast<int64_t>(a.plan.own_rows) * block;
}

// A kernel may be launched while the one before it in the stream still runs
// (after that one's pdl_launch_dependents); pdl_wait returns when that one has
// ended and its writes are visible.
__device__ __forceinline__ void pdl_launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

__device__ __forceinline__ void cp16(uint32_t dst, const void* src, bool real) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(real ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}
__device__ __forceinline__ uint4 lds128(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0,%1,%2,%3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
  return v;
}
__device__ __forceinline__ void sts128(uint32_t a, uint4 v) {
  asm volatile("st.shared.v4.b32 [%0], {%1,%2,%3,%4};" ::"r"(a), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// Two codes, as bytes code + 128 picked by `sel` from w, to a pair of fp16:
// under the exponent byte 0x64 a byte b reads as 1024 + b, exactly.
__device__ __forceinline__ uint32_t codes2(uint32_t w, uint32_t sel) {
  const uint32_t x = __byte_perm(w, 0x64646464u, sel);
  const __half2 v = __hsub2(*reinterpret_cast<const __half2*>(&x), __float2half2_rn(1152.0f));
  return *reinterpret_cast<const uint32_t*>(&v);
}

// How K and V pass through L2: keys that one row block alone reads make room
// first, so that the partial results stay for the join (64 tokens behind 32768
// positions: 78 us without the hint, 72 us with it); others stay for the next block.
__device__ __forceinline__ uint64_t keys_policy(int row_blocks) {
  uint64_t policy;
  if (row_blocks == 1) asm volatile("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(policy));
  else asm volatile("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(policy));
  return policy;
}
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, uint32_t bar, int32_t c0, int32_t c1,
                                            int32_t c2, int32_t c3, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.L2::cache_hint"
      " [%0], [%1, {%3, %4, %5, %6}], [%2], %7;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3), "l"(policy)
      : "memory");
}

// Dynamic shared memory of a kernel, allowed once for each device.
template <typename K>
tm_status prepare_smem(K kernel, int smem, std::atomic<uint64_t>& prepared) {
  int dev = 0;
  tm_status st = check_cuda(cudaGetDevice(&dev));
  if (st != TM_OK) return st;
  const uint64_t bit = 1ull << (dev & 63);
  if (prepared.load(std::memory_order_relaxed) & bit) return TM_OK;
  st = check_cuda(cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem));
  if (st == TM_OK) prepared.fetch_or(bit, std::memory_order_relaxed);
  return st;
}

// overlap: the kernel may start before the previous one of the stream has ended.
template <typename... P, typename... A>
tm_status launch_kernel(void (*kernel)(P...), int64_t blocks, int threads, int smem, bool overlap, cudaStream_t stream,
                        const A&... args) {
  if (blocks > 0x7fffffff) return TM_ERR_UNSUPPORTED;
  if (blocks <= 0) return TM_OK;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>(blocks));
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = overlap ? 1 : 0;
  return check_cuda(cudaLaunchKernelEx(&cfg, kernel, args...));
}

// TMA maps of a page pool, [page][slot or head][head or slot][d], for copies of
// `rows` slots of one head (64 columns of fp16, whole rows of codes).
struct PageMaps {
  CUtensorMap k, v;
  int ok;             // 0 where the driver has no map for the layout: rows are copied one by one
  int heads_inner;    // order of the middle dimensions: (heads, slots) or (slots, heads)
};
PageMaps page_maps(const PagedPool& pool, int d, bool int8, int rows);

// tm_attn_shared_tile.cu: the prefix's (or the own tokens') part on the tile kernel.
tm_status shared_tile(const SharedArgs& a, int d, bool int8, bool prefix, bool overlap, DevErr err,
                      cudaStream_t stream);

}  // namespace tmk
