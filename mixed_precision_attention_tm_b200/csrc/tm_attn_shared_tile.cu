// tm_attn_shared_tile.cu -- attention over a paged cache for many rows
// (tm_attn_shared_prefix): 256 packed rows of one K/V head against a range of
// keys on tcgen05, K and V gathered from their pages on the way in.
//
// One CTA holds two 128-row query tiles, whose softmax warpgroups alternate on
// the tensor core; a tile's 128 score columns are two 64-key halves, and
// S(c + 2) follows P.V(c) into the half that P(c) leaves, so the next scores are
// computed while the softmax works on the current ones.  O stays in tensor
// memory over the whole range; a row's reference maximum is raised (and O
// rescaled) only when a weight would exceed 2^kTopTile.
//
// Loads: one warp brings K and V with a TMA copy for each page (or 128 slots of
// it) into the 128-byte-swizzled layout that the MMAs read, through a ring of
// 128 KB.  A tile that the range ends in, or with a page that cannot be used,
// is copied row by row (cp.async) instead, the rows past the end as zeros, so
// that nothing behind a sequence's end is ever used.
//
// INT8 pages: the copies bring the codes, which two more warpgroups (one
// for K, one for V) turn into fp16 in place, exactly: K stays codes, V is code
// times the largest power of two in its scale, up to 2^8 (a code is 128 at most:
// fp16 holds 2^15).  A key's K scale multiplies its scores in fp32 and the rest of
// its V scale (between 1 and 2, of scales from 512 on up to 256) its weight before
// that is rounded, so that the scales add no rounding.  (V rounded to fp16
// (code * scale) is a shared-memory pass less, and 1.2 times the error.)
//
// The prefix's work is cut into equal pieces of key tiles, one for each SM, so
// that all finish together: pieces of every row block where that divides well,
// else of one line of key tiles, row block by row block, on which a CTA whose
// piece crosses a row block's end writes one partial result for each block.
//
// Bounds, for a 64-key step of both tiles (d = 128): its MMAs take 1280 SM cycles (the
// score products read Q from shared memory again for every 64 keys), its
// exponentials on the special function unit alone 1024, the rest of the softmax a few hundred issue
// slots of each warp; together 1460 to 1550 cycles, about 1.2 PFLOP/s (7200 packed
// rows of 8 K/V heads behind 16384 positions: 400 us).  With few key tiles for a CTA
// its start (setup, first copies, cold instructions: 5 us) and its results (128 KB)
// count as much.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <atomic>

#include "tm_attn_shared.cuh"
#include "tm_host.h"

namespace tmk {
namespace {

// 2^kPOffset is the largest weight when the reference is the maximum (far from zero
// 1); scores above it are left alone up to this exponent: 2^15 at most, inside fp16, with
// what INT8 V scales multiply in (less than 2; where one of 64 keys multiplies in
// up to 256, these are left alone up to 7 less).
template <bool INT8>
constexpr float kTopTile = INT8 ? 14.0f : 15.0f;

// fp16 pages: an exponent is one FMA of an unrounded score product, a reference
// rounded (with INT8 pages both come from products rounded with the K scale).  Up to
// this distance from zero (in powers of two; fp16 scores reach 2^36) they differ
// by an eighth at most; a row whose reference lies further out has its products
// taken from that reference, which is exact for those that count.
constexpr float kFarScore = 4194304.0f;

// Of every 8 pairs of exponentials, how many run on the FMA pipe: the special
// function unit alone takes as long as the MMAs of a tile.  fp16, 7200 packed rows of 8
// K/V heads behind 16384 positions: 545 us a call with 0, 510 with 2, 520 with 3, 535 with 4 (in
// another run 510 with 1, 494 with 2, 500 with 3).  With INT8 pages the conversion
// warps want the same pipes: 1024 tokens of 4 K/V heads behind 16384 positions 374 us
// with 0, 379 with 1, 390 with 2.
template <bool INT8>
constexpr int kFmaPairs = INT8 ? 0 : 2;

template <int D, bool INT8>
struct CfgT {
  static constexpr int BM = 128, BN = 128;
  static constexpr int HALF = 128 * 128;               // one 64-column slab of a tile
  static constexpr int SLOT = BN * D * 2;              // an fp16 K or V tile
  static constexpr int NSLOT = 131072 / SLOT;          // 4 (d = 128) or 8 (d = 64)
  static constexpr int STAGES = NSLOT / 2 + 1;         // of scales
  static constexpr int Q_BYTES = BM * D * 2;
  static constexpr int OFF_SLOT = 2 * Q_BYTES;
  static constexpr int OFF_SCALE = OFF_SLOT + NSLOT * SLOT;         // INT8: [STAGES][2][128] scales
  static constexpr int OUT_COLS = INT8 ? 16 : 32;                   // of results on their way out, 32 rows of each softmax warp
  static constexpr int OFF_OUT = OFF_SCALE + (INT8 ? STAGES * 256 * 4 : 0);
  static constexpr int OFF_BAR = OFF_OUT + 8 * 32 * OUT_COLS * 4;
  static constexpr int SMEM = OFF_BAR + 512 + 1024;
  static constexpr uint32_t IDESC_S = idesc_f16(BM, 64, false);
  static constexpr uint32_t IDESC_PV = idesc_f16(BM, D, true);
  static constexpr int CODES = BN * D;                 // INT8: a K or V tile's codes, in the slot's upper half
  static constexpr int LOADED = INT8 ? CODES : SLOT;   // bytes that a tile's copies bring
  // Registers at launch, and after the split over softmax, control and (INT8) two conversion warpgroups.
  static constexpr int THREADS = INT8 ? 640 : 384, LAUNCH_REGS = INT8 ? 96 : 168;
  static constexpr int SOFTMAX_REGS = INT8 ? 152 : 216, CONTROL_REGS = INT8 ? 64 : 72, CONVERT_REGS = INT8 ? 56 : 0;
  static_assert(2 * 128 * SOFTMAX_REGS + 128 * CONTROL_REGS + 256 * CONVERT_REGS == THREADS * LAUNCH_REGS,
                "register split");
  static_assert(SMEM <= 232448, "shared memory per CTA");
  __host__ __device__ static constexpr uint32_t s_col(int t) { return 128u * t; }
  __host__ __device__ static constexpr uint32_t o_col(int t) { return 256u + D * t; }
};

enum {
  T_QFULL = 0,
  T_QEMPTY = 1,
  T_SFULL = 2,    // +4: 2 tiles x 2 halves
  T_ODONE = 6,    // +2
  T_DRAIN = 8,    // +2
  T_FULL = 10,    // +NSLOT
  T_EMPTY = 18,   // +NSLOT
  T_OLAST = 26,   // +2: a segment's last P.V (T_ODONE's parity cannot tell it from the one two before)
  T_CODES = 28,   // +NSLOT: INT8, a tile's codes landed
  T_COUNT = 36
};
// Named barriers: NB_P + 2 t + half softmax t -> issuer t (P stored); NB_KV + t
// wait helper -> issuer t (operands landed); NB_TURN + t the other softmax ->
// softmax t (its turn); NB_CVT the conversion warps.
enum : int { NB_P = 1, NB_KV = 5, NB_TURN = 7, NB_CVT = 9 };

// One row block against one range of keys (packed rows, keys and key tiles of
// the line all stay below 2^31).
struct Segment {
  int kvh, b, slot, rows;     // rows of the block: 1 .. 256
  int row0, start;            // first packed row (of the batch or the sequence), first token
  int key0;                   // first key: of the prefix, or of the prefix's whole tiles (where they are folded in) and own tokens behind them
  int lk;                     // own keys (of the prefix: its length)
  int hidden;                 // own, causal: token i of the sequence sees own keys below hidden + i
  int nj[2];                  // key tiles that each query tile sees
};

// 2^y for y <= 15 on the FMA pipe, two lanes at a time: y = n + f, n = rne(y)
// by adding 1.5 * 2^23, 2^f by a degree-4 minimax polynomial on [-1/2, 1/2]
// (relative error below 2^-18 with its fp32 roundings; coefficients from a Remez
// exchange), n into the exponent field.  y is clamped at -125, so that masked
// scores give 2^-125, which is 0 in fp16 and nothing in a row's sum.
__device__ __forceinline__ void exp2_fma2(uint64_t y2, float& p0, float& p1) {
  float y0, y1;
  f2unpack(y2, y0, y1);
  y2 = f2pack(fmaxf(y0, -125.0f), fmaxf(y1, -125.0f));
  const uint64_t t2 = f2add(y2, f2pack(12582912.0f, 12582912.0f));
  const uint64_t n2 = f2add(t2, f2pack(-12582912.0f, -12582912.0f));
  const uint64_t f2 = f2fma(n2, f2pack(-1.0f, -1.0f), y2);
  uint64_t q = f2fma(f2pack(0.009570102f, 0.009570102f), f2, f2pack(0.05591786f, 0.05591786f));
  q = f2fma(q, f2, f2pack(0.24024744f, 0.24024744f));
  q = f2fma(q, f2, f2pack(0.6931218f, 0.6931218f));
  q = f2fma(q, f2, f2pack(0.9999993f, 0.9999993f));
  float q0, q1, t0, t1;
  f2unpack(q, q0, q1);
  f2unpack(t2, t0, t1);
  p0 = __int_as_float(__float_as_int(q0) + (__float_as_int(t0) << 23));
  p1 = __int_as_float(__float_as_int(q1) + (__float_as_int(t1) << 23));
}

// codes2 times a scale: a code and a product's one rounding
__device__ __forceinline__ uint32_t scaled2(uint32_t w, uint32_t sel, __half2 by) {
  const uint32_t c = codes2(w, sel);
  const __half2 v = __hmul2(*reinterpret_cast<const __half2*>(&c), by);
  return *reinterpret_cast<const uint32_t*>(&v);
}

// row_max, NaN where any value is
__device__ __forceinline__ float nan_max3(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
template <int N>
__device__ __forceinline__ float nan_row_max(const float* x) {
  static_assert(N == 64, "eight values behind each of eight chains");
  float a[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    a[k] = x[k];
#pragma unroll
    for (int t = 1; t < 7; t += 2) a[k] = nan_max3(a[k], x[k + 8 * t], x[k + 8 * (t + 1)]);
    a[k] = nan_max3(a[k], x[k + 56], x[k + 56]);
  }
  a[0] = nan_max3(a[0], a[1], a[2]);
  return nan_max3(a[0], nan_max3(a[3], a[4], a[5]), nan_max3(a[6], a[7], a[7]));
}

struct TileMaps {
  CUtensorMap q;
  int q_tma;          // Q through its map: 128 rows are whole tokens
  PageMaps kv;
};

template <int D, bool INT8, bool prefix>
__global__ void __launch_bounds__(CfgT<D, INT8>::THREADS, 1)
    tile_kernel(const __grid_constant__ SharedArgs a, const __grid_constant__ TileMaps maps, DevErr err) {
  using C = CfgT<D, INT8>;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw_s = smem_u32(smem_raw);
  const uint32_t pad = (1024u - (raw_s & 1023u)) & 1023u;
  uint8_t* smem = smem_raw + pad;
  const uint32_t sbase = raw_s + pad;
  auto bar = [&](int i) -> uint32_t { return sbase + C::OFF_BAR + 8u * static_cast<uint32_t>(i); };
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 8 * T_COUNT);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + C::OFF_BAR + 8 * T_COUNT + 4);
  float* scales = reinterpret_cast<float*>(smem + C::OFF_SCALE);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const SharedPlan& p = a.plan;
  const int H = a.pool.H, g = p.group, Hq = H * g;

  pdl_launch_dependents();

  // Own tokens with the prefix folded in: keys below `fold` are the prefix's, own key k is key fold + k (a whole tile's
  // boundary).
  const int fold = prefix ? 1 << 30 : p.fold * 128;

  // ---- this CTA's segments, walked by every role alike
  // prefix: key tiles of the line; own: items (a row block against a split), every gridDim.x-th
  int unit = blockIdx.x, unit_end = p.own_splits * a.batch * p.own_rows * H;
  if (prefix) {
    if (p.pre_pieces > 0) {
      const int rb = static_cast<int>(blockIdx.x) / p.pre_pieces, piece = static_cast<int>(blockIdx.x) - rb * p.pre_pieces;
      unit = rb * p.pre_tiles + piece * p.pre_chunk;
      unit_end = min(unit + p.pre_chunk, (rb + 1) * p.pre_tiles);
    } else {
      const int line = H * p.pre_rows * p.pre_tiles;
      unit = blockIdx.x * p.pre_chunk;
      unit_end = p.pre_chunk < line - unit ? unit + p.pre_chunk : line;
    }
  }
  auto next_segment = [&](int& u, Segment& s) -> bool {
    if (u >= unit_end) return false;
    s.b = s.start = s.hidden = s.nj[0] = s.nj[1] = 0;
    if (prefix) {
      const int rb = u / p.pre_tiles;
      const int first = u - rb * p.pre_tiles;
      const int count = min(p.pre_tiles - first, unit_end - u);
      s.slot = p.pre_pieces > 0 ? first / p.pre_chunk : static_cast<int>(blockIdx.x) - (u - first) / p.pre_chunk;
      u += count;
      s.kvh = rb / p.pre_rows;
      s.row0 = (rb - s.kvh * p.pre_rows) * 256;
      s.key0 = first * 128;
      s.lk = static_cast<int>(a.prefix_len);
      s.rows = max(0, min(static_cast<int>(rows_in_use(a)) * g - s.row0, 256));
      if (s.rows > 0) s.nj[0] = count;
      if (s.rows > 128) s.nj[1] = count;
      return true;
    }
    int item = u / H;
    s.kvh = u - item * H;
    u += gridDim.x;
    const int per = a.batch * p.own_rows;
    const int split = item / per;
    item -= split * per;
    s.b = item / p.own_rows;
    s.row0 = (item - s.b * p.own_rows) * 256;
    s.slot = p.pre_splits + split;
    s.key0 = split * p.own_chunk;
    s.rows = 0;
    int64_t start, n64;
    seq_rows(a, s.b, start, n64);
    const bool outside = rows_outside(a, start, n64, 256);
    if (outside && threadIdx.x == 0) dev_error(err, TM_DEVERR_SEQLEN);
    const int n = static_cast<int>(n64);
    if (outside || s.row0 >= n * g) return true;
    s.start = static_cast<int>(start);
    s.rows = min(n * g - s.row0, 256);
    int lk = __ldg(a.kv_lens + s.b);
    if (lk > a.max_kv) {
      if (threadIdx.x == 0) dev_error(err, TM_DEVERR_SEQLEN);
      lk = static_cast<int>(a.max_kv);
    }
    s.hidden = lk - n + 1;
    s.lk = max(0, lk);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (s.rows <= 128 * t) continue;
      int seen = s.lk;
      if (a.causal) seen = min(seen, s.hidden + (s.row0 + min(s.rows, 128 * (t + 1)) - 1) / g);
      seen = min(fold + max(seen, 0), s.key0 + p.own_chunk);
      s.nj[t] = seen > s.key0 ? (seen - s.key0 + 127) / 128 : 0;
    }
    return true;
  };

  // Page of key `key` of a segment: -1 behind its end, -2 where it cannot be used
  const int shift = a.pool.page_shift;
  const int page_mask = (1 << shift) - 1;
  const int prefix_len = static_cast<int>(a.prefix_len);
  auto place = [&](int key) { return key < fold ? key : key - fold; };                       // within prefix or sequence
  auto keys_of = [&](const Segment& s, int key) { return key < fold ? prefix_len : s.lk; };  // how many there are
  auto entry_at = [&](const Segment& s, int key) -> int32_t {     // as the table has it
    const int k = place(key), col = k >> shift;
    if (k >= keys_of(s, key) || (key >= fold && col >= a.pt.cols)) return -1;
    return __ldg(key < fold ? a.prefix_pages + col : a.pt.table + s.b * a.pt.stride + col);
  };
  auto page_at = [&](const Segment& s, int key) -> int32_t {
    if (place(key) >= keys_of(s, key)) return -1;
    const int32_t page = entry_at(s, key);
    return page_ok(page, a.pool.num_pages) ? page : -2;
  };

  // ---- setup.  The loader makes its own barriers and begins at once; the others wait for them and for tensor
  // memory at the first __syncthreads, which it joins after its first copies.
  int u = unit;
  Segment sg{};
  if (warp >= 8 && warp < 12) {
  // One setmaxnreg for the four control warps: all of a warpgroup have to execute the same one.
  regs_dec<C::CONTROL_REGS>();
  if (warp == 8) {
    if (lane == 0) {
      prefetch_tmap(&maps.q);
      prefetch_tmap(&maps.kv.k);
      prefetch_tmap(&maps.kv.v);
      mbar_init(bar(T_QFULL), 1);
      mbar_init(bar(T_QEMPTY), 2);
      for (int i = 0; i < 4; ++i) mbar_init(bar(T_SFULL + i), 1);
      for (int t = 0; t < 2; ++t) {
        mbar_init(bar(T_ODONE + t), 1);
        mbar_init(bar(T_DRAIN + t), 1);
        mbar_init(bar(T_OLAST + t), 1);
      }
      for (int s = 0; s < C::NSLOT; ++s) {
        mbar_init(bar(T_FULL + s), INT8 ? 4 : 1);
        mbar_init(bar(T_EMPTY + s), 2);
        if (INT8) mbar_init(bar(T_CODES + s), 1);
      }
      *abort_flag = 0;
      fence_barrier_init();
    }
    __syncwarp();
    // ======================= loader =======================
    uint32_t n = 0, qn = 0;
    const int box_shift = shift < 7 ? shift : 7;       // key rows of a copy
    const int boxes = 128 >> box_shift;
    const int LANDED = INT8 ? T_CODES : T_FULL;
    constexpr uint32_t DST = INT8 ? C::SLOT / 2 : 0;
    const uint64_t policy = keys_policy(prefix ? p.pre_rows : p.fold > 0 ? 2 : p.own_rows);
    // a whole tile: lane i copies box i, whose page it holds
    auto copy_boxes = [&](const CUtensorMap* map, uint32_t slot, int32_t page, int key) {
      const uint32_t tile = sbase + C::OFF_SLOT + slot * C::SLOT + DST;
      if (lane == 0) mbar_arrive_expect_tx(bar(LANDED + slot), C::LOADED);
      __syncwarp();
      if (lane < boxes) {
        const int32_t s0 = place(key) & page_mask;
        const int32_t c1 = maps.kv.heads_inner ? sg.kvh : s0, c2 = maps.kv.heads_inner ? s0 : sg.kvh;
#pragma unroll
        for (int hh = 0; hh < (INT8 ? 1 : D / 64); ++hh)
          tma_load_4d(tile + hh * C::HALF + (lane << box_shift) * (INT8 ? D : 128), map, bar(LANDED + slot), hh * 64,
                      c1, c2, page, policy);
      }
      __syncwarp();
    };
    // a ragged tile: row by row; the page of each run of 16 keys is in lane `run`
    auto copy_rows = [&](const uint8_t* base, uint32_t slot, int32_t page, int tile_key) {
      const int key0 = place(tile_key), end = keys_of(sg, tile_key);
      constexpr int ROW = D * (INT8 ? 1 : 2), PIECES = ROW / 16, RPI = 32 / PIECES;
      const uint32_t tile = sbase + C::OFF_SLOT + slot * C::SLOT + DST;
      const int c = lane % PIECES;
#pragma unroll 1
      for (int run = 0; run < 8; ++run) {
        const int32_t pg = __shfl_sync(0xffffffffu, page, run);
        const int key = key0 + 16 * run;
        const uint8_t* src = base + c * 16 + (pg >= 0 ? pg * a.pool.stride_page + (key & page_mask) * a.pool.stride_t : 0);
#pragma unroll
        for (int i = 0; i < 16 / RPI; ++i) {
          const int rr = i * RPI + lane / PIECES;
          const int r = 16 * run + rr;
          const uint32_t dst = INT8 && D == 64 ? tile + r * 64 + ((c ^ ((r >> 1) & 3)) << 4)
                                               : tile + (c >> 3) * C::HALF + r * 128 + (((c & 7) ^ (r & 7)) << 4);
          const bool real = pg >= 0 && key + rr < end;
          cp16(dst, real ? src + rr * a.pool.stride_t : base, real);
        }
      }
      cp_commit();
    };
    auto acquire = [&](uint32_t i) {
      if (i >= C::NSLOT) mbar_wait_warp(bar(T_EMPTY + i % C::NSLOT), (i / C::NSLOT - 1) & 1, err, abort_flag);
    };
    auto landed = [&](uint32_t b) {
      fence_async_shared();      // read by tcgen05.mma
      __syncwarp();
      if (lane == 0) mbar_arrive(b);
    };
    bool met = false;          // the setup's __syncthreads
    auto meet = [&]() {
      if (!met) __syncthreads();
      met = true;
    };
    while (next_segment(u, sg)) {
      const int nj = sg.nj[0] > sg.nj[1] ? sg.nj[0] : sg.nj[1];
      if (nj == 0) continue;
      // pages of key tile j: box i's in lane i
      const int step = 128 / boxes;
      auto my_page = [&](int j) -> int32_t {
        const int key = sg.key0 + j * 128 + lane * step;
        return j < nj && lane < boxes ? page_at(sg, key) : -1;
      };
      int32_t page = my_page(0);
      // Q of both tiles, once the MMAs of the last segment have read theirs
      if (qn > 0) mbar_wait_warp(bar(T_QEMPTY), (qn - 1) & 1, err, abort_flag);
      ++qn;
      const uint32_t gg = static_cast<uint32_t>(g);
      if (maps.q_tma) {
        if (lane == 0) mbar_arrive_expect_tx(bar(T_QFULL), 2 * C::Q_BYTES);
        __syncwarp();
        if (lane < 2 * (D / 64)) {
          const int t = lane & 1, hh = lane >> 1;
          const int32_t token = sg.start + (sg.row0 + 128 * t) / g;
          tma_load_3d(sbase + t * C::Q_BYTES + hh * C::HALF, &maps.q, bar(T_QFULL), hh * 64, sg.kvh * g, token);
        }
        __syncwarp();
      } else {
        constexpr int QP = D / 8;
        const int qc = lane % QP;
        const uint32_t row0 = static_cast<uint32_t>(sg.row0);
        const __half* qbase = a.q + static_cast<int64_t>(sg.start) * a.q_t + static_cast<int64_t>(sg.kvh) * g * a.q_h + qc * 8;
#pragma unroll 2
        for (int i = 0; i < 8 * QP; ++i) {
          const int pr = i * (32 / QP) + lane / QP;
          const bool real = pr < sg.rows;
          const uint32_t row = row0 + pr, tok = row / gg;
          const __half* src = real ? qbase + tok * a.q_t + (row - tok * gg) * a.q_h : a.q;
          const int r = pr & 127;
          cp16(sbase + (pr >> 7) * C::Q_BYTES + (qc >> 3) * C::HALF + r * 128 + (((qc & 7) ^ (r & 7)) << 4), src, real);
        }
        cp_commit();
        cp_wait<0>();
        landed(bar(T_QFULL));
      }
      for (int j = 0; j < nj; ++j, ++n) {
        const int key0 = sg.key0 + j * 128;
        const int32_t next = my_page(j + 1);
        if (page == -2) dev_error(err, TM_DEVERR_SEQLEN);
        const uint32_t i = 2 * n;
        if (maps.kv.ok && place(key0) + 128 <= keys_of(sg, key0) && __all_sync(0xffffffffu, lane >= boxes || page >= 0)) {
          const int key = key0 + lane * step;
          acquire(i);
          copy_boxes(&maps.kv.k, i % C::NSLOT, page, key);
          acquire(i + 1);
          copy_boxes(&maps.kv.v, (i + 1) % C::NSLOT, page, key);
        } else {
          const int32_t run_page = __shfl_sync(0xffffffffu, page, ((lane & 7) * 16) >> box_shift);
          acquire(i);
          copy_rows(a.pool.k + sg.kvh * a.pool.stride_h, i % C::NSLOT, run_page, key0);
          acquire(i + 1);
          copy_rows(a.pool.v + sg.kvh * a.pool.stride_h, (i + 1) % C::NSLOT, run_page, key0);
          cp_wait<1>();
          landed(bar(LANDED + i % C::NSLOT));
          cp_wait<0>();
          landed(bar(LANDED + (i + 1) % C::NSLOT));
        }
        page = next;
        meet();
      }
    }
    meet();
    // every copy has landed before the block may end
    volatile int never = 0;
    if (qn > 0) mbar_wait_warp(bar(T_QFULL), (qn - 1) & 1, err, &never);
    for (uint32_t i = 2 * n > C::NSLOT ? 2 * n - C::NSLOT : 0; i < 2 * n; ++i)
      mbar_wait_warp(bar(LANDED + i % C::NSLOT), (i / C::NSLOT) & 1, err, &never);
  } else {
    if (warp == 9) {
      tmem_alloc(smem_u32(tmem_slot), 512);
      tmem_relinquish();
      tc_fence_before();
    }
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (warp == 9 || warp == 10) {
      // ======================= tcgen05 issuers (warp 9: tile A, warp 10: tile B) ====
      // They never touch shared memory: the wait helper polls for them.
      const int t = warp - 9;
      uint32_t n = 0;
      bool any = false;
      const uint32_t d_s = tmem + C::s_col(t), d_o = tmem + C::o_col(t);
      auto kv_handoff = [&]() {
        named_bar_sync(NB_KV + t, 64);
        tc_fence_after();
      };
      auto commit = [&](uint32_t b, int times) {
        if (elect_one()) {
          tc_commit(b);
          if (times > 1) tc_commit(b);
        }
        __syncwarp();
      };
      auto issue_s = [&](uint32_t kslot, int c) {
        const uint32_t kb = sbase + C::OFF_SLOT + kslot * C::SLOT + (c & 1) * 8192;
        const uint32_t qa = sbase + t * C::Q_BYTES;
        uint64_t ad[D / 16], bd[D / 16];
#pragma unroll
        for (int kk = 0; kk < D / 16; ++kk) {
          const uint32_t off = (kk >> 2) * C::HALF + (kk & 3) * 32;
          ad[kk] = smem_desc(qa + off, 16, 1024, kSwizzle128);
          bd[kk] = smem_desc(kb + off, 16, 1024, kSwizzle128);
        }
        if (elect_one()) {
          mma_f16_ss_n<D / 16>(d_s + 64u * static_cast<uint32_t>(c & 1), ad, bd, C::IDESC_S, 0u);
          tc_commit(bar(T_SFULL + 2 * t + (c & 1)));
        }
        __syncwarp();
      };
      auto issue_pv = [&](int c, uint32_t vslot) {
        const uint32_t vb = sbase + C::OFF_SLOT + vslot * C::SLOT;
        uint32_t at[4];
        uint64_t bd[4];
#pragma unroll
        for (int kk = 0; kk < 4; ++kk) {
          at[kk] = d_s + 64u * static_cast<uint32_t>(c & 1) + kk * 8;
          bd[kk] = smem_desc(vb + ((c & 1) * 4 + kk) * 2048, C::HALF, 1024, kSwizzle128);
        }
        named_bar_sync(NB_P + 2 * t + (c & 1), 160);      // softmax t stored P_t(c)
        tc_fence_after();
        if (elect_one()) {
          mma_f16_ts_n<4>(d_o, at, bd, C::IDESC_PV, c > 0 ? 1u : 0u);
          tc_commit(bar(T_ODONE + t));
        }
        __syncwarp();
      };
      while (next_segment(u, sg)) {
        const int nt = sg.nj[t], no = sg.nj[1 - t], nj = nt > no ? nt : no;
        if (nt > 0) {
          any = true;
          kv_handoff();       // Q landed
          uint32_t v_prev = 0;
          for (int j = 0; j < nt; ++j) {
            const uint32_t sk = (2 * (n + j)) % C::NSLOT, sv = (2 * (n + j) + 1) % C::NSLOT;
            const int share = j >= no ? 2 : 1;           // also the other tile's release where it has no tile j
            kv_handoff();     // K of j (and V of j - 1) landed
            if (j > 0) issue_pv(2 * j - 2, v_prev);
            issue_s(sk, 2 * j);
            if (j > 0) {
              issue_pv(2 * j - 1, v_prev);
              commit(bar(T_EMPTY + v_prev), j - 1 >= no ? 2 : 1);
            }
            issue_s(sk, 2 * j + 1);
            commit(bar(T_EMPTY + sk), share);
            if (j == nt - 1) commit(bar(T_QEMPTY), no == 0 ? 2 : 1);
            v_prev = sv;
          }
          kv_handoff();       // V of the last key tile landed
          issue_pv(2 * nt - 2, v_prev);
          issue_pv(2 * nt - 1, v_prev);
          commit(bar(T_OLAST + t), 1);
          commit(bar(T_EMPTY + v_prev), nt - 1 >= no ? 2 : 1);
        }
        n += nj;
      }
      if (any) {
        commit(bar(T_DRAIN + t), 1);
        if (lane == 0) {
          volatile int never = 0;
          mbar_wait(bar(T_DRAIN + t), 0, err, &never);
        }
        __syncwarp();
      }
    } else if (warp == 11) {
      // ======================= wait helper =======================
      uint32_t n = 0, qn = 0;
      auto wait1 = [&](uint32_t b, uint32_t par) {
        if (lane == 0) mbar_wait(b, par, err, abort_flag);
      };
      auto wait_slot = [&](uint32_t i) { wait1(bar(T_FULL + i % C::NSLOT), (i / C::NSLOT) & 1); };
      auto handoff = [&](int t) {
        __syncwarp();
        named_bar_sync(NB_KV + t, 64);
      };
      while (next_segment(u, sg)) {
        const int na = sg.nj[0], nb = sg.nj[1], nj = na > nb ? na : nb;
        if (nj == 0) continue;
        wait1(bar(T_QFULL), qn & 1);
        ++qn;
        if (na > 0) handoff(0);
        if (nb > 0) handoff(1);
        for (int j = 0; j < nj; ++j, ++n) {
          if (j > 0) wait_slot(2 * n - 1);
          wait_slot(2 * n);
          if (j < na) handoff(0);
          if (j < nb) handoff(1);
          if (j == na - 1 || j == nb - 1) wait_slot(2 * n + 1);
          if (j == na - 1) handoff(0);
          if (j == nb - 1) handoff(1);
        }
      }
    }
  }
  } else {
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (INT8 && warp >= 12) {
    // ======================= conversion of codes (warpgroup v: K or V; thread r: key row r of each tile) ====
    regs_dec<C::CONVERT_REGS>();
    const int v = (warp - 12) >> 2;
    const int r = threadIdx.x & 127;
    uint32_t i = v;
    while (next_segment(u, sg)) {
      const int nj = sg.nj[0] > sg.nj[1] ? sg.nj[0] : sg.nj[1];
      // this row's page and scale, loaded two and one key tiles ahead
      auto entry_of = [&](int j) { return j < nj ? entry_at(sg, sg.key0 + j * 128 + r) : -1; };
      auto scales_at = [&](int j, int32_t page, __half& ks, __half& vs) {
        ks = vs = __float2half(0.f);
        if (!page_ok(page, a.pool.num_pages)) return;
        const int64_t at = page * a.pool.sstride_page + (place(sg.key0 + j * 128 + r) & page_mask) * a.pool.sstride_t +
                           sg.kvh * a.pool.sstride_h;
        if (v == 0) ks = a.pool.ks[at];
        vs = a.pool.vs[at];
      };
      int32_t entry = entry_of(0);
      __half ks, vs, next_ks, next_vs;
      scales_at(0, entry, next_ks, next_vs);
      entry = entry_of(1);
      for (int j = 0; j < nj; ++j, i += 2) {
        ks = next_ks;
        vs = next_vs;
        scales_at(j + 1, entry, next_ks, next_vs);
        entry = entry_of(j + 2);
        {
          const uint32_t slot = i % C::NSLOT;
          mbar_wait_warp(bar(T_CODES + slot), (i / C::NSLOT) & 1, err, abort_flag);
          const uint32_t tile = sbase + C::OFF_SLOT + slot * C::SLOT;
          // The scales outlive K's slot: the softmax reads those of key tile j until P(2 j + 1).  With one stage more
          // than the ring has key tiles, the next tile in this stage lands behind a release of key tile j + 1, whose
          // last S is issued behind P.V(2 j + 1).
          const uint32_t bits = __float_as_uint(__half2float(vs));
          const uint32_t power = min(bits & 0x7f800000u, 0x43800000u);      // 2^8 at most
          if (v == 0) {
            float* sc = scales + ((i / 2) % C::STAGES) * 256;
            const uint32_t rest = bits - power + 0x3f800000u;               // V scale / power; of a zero scale: 1
            sc[r] = __half2float(ks) * a.scale_log2;
            sc[128 + r] = __uint_as_float(rest);
          }
          const __half2 by = __half2half2(__float2half(v ? __uint_as_float(power) : 1.f));
          auto widen = [&](uint4 c, uint32_t at, int q) {      // 16 codes to pieces 2 q and 2 q + 1 of a row
            const uint32_t x[4] = {c.x ^ 0x80808080u, c.y ^ 0x80808080u, c.z ^ 0x80808080u, c.w ^ 0x80808080u};
            sts128(at + (((2 * q) ^ (r & 7)) << 4),
                   make_uint4(scaled2(x[0], 0x4140u, by), scaled2(x[0], 0x4342u, by), scaled2(x[1], 0x4140u, by),
                              scaled2(x[1], 0x4342u, by)));
            sts128(at + (((2 * q + 1) ^ (r & 7)) << 4),
                   make_uint4(scaled2(x[2], 0x4140u, by), scaled2(x[2], 0x4342u, by), scaled2(x[3], 0x4140u, by),
                              scaled2(x[3], 0x4342u, by)));
          };
          if (D == 128) {
            // The codes lie where the upper 64 columns go, row r's in row r's place; there piece q's output covers
            // code pieces up to q, which have been read.  A rolled loop: the softmax needs the instruction cache.
            const uint32_t src = tile + C::HALF + r * 128;
            uint4 c = lds128(src + ((r & 7) << 4));
#pragma unroll 1
            for (int q = 0; q < 8; ++q) {
              const uint4 after = lds128(src + ((((q + 1) & 7) ^ (r & 7)) << 4));
              widen(c, tile + (q >> 2) * C::HALF + r * 128, q & 3);
              c = after;
            }
          } else {
            // 64-byte rows over other rows' places: all are read before any is written
            const uint32_t src = tile + C::CODES + r * 64;
            uint4 c[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) c[q] = lds128(src + ((q ^ ((r >> 1) & 3)) << 4));
            named_bar_sync(NB_CVT + v, 128);
#pragma unroll
            for (int q = 0; q < 4; ++q) widen(c[q], tile + r * 128, q);
          }
          fence_async_shared();    // read by tcgen05.mma
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(T_FULL + slot));
        }
      }
    }
  } else {
    // ======================= softmax (warpgroup t = query tile t) =======================
    regs_inc<C::SOFTMAX_REGS>();
    constexpr int HN = 64;
    const int t = warp >> 2;
    const int r = threadIdx.x & 127;                 // row in the tile = TMEM lane
    const uint32_t lane_addr = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
    const uint32_t s_addr = lane_addr + C::s_col(t), o_addr = lane_addr + C::o_col(t);
    uint32_t cc = 0;      // chunks of this query tile so far, over all segments
    uint32_t n = 0;       // key tiles so far
    uint32_t segs = 0;    // segments of this query tile so far
    bool owed = false;    // tile 0: the other warpgroup's arrival for its last turn has not been met
    const int64_t total = a.T * Hq;
    const bool direct = p.slots == 1;
    const float cs = INT8 ? 1.f : a.scale_log2;      // INT8: in the K scales
    while (next_segment(u, sg)) {
      const int nt = sg.nj[t];
      const int pr = 128 * t + r;
      const bool row_ok = pr < sg.rows;
      const int prow = sg.row0 + pr, tok_in = prow / g;
      const int tok = sg.start + tok_in, head = sg.kvh * g + prow - tok_in * g;
      // keys below these are seen, in the prefix and behind it
      const int lim_prefix = row_ok ? prefix_len : 0;
      int lim_own = fold;
      if (row_ok && !prefix) lim_own += max(0, a.causal ? min(sg.lk, sg.hidden + tok_in) : sg.lk);
      // Reference (a score product of the row, counted from `base`), and the exponent of product x by it: x * cs - less.
      // Before the first one every finite product exceeds it, and a hidden one's exponent is -inf.
      float x_ref = -INFINITY, base = 0.f, less = -1e30f, l = 0.f;
      bool saw = false;      // a key
      // The two softmax warpgroups take turns at their exponentials: side by side they would slow each other down
      // into lockstep, and stores, waits and handoffs of both would leave the SM idle at the same time.
      // Strictly in turns, over segments' ends too: tile 0 meets tile 1's last arrival before its next first turn.
      // (An arrival that ran ahead would complete a barrier that tile 1 has not come to, and leave it there.)
      const int turns = 2 * min(sg.nj[0], sg.nj[1]);
      for (int c = 0; c < 2 * nt; ++c, ++cc) {
        const int sl = c & 1;
        const uint32_t s_c = s_addr + HN * sl;
        mbar_wait(bar(T_SFULL + 2 * t + sl), (cc >> 1) & 1, err, abort_flag);
        tc_fence_after();
        __syncwarp();
        float2 mine = make_float2(1.f, 1.f);      // INT8: what two of the keys' V scales multiply in
        if (INT8) mine = *reinterpret_cast<const float2*>(scales + ((n + (c >> 1)) % C::STAGES) * 256 + 128 + HN * sl + 2 * lane);
        float x[HN], alpha = 1.f;
        for (;;) {
          {
            uint32_t v[HN];
#pragma unroll
            for (int q = 0; q < HN / 32; ++q) tmem_ld32p(s_c + q * 32, v + q * 32);
            tmem_wait_ld_regs<HN>(v);
#pragma unroll
            for (int e = 0; e < HN; ++e) x[e] = __uint_as_float(v[e]);
          }
          if (INT8) {
            const float* sc = scales + ((n + (c >> 1)) % C::STAGES) * 256 + HN * sl;
#pragma unroll
            for (int e = 0; e < HN; e += 4) {
              const float4 k4 = *reinterpret_cast<const float4*>(sc + e);
              f2unpack(f2mul(f2pack(x[e], x[e + 1]), f2pack(k4.x, k4.y)), x[e], x[e + 1]);
              f2unpack(f2mul(f2pack(x[e + 2], x[e + 3]), f2pack(k4.z, k4.w)), x[e + 2], x[e + 3]);
            }
          }
          const int key0 = sg.key0 + c * HN;
          const int nv = max(0, min((key0 < fold ? lim_prefix : lim_own) - key0, HN));
          if (!__all_sync(0xffffffffu, nv == HN && (INT8 || base == 0.f))) {
#pragma unroll
            for (int e = 0; e < HN; ++e) x[e] = (e < nv) ? (INT8 ? x[e] : x[e] - base) : -INFINITY;
          }
          float room = kTopTile<INT8>;
          if (INT8 && __any_sync(0xffffffffu, fmaxf(fabsf(mine.x), fabsf(mine.y)) >= 2.f)) room -= 7.f;
          bool far = false;
          if (nv > 0) {
            const float top = nan_row_max<HN>(x);
            saw = true;
            if (!(fmaf(top, cs, -less) <= room)) {      // a NaN too: alpha, and with it l, is NaN from there on
              far = !INT8 && fabsf(top * cs) > kFarScore;
              if (far) base += top;
              x_ref = far ? 0.f : top;
              const float before = far ? fmaf(-top, cs, less) : less;
              less = __fsub_rn(__fmul_rn(x_ref, cs), base == 0.f ? kPOffset : 0.f);      // 6 would be lost next to base * cs
              alpha = ex2_approx(before - less);
            }
          }
          // with a new base once more, from the scores in tensor memory
          if (INT8 || !__any_sync(0xffffffffu, far)) break;
        }
        if (c < turns && (t == 1 || c > 0 || owed)) named_bar_sync(NB_TURN + t, 256);
        const uint64_t c2 = f2pack(cs, cs), nm2 = f2pack(-less, -less);
        uint32_t pk[HN / 2];
        uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int e = 0; e < HN; e += 2) {
          const uint64_t y2 = f2fma(f2pack(x[e], x[e + 1]), c2, nm2);
          float p0, p1;
          if (((e >> 1) & 7) < kFmaPairs<INT8>) {
            exp2_fma2(y2, p0, p1);
          } else {
            float y0, y1;
            f2unpack(y2, y0, y1);
            p0 = ex2_approx(y0);
            p1 = ex2_approx(y1);
          }
          acc2[(e >> 1) & 3] = f2add(acc2[(e >> 1) & 3], f2pack(p0, p1));
          if (INT8) {
            const float2 f = *reinterpret_cast<const float2*>(scales + ((n + (c >> 1)) % C::STAGES) * 256 + 128 + HN * sl + e);
            f2unpack(f2mul(f2pack(p0, p1), f2pack(f.x, f.y)), p0, p1);
          }
          pk[e >> 1] = pack_half2(p0, p1);
        }
        {
          const uint64_t s2 = f2add(f2add(acc2[0], acc2[1]), f2add(acc2[2], acc2[3]));
          float s0, s1;
          f2unpack(s2, s0, s1);
          l = l * alpha + (s0 + s1);
        }
        if (c < turns) named_bar_arrive(NB_TURN + 1 - t, 256);
        __syncwarp();
        tmem_st32p(s_c, pk);      // P(c) over the first 32 columns of its half
        // P.V(c - 1) must have completed before O is rescaled; phases up to
        // c - 2 are complete (S(c) was issued behind P.V(c - 2))
        if (c > 0 && __any_sync(0xffffffffu, alpha != 1.f)) {
          mbar_wait(bar(T_ODONE + t), (cc - 1) & 1, err, abort_flag);
          tc_fence_after();
          __syncwarp();
          const uint64_t a2 = f2pack(alpha, alpha);
#pragma unroll 1
          for (int q = 0; q < D / 32; ++q) {
            uint32_t o[32];
            tmem_ld32p(o_addr + q * 32, o);
            tmem_wait_ld_regs<32>(o);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float o0, o1;
              f2unpack(f2mul(f2pack(__uint_as_float(o[e]), __uint_as_float(o[e + 1])), a2), o0, o1);
              o[e] = __float_as_uint(o0);
              o[e + 1] = __float_as_uint(o1);
            }
            tmem_st32p(o_addr + q * 32, o);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        // not waiting: this half's next P follows an S that is issued behind this one's P.V
        named_bar_arrive(NB_P + 2 * t + sl, 160);
      }
      if (turns > 0) owed = t == 0;
      n += sg.nj[0] > sg.nj[1] ? sg.nj[0] : sg.nj[1];

      // ---- the row's result: partial (O, m, l), or the output
      // A row that saw nothing has no weight.  Of a query that is not finite all scores are NaN or infinities: NaN, which
      // the weights alone need not show (the exponentials on the FMA pipe clamp a NaN to 2^-125).
      if (!saw) l = 0.f;
      else if (!(fabsf(base + x_ref) < INFINITY)) l = NAN;
      if (nt > 0) {
        mbar_wait(bar(T_OLAST + t), segs & 1, err, abort_flag);
        ++segs;
        tc_fence_after();
        __syncwarp();
      }
      const int64_t idx = static_cast<int64_t>(tok) * Hq + head;
      if (row_ok && !direct) a.ml[sg.slot * total + idx] = make_float2(x_ref == -INFINITY ? x_ref : base * cs + less, l);
      const float inv = !direct ? 1.f : (l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l));
      if (nt > 0 || direct) {
        // OUT_COLS columns of the warp's 32 rows at a time through shared memory, so that a store instruction writes
        // whole lines (or halves) of a few rows instead of 32 rows' halves of sectors
        constexpr int PR = C::OUT_COLS / 4, RPI = 32 / PR;        // 16-byte pieces of a row, rows of an instruction
        const uint32_t stage = sbase + C::OFF_OUT + warp * (32 * C::OUT_COLS * 4);
        auto place = [&](int row, int e) {
          return stage + row * (PR * 16) + ((PR == 8 ? e ^ (row & 7) : e ^ ((row >> 1) & 3)) << 4);
        };
        const bool wanted = row_ok && !(prefix && direct && tok < first_row(a));
        const int64_t mine = wanted ? (direct ? tok * a.o_t + head * a.o_h : (sg.slot * total + idx) * D) : -1;
        int64_t at[PR];       // where rows lane / PR + RPI i go
#pragma unroll
        for (int i = 0; i < PR; ++i) at[i] = __shfl_sync(0xffffffffu, mine, RPI * i + lane / PR);
#pragma unroll 1
        for (int q = 0; q < D / 32; ++q) {
          uint32_t o[32];
          if (nt > 0) {
            tmem_ld32p(o_addr + q * 32, o);
            tmem_wait_ld_regs<32>(o);
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
#pragma unroll
          for (int hh = 0; hh < 32 / C::OUT_COLS; ++hh) {
#pragma unroll
            for (int e = 0; e < PR; ++e) {
              const uint32_t* x = o + hh * C::OUT_COLS + 4 * e;
              sts128(place(lane, e), make_uint4(__float_as_uint(__uint_as_float(x[0]) * inv),
                                                __float_as_uint(__uint_as_float(x[1]) * inv),
                                                __float_as_uint(__uint_as_float(x[2]) * inv),
                                                __float_as_uint(__uint_as_float(x[3]) * inv)));
            }
            __syncwarp();
#pragma unroll
            for (int i = 0; i < PR; ++i) {
              const int row = RPI * i + lane / PR, e = lane % PR;
              const uint4 v = lds128(place(row, e));
              if (at[i] < 0) continue;
              const int col = q * 32 + hh * C::OUT_COLS + e * 4;
              if (direct)
                *reinterpret_cast<uint2*>(a.out + at[i] + col) =
                    make_uint2(pack_half2(__uint_as_float(v.x), __uint_as_float(v.y)),
                               pack_half2(__uint_as_float(v.z), __uint_as_float(v.w)));
              else
                *reinterpret_cast<uint4*>(a.o + at[i] + col) = v;
            }
            __syncwarp();         // tensor-memory loads and the stage are the whole warp's
          }
        }
        tc_fence_before();      // these reads of O come before the next segment's first P.V
      }
    }
    if (owed) named_bar_sync(NB_TURN + t, 256);
  }
  }

  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(*tmem_slot, 512);
  }
  pdl_wait();      // whoever waits for this kernel has waited for the one before it
}

}  // namespace

PageMaps page_maps(const PagedPool& pool, int d, bool int8, int rows) {
  PageMaps m{};
  m.heads_inner = pool.stride_h < pool.stride_t;
  const int64_t page_size = 1ll << pool.page_shift;
  const int box_rows = page_size < rows ? static_cast<int>(page_size) : rows;
  const int64_t dims[4] = {d, m.heads_inner ? pool.H : page_size, m.heads_inner ? page_size : pool.H, pool.num_pages};
  const int64_t strides[3] = {m.heads_inner ? pool.stride_h : pool.stride_t, m.heads_inner ? pool.stride_t : pool.stride_h,
                              pool.stride_page};
  const int box[4] = {int8 ? d : 64, m.heads_inner ? 1 : box_rows, m.heads_inner ? box_rows : 1, 1};
  const CUtensorMapDataType type = int8 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16;
  const CUtensorMapSwizzle swz = int8 && d == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B;
  m.ok = encode_tiled_map(&m.k, pool.k, type, 4, dims, strides, box, swz) &&
         encode_tiled_map(&m.v, pool.v, type, 4, dims, strides, box, swz);
  return m;
}

template <int D, bool INT8, bool prefix>
static tm_status launch_tile(const SharedArgs& a, bool overlap, DevErr err, cudaStream_t stream) {
  using C = CfgT<D, INT8>;
  static std::atomic<uint64_t> prepared{0};
  tm_status st = prepare_smem(tile_kernel<D, INT8, prefix>, C::SMEM, prepared);
  if (st != TM_OK) return st;
  const SharedPlan& p = a.plan;
  TileMaps m{};
  const int g = p.group, Hq = a.pool.H * g;
  m.kv = page_maps(a.pool, D, INT8, 128);
  if (128 % g == 0) {
    const int64_t qdims[3] = {D, Hq, a.T};
    const int64_t qstrides[2] = {(Hq > 1 ? a.q_h : D) * 2, (a.T > 1 ? a.q_t : D * Hq) * 2};
    const int qbox[3] = {64, g, 128 / g};
    m.q_tma = encode_tiled_map(&m.q, a.q, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 3, qdims, qstrides, qbox,
                               CU_TENSOR_MAP_SWIZZLE_128B);
  }
  int64_t items = p.pre_ctas;
  if (!prefix) {
    // one CTA for each SM, which goes through several items: a CTA's start (setup, first copies, cold instructions) is
    // as long as five key tiles
    items = static_cast<int64_t>(p.own_splits) * a.batch * p.own_rows * a.pool.H;
    if (items > 0x7fffffff) return TM_ERR_UNSUPPORTED;
    if (items > kSmsB200) items = kSmsB200;
  }
  return launch_kernel(tile_kernel<D, INT8, prefix>, items, C::THREADS, C::SMEM, overlap, stream, a, m, err);
}

template <int D, bool INT8>
static tm_status launch_tile_of(const SharedArgs& a, bool prefix, bool overlap, DevErr err, cudaStream_t stream) {
  return prefix ? launch_tile<D, INT8, true>(a, overlap, err, stream) : launch_tile<D, INT8, false>(a, overlap, err, stream);
}

tm_status shared_tile(const SharedArgs& a, int d, bool int8, bool prefix, bool overlap, DevErr err,
                      cudaStream_t stream) {
  if (d == 128) return int8 ? launch_tile_of<128, true>(a, prefix, overlap, err, stream)
                            : launch_tile_of<128, false>(a, prefix, overlap, err, stream);
  return int8 ? launch_tile_of<64, true>(a, prefix, overlap, err, stream)
              : launch_tile_of<64, false>(a, prefix, overlap, err, stream);
}

}  // namespace tmk
