// tm_attn_shared_tile.cu -- attention over a paged cache for many rows
// (tm_attn_shared_prefix): 256 packed rows of one K/V head against a range of
// keys on tcgen05, K and V gathered from their pages on the way in.
//
// One CTA holds two 128-row query tiles, whose softmax warpgroups alternate on
// the tensor core; a tile's 128 score columns are two 64-key halves, and
// S(c + 2) follows P.V(c) into the half that P(c) leaves, so the next scores are
// computed while the softmax works on the current ones.  O stays in tensor
// memory over the whole range; a row's reference maximum is raised (and O
// rescaled) only when a score exceeds it by 2^kLazy.
//
// Loads: four warps copy rows of 16-byte pieces (cp.async) from wherever the
// block table puts them straight into the 128-byte-swizzled layout that the
// MMAs read; rows past the range are filled with zeros and never read from
// memory, so pages of any size and strides need no special cases.  A ring of
// 128 KB keeps two key tiles in flight.
//
// INT8 pages: the copies bring the codes, which the same warps turn into fp16
// in place (exactly).  The scales never touch the codes: with t_j = s_j ks_j +
// log2 vs_j the weights 2^(t_j - m) of the P.V product carry the V scale, and
// the row sum takes 2^(t_j - m) / vs_j; both cost no more than scaling the
// scores, and the weights keep fp16's full range whatever the scales are.
//
// The prefix's work is one line of key tiles (row block by row block) cut into
// equal pieces, one for each CTA, so that all SMs finish together; a CTA whose
// piece crosses a row block's end writes one partial result for each block.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <atomic>

#include "tm_attn_shared.cuh"
#include "tm_host.h"

namespace tmk {
namespace {

constexpr int kThreads = 512;
// 2^kPOffset is the largest weight when the reference is the maximum; scores
// up to 2^kLazy above it are left alone: 2^15 at most, inside fp16.
constexpr float kLazy = 15.0f - kPOffset;

// Of every 8 pairs of exponentials, how many run on the FMA pipe: the special
// function unit alone takes as long as the MMAs of a tile.
#ifndef TM_FMA_PAIRS
#define TM_FMA_PAIRS 3
#endif
constexpr int kFmaPairs = TM_FMA_PAIRS;

template <int D>
struct CfgT {
  static constexpr int BM = 128, BN = 128;
  static constexpr int HALF = 128 * 128;               // one 64-column slab of a tile
  static constexpr int SLOT = BN * D * 2;              // an fp16 K or V tile
  static constexpr int NSLOT = 131072 / SLOT;          // 4 (d = 128) or 8 (d = 64)
  static constexpr int STAGES = NSLOT / 2;
  static constexpr int Q_BYTES = BM * D * 2;
  static constexpr int OFF_SLOT = 2 * Q_BYTES;
  static constexpr int OFF_SCALE = OFF_SLOT + NSLOT * SLOT;       // [STAGES][3][128] floats
  static constexpr int OFF_BAR = OFF_SCALE + STAGES * 3 * 128 * 4;
  static constexpr int SMEM = OFF_BAR + 512 + 1024;
  static constexpr uint32_t IDESC_S = idesc_f16(BM, 64, false);
  static constexpr uint32_t IDESC_PV = idesc_f16(BM, D, true);
  // registers: 512 x 128 at launch; 2 x 128 x 200 + 256 x 56 after the split
  static constexpr int SOFTMAX_REGS = 200, OTHER_REGS = 56;
  static_assert(2 * 128 * SOFTMAX_REGS + 256 * OTHER_REGS == 512 * 128, "register split");
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
  T_COUNT = 28
};
// Named barriers: NB_P + t softmax t -> issuer t (P stored); NB_KV + t wait
// helper -> issuer t (operands landed); NB_START softmax A -> issuer B.
enum : int { NB_P = 1, NB_KV = 3, NB_START = 5 };

// One row block against one range of keys.
struct Segment {
  int kvh, b, slot, rows;     // rows of the block: 1 .. 256
  int64_t row0, start;        // first packed row (of the batch or the sequence), first token
  int64_t key0, lk;           // first key, keys that exist
  int64_t hidden;             // own, causal: token i of the sequence sees keys below hidden + i
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

template <int D, bool INT8>
__global__ void __launch_bounds__(kThreads, 1) tile_kernel(const __grid_constant__ SharedArgs a, int prefix,
                                                           DevErr err) {
  using C = CfgT<D>;
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

  // ---- this CTA's segments, walked by every role alike
  int64_t unit = 0, unit_end = 1;         // prefix: key tiles of the line
  if (prefix) {
    unit = static_cast<int64_t>(blockIdx.x) * p.pre_chunk;
    const int64_t line = static_cast<int64_t>(H) * p.pre_rows * p.pre_tiles;
    unit_end = unit + p.pre_chunk < line ? unit + p.pre_chunk : line;
  }
  auto next_segment = [&](int64_t& u, Segment& s) -> bool {
    if (u >= unit_end) return false;
    s.b = 0;
    s.start = s.hidden = 0;
    s.nj[0] = s.nj[1] = 0;
    if (prefix) {
      const int64_t rb = u / p.pre_tiles;
      const int64_t first = u - rb * p.pre_tiles;
      int64_t count = p.pre_tiles - first;
      if (count > unit_end - u) count = unit_end - u;
      u += count;
      s.kvh = static_cast<int>(rb / p.pre_rows);
      s.row0 = (rb - static_cast<int64_t>(s.kvh) * p.pre_rows) * 256;
      s.slot = static_cast<int>(blockIdx.x - rb * p.pre_tiles / p.pre_chunk);
      s.key0 = first * 128;
      s.lk = a.prefix_len;
      const int64_t n = rows_in_use(a) * g - s.row0;
      s.rows = n < 0 ? 0 : (n < 256 ? static_cast<int>(n) : 256);
      if (s.rows > 0) s.nj[0] = static_cast<int>(count);
      if (s.rows > 128) s.nj[1] = static_cast<int>(count);
      return true;
    }
    u = unit_end;
    int64_t item = blockIdx.x;
    s.kvh = static_cast<int>(item % H);
    item /= H;
    const int64_t per = static_cast<int64_t>(a.batch) * p.own_rows;
    const int split = static_cast<int>(item / per);
    item %= per;
    s.b = static_cast<int>(item / p.own_rows);
    s.row0 = (item % p.own_rows) * 256;
    s.slot = p.pre_splits + split;
    s.key0 = static_cast<int64_t>(split) * p.own_chunk;
    int64_t n;
    seq_rows(a, s.b, s.start, n);
    s.rows = 0;
    const bool outside = s.start < 0 || n < 0 || s.start + n > a.T || n * g > static_cast<int64_t>(p.own_rows) * 256;
    if (outside && threadIdx.x == 0) dev_error(err, TM_DEVERR_SEQLEN);
    if (outside || s.row0 >= n * g) return true;
    s.rows = static_cast<int>(n * g - s.row0 < 256 ? n * g - s.row0 : 256);
    s.lk = __ldg(a.kv_lens + s.b);
    if (s.lk > a.max_kv) {
      if (threadIdx.x == 0) dev_error(err, TM_DEVERR_SEQLEN);
      s.lk = a.max_kv;
    }
    s.hidden = s.lk - n + 1;
    int64_t end = s.key0 + p.own_chunk < s.lk ? s.key0 + p.own_chunk : s.lk;
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      if (s.rows <= 128 * t) continue;
      int64_t seen = end;
      if (a.causal) {
        const int64_t last = s.row0 + (s.rows < 128 * (t + 1) ? s.rows : 128 * (t + 1)) - 1;
        const int64_t l = s.hidden + last / g;
        if (l < seen) seen = l;
      }
      s.nj[t] = seen > s.key0 ? static_cast<int>((seen - s.key0 + 127) / 128) : 0;
    }
    s.lk = end > 0 ? end : 0;
    return true;
  };

  // ---- setup
  if (threadIdx.x == 0) {
    mbar_init(bar(T_QFULL), 4);
    mbar_init(bar(T_QEMPTY), 2);
    for (int i = 0; i < 4; ++i) mbar_init(bar(T_SFULL + i), 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(bar(T_ODONE + t), 1);
      mbar_init(bar(T_DRAIN + t), 1);
      mbar_init(bar(T_OLAST + t), 1);
    }
    for (int s = 0; s < C::NSLOT; ++s) {
      mbar_init(bar(T_FULL + s), 4);
      mbar_init(bar(T_EMPTY + s), 2);
    }
    *abort_flag = 0;
    fence_barrier_init();
  }
  if (warp == 9) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
    tc_fence_before();
  }
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  int64_t u = unit;
  Segment sg;

  if (warp >= 12) {
    // ======================= loaders (warp w: rows 32 w .. of each tile) ====
    regs_dec<C::OTHER_REGS>();
    const int w = warp - 12;
    const int shift = a.pool.page_shift;
    const int64_t page_mask = (1ll << shift) - 1;
    constexpr int ROW = D * (INT8 ? 1 : 2), PIECES = ROW / 16, RPI = 32 / PIECES;
    constexpr int CODE_OFF = INT8 && D == 128 ? C::HALF : 0;   // codes wait inside their own row's fp16 place
    // up to three groups of copies in flight, oldest first: barrier to signal and (INT8) the tile to convert
    uint32_t pb0 = 0, pb1 = 0, pb2 = 0, pt0 = 0, pt1 = 0, pt2 = 0;
    int np = 0;
    auto finish_oldest = [&]() {
      if (np == 3) cp_wait<2>();
      else if (np == 2) cp_wait<1>();
      else cp_wait<0>();
      __syncwarp();
      if (INT8 && pt0 != 0) {
        const int r = 32 * w + lane;
        const uint32_t row = pt0 + r * 128;
#pragma unroll
        for (int half = 0; half < D / 64; ++half) {
          uint4 c[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) c[i] = lds128(row + CODE_OFF + (((4 * half + i) ^ (r & 7)) << 4));
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t x[4] = {c[i].x ^ 0x80808080u, c[i].y ^ 0x80808080u, c[i].z ^ 0x80808080u,
                                   c[i].w ^ 0x80808080u};
            const uint32_t at = row + half * C::HALF;
            sts128(at + (((2 * i) ^ (r & 7)) << 4), make_uint4(codes2(x[0], 0x4140u), codes2(x[0], 0x4342u),
                                                               codes2(x[1], 0x4140u), codes2(x[1], 0x4342u)));
            sts128(at + (((2 * i + 1) ^ (r & 7)) << 4), make_uint4(codes2(x[2], 0x4140u), codes2(x[2], 0x4342u),
                                                                   codes2(x[3], 0x4140u), codes2(x[3], 0x4342u)));
          }
        }
      }
      fence_async_shared();    // these stores are read by tcgen05.mma
      __syncwarp();
      if (lane == 0) mbar_arrive(pb0);
      pb0 = pb1;
      pb1 = pb2;
      pt0 = pt1;
      pt1 = pt2;
      --np;
    };
    // Waits for a barrier; groups that have not been signalled yet come first when it is not free.
    auto acquire = [&](uint32_t b, uint32_t parity) {
      if (np == 3) finish_oldest();
      while (np > 0 && !__shfl_sync(0xffffffffu, static_cast<int>(mbar_test_wait(b, parity)), 0)) finish_oldest();
      mbar_wait_warp(b, parity, err, abort_flag);
    };
    auto pushed = [&](uint32_t b, uint32_t tile) {
      cp_commit();
      if (np == 0) { pb0 = b; pt0 = tile; }
      else if (np == 1) { pb1 = b; pt1 = tile; }
      else { pb2 = b; pt2 = tile; }
      ++np;
    };
    uint32_t n = 0, qn = 0;
    const int64_t st = a.pool.stride_t;
    const int c = lane % PIECES, sub = lane / PIECES;
    while (next_segment(u, sg)) {
      const int nj = sg.nj[0] > sg.nj[1] ? sg.nj[0] : sg.nj[1];
      if (nj == 0) continue;
      const uint8_t* kbase = a.pool.k + sg.kvh * a.pool.stride_h + c * 16;
      const uint8_t* vbase = a.pool.v + sg.kvh * a.pool.stride_h + c * 16;
      const int64_t first = sg.key0 + 32 * w;        // this warp's first key of tile 0
      // Pages of this warp's two runs of 16 keys of key tile j (a run never crosses a page), -1 where there is
      // nothing to read.  Loaded one tile ahead.
      auto page_at = [&](int j, int run) -> int32_t {
        const int64_t key = first + static_cast<int64_t>(j) * 128 + 16 * run;
        if (j >= nj || key >= sg.lk) return -1;
        const int64_t col = key >> shift;
        if (prefix) return __ldg(a.prefix_pages + col);
        return col < a.pt.cols ? __ldg(a.pt.table + sg.b * a.pt.stride + col) : -2;
      };
      // Copies this warp's rows of one tile; base[run]: the run's first row, valid[run]: its rows to read
      auto copy_rows = [&](uint32_t tile, const uint8_t* base, const int64_t (&off)[2], const int (&valid)[2]) {
#pragma unroll
        for (int run = 0; run < 2; ++run) {
          const uint8_t* src = base + off[run];
#pragma unroll
          for (int i = 0; i < 16 / RPI; ++i) {
            const int rr = i * RPI + sub;
            const int r = 32 * w + 16 * run + rr;
            const uint32_t dst = tile + (INT8 ? CODE_OFF : (c >> 3) * C::HALF) + r * 128 + (((c & 7) ^ (r & 7)) << 4);
            const bool real = rr < valid[run];
            cp16(dst, real ? src + rr * st : base, real);
          }
        }
      };
      int32_t page[2] = {page_at(0, 0), page_at(0, 1)};
      // Q of both tiles, once the MMAs of the last segment have read theirs
      if (np == 3) finish_oldest();
      if (qn > 0) acquire(bar(T_QEMPTY), (qn - 1) & 1);
      ++qn;
      {
        constexpr int QP = D / 8;
        const int qc = lane % QP;
        const uint32_t row0 = static_cast<uint32_t>(sg.row0), gg = static_cast<uint32_t>(g);
        const __half* qbase = a.q + sg.start * a.q_t + static_cast<int64_t>(sg.kvh) * g * a.q_h + qc * 8;
#pragma unroll 4
        for (int i = 0; i < 2 * QP; ++i) {      // 64 rows of this warp, 32 / QP at a time
          const int k = i * (32 / QP) + lane / QP;
          const int t = k >> 5, r = 32 * w + (k & 31);
          const int pr = 128 * t + r;
          const bool real = pr < sg.rows;
          const uint32_t row = row0 + pr, tok = row / gg;
          const __half* src = real ? qbase + tok * a.q_t + (row - tok * gg) * a.q_h : a.q;
          cp16(sbase + t * C::Q_BYTES + (qc >> 3) * C::HALF + r * 128 + (((qc & 7) ^ (r & 7)) << 4), src, real);
        }
        pushed(bar(T_QFULL), 0);
      }
      float nks = 0.f, nvs = 0.f;      // INT8: scales of this lane's key, loaded while K is copied
      for (int j = 0; j < nj; ++j, ++n) {
        int64_t off[2];
        int valid[2];
#pragma unroll
        for (int run = 0; run < 2; ++run) {
          const int64_t key = first + static_cast<int64_t>(j) * 128 + 16 * run;
          const int64_t left = sg.lk - key;
          bool use = left > 0;
          if (use && !page_ok(page[run], a.pool.num_pages)) {
            if (lane == 0) dev_error(err, TM_DEVERR_SEQLEN);
            use = false;
          }
          valid[run] = use ? (left < 16 ? static_cast<int>(left) : 16) : 0;
          off[run] = use ? page[run] * a.pool.stride_page + (key & page_mask) * a.pool.stride_t : 0;
        }
        if (INT8) {
          const int run = lane >> 4;
          const int64_t key = first + static_cast<int64_t>(j) * 128 + lane;
          nks = nvs = 0.f;
          if ((lane & 15) < valid[run]) {
            const int64_t so = page[run] * a.pool.sstride_page + (key & page_mask) * a.pool.sstride_t +
                               sg.kvh * a.pool.sstride_h;
            nks = __half2float(a.pool.ks[so]);
            nvs = __half2float(a.pool.vs[so]);
          }
        }
        page[0] = page_at(j + 1, 0);
        page[1] = page_at(j + 1, 1);
#pragma unroll
        for (int v = 0; v < 2; ++v) {
          const uint32_t i = 2 * n + v, slot = i % C::NSLOT, lap = i / C::NSLOT;
          if (lap > 0) acquire(bar(T_EMPTY + slot), (lap - 1) & 1);
          else if (np == 3) finish_oldest();
          const uint32_t tile = sbase + C::OFF_SLOT + slot * C::SLOT;
          copy_rows(tile, v ? vbase : kbase, off, valid);
          if (INT8 && v) {      // the V tile's release frees its stage of scales
            float* s = scales + (slot >> 1) * 384 + 32 * w + lane;
            const float f = nvs == 0.f ? 5.9604645e-8f : nvs;   // a zero scale (codes all 0) counts in the row sum alone
            s[0] = nks * a.scale_log2;
            s[128] = log2f(f);
            s[256] = 1.0f / f;
          }
          pushed(bar(T_FULL + slot), INT8 ? tile : 0u);
        }
      }
    }
    while (np > 0) finish_oldest();
  } else if (warp >= 8) {
    regs_dec<C::OTHER_REGS>();
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
        named_bar_sync(NB_P + t, 160);      // softmax t stored P_t(c)
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
            if (t == 1 && j == 0 && no > 0) named_bar_sync(NB_START, 160);
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
    const int64_t total = a.T * Hq;
    const bool direct = p.slots == 1;
    while (next_segment(u, sg)) {
      const int nt = sg.nj[t];
      const int pr = 128 * t + r;
      const bool row_ok = pr < sg.rows;
      const int64_t prow = sg.row0 + pr;
      const int64_t tok_in = prow / g;
      const int64_t tok = sg.start + tok_in;
      const int head = sg.kvh * g + static_cast<int>(prow - tok_in * g);
      int64_t lim = 0;
      if (row_ok) {
        lim = sg.lk;
        if (!prefix && a.causal && sg.hidden + tok_in < lim) lim = sg.hidden + tok_in;
      }
      float m_used = -INFINITY, l = 0.f;
      for (int c = 0; c < 2 * nt; ++c, ++cc) {
        const int sl = c & 1;
        const uint32_t s_c = s_addr + HN * sl;
        mbar_wait(bar(T_SFULL + 2 * t + sl), (cc >> 1) & 1, err, abort_flag);
        const uint32_t vi = 2 * (n + (c >> 1)) + 1;   // ring position of this key tile's V
        if (INT8 && sl == 0) mbar_wait(bar(T_FULL + vi % C::NSLOT), (vi / C::NSLOT) & 1, err, abort_flag);
        tc_fence_after();
        __syncwarp();
        float x[HN];
        {
          uint32_t v[HN];
#pragma unroll
          for (int q = 0; q < HN / 32; ++q) tmem_ld32p(s_c + q * 32, v + q * 32);
          tmem_wait_ld_regs<HN>(v);
#pragma unroll
          for (int e = 0; e < HN; ++e) x[e] = __uint_as_float(v[e]);
        }
        const float* sc = scales + ((vi % C::NSLOT) >> 1) * 384 + HN * sl;
        if (INT8) {
#pragma unroll
          for (int e = 0; e < HN; e += 4) {
            const float4 k4 = *reinterpret_cast<const float4*>(sc + e);
            const float4 v4 = *reinterpret_cast<const float4*>(sc + 128 + e);
            f2unpack(f2fma(f2pack(x[e], x[e + 1]), f2pack(k4.x, k4.y), f2pack(v4.x, v4.y)), x[e], x[e + 1]);
            f2unpack(f2fma(f2pack(x[e + 2], x[e + 3]), f2pack(k4.z, k4.w), f2pack(v4.z, v4.w)), x[e + 2], x[e + 3]);
          }
        }
        const float cs = INT8 ? 1.0f : a.scale_log2;
        const int64_t nv64 = lim - (sg.key0 + static_cast<int64_t>(c) * HN);
        const int nv = nv64 <= 0 ? 0 : (nv64 >= HN ? HN : static_cast<int>(nv64));
        if (!__all_sync(0xffffffffu, nv == HN)) {
#pragma unroll
          for (int e = 0; e < HN; ++e) x[e] = (e < nv) ? x[e] : -INFINITY;
        }
        float alpha = 1.f;
        if (nv > 0) {
          const float mt = row_max<HN>(x) * cs;
          if (mt > m_used + kLazy) {
            alpha = ex2_approx(m_used - mt);
            m_used = mt;
          }
        }
        const float msub = (m_used == -INFINITY) ? 0.f : m_used - kPOffset;
        const uint64_t c2 = f2pack(cs, cs), nm2 = f2pack(-msub, -msub);
        uint32_t pk[HN / 2];
        uint64_t acc2[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
        for (int e = 0; e < HN; e += 2) {
          const uint64_t y2 = INT8 ? f2add(f2pack(x[e], x[e + 1]), nm2) : f2fma(f2pack(x[e], x[e + 1]), c2, nm2);
          float p0, p1;
          if (((e >> 1) & 7) < kFmaPairs) {
            exp2_fma2(y2, p0, p1);
          } else {
            float y0, y1;
            f2unpack(y2, y0, y1);
            p0 = ex2_approx(y0);
            p1 = ex2_approx(y1);
          }
          if (INT8) {
            const float2 iv = *reinterpret_cast<const float2*>(sc + 256 + e);
            acc2[(e >> 1) & 3] = f2fma(f2pack(p0, p1), f2pack(iv.x, iv.y), acc2[(e >> 1) & 3]);
          } else {
            acc2[(e >> 1) & 3] = f2add(acc2[(e >> 1) & 3], f2pack(p0, p1));
          }
          pk[e >> 1] = pack_half2(p0, p1);
        }
        {
          const uint64_t s2 = f2add(f2add(acc2[0], acc2[1]), f2add(acc2[2], acc2[3]));
          float s0, s1;
          f2unpack(s2, s0, s1);
          l = l * alpha + (s0 + s1);
        }
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
        if (t == 0 && c == 0 && sg.nj[1] > 0) named_bar_arrive(NB_START, 160);
        named_bar_sync(NB_P + t, 160);
      }
      n += sg.nj[0] > sg.nj[1] ? sg.nj[0] : sg.nj[1];

      // ---- the row's result: partial (O, m, l), or the output
      if (m_used == -INFINITY) l = 0.f;      // a row that saw nothing
      if (nt > 0) {
        mbar_wait(bar(T_OLAST + t), segs & 1, err, abort_flag);
        ++segs;
        tc_fence_after();
        __syncwarp();
      }
      const int64_t idx = sg.slot * total + tok * Hq + head;
      if (row_ok && !direct) a.ml[idx] = make_float2(m_used, l);
      const float inv = l > 0.f ? 1.f / l : (l == 0.f ? 0.f : l);
      if (nt > 0 || direct) {
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
          if (row_ok && direct) {
            __half* dst = a.out + tok * a.o_t + head * a.o_h + q * 32;
#pragma unroll
            for (int e = 0; e < 32; e += 8) {
              uint32_t h[4];
#pragma unroll
              for (int i = 0; i < 4; ++i)
                h[i] = pack_half2(__uint_as_float(o[e + 2 * i]) * inv, __uint_as_float(o[e + 2 * i + 1]) * inv);
              *reinterpret_cast<uint4*>(dst + e) = make_uint4(h[0], h[1], h[2], h[3]);
            }
          } else if (row_ok) {
            float* dst = a.o + idx * D + q * 32;
#pragma unroll
            for (int e = 0; e < 32; e += 4)
              *reinterpret_cast<uint4*>(dst + e) = make_uint4(o[e], o[e + 1], o[e + 2], o[e + 3]);
          }
          __syncwarp();           // tensor-memory loads are the whole warp's
        }
        tc_fence_before();      // these reads of O come before the next segment's first P.V
      }
    }
  }

  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  pdl_wait();      // whoever waits for this kernel has waited for the one before it
}

}  // namespace

template <int D, bool INT8>
static tm_status launch_tile(const SharedArgs& a, bool prefix, bool overlap, DevErr err, cudaStream_t stream) {
  constexpr int smem = CfgT<D>::SMEM;
  static std::atomic<uint64_t> prepared{0};
  tm_status st = prepare_smem(tile_kernel<D, INT8>, smem, prepared);
  if (st != TM_OK) return st;
  const SharedPlan& p = a.plan;
  const int64_t items = prefix ? p.pre_ctas : static_cast<int64_t>(p.own_splits) * a.batch * p.own_rows * a.pool.H;
  return launch_kernel(tile_kernel<D, INT8>, items, kThreads, smem, overlap, stream, a, prefix ? 1 : 0, err);
}

tm_status shared_tile(const SharedArgs& a, int d, bool int8, bool prefix, bool overlap, DevErr err,
                      cudaStream_t stream) {
  if (d == 128) return int8 ? launch_tile<128, true>(a, prefix, overlap, err, stream)
                            : launch_tile<128, false>(a, prefix, overlap, err, stream);
  return int8 ? launch_tile<64, true>(a, prefix, overlap, err, stream)
              : launch_tile<64, false>(a, prefix, overlap, err, stream);
}

}  // namespace tmk
