// tm_attn_shared.cu -- attention of a batch over a paged cache behind a shared
// prefix (tm_attn_shared_prefix): the split-key kernel for few rows, and the
// join of partial results.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include <atomic>

#include "tm_attn_shared.cuh"

namespace tmk {

SharedPlan shared_plan(int64_t T, int32_t Hq, int32_t Hkv, int32_t d, bool int8, int32_t batch, int64_t max_seqlen,
                       int64_t prefix_len, int64_t max_kv_len) {
  SharedPlan p{};
  p.group = Hq / Hkv;
  if (max_seqlen > T) max_seqlen = T;      // no sequence has more rows
  if (max_seqlen < 1) max_seqlen = 1;      // of 0: sequences that have rows all the same are to be met
  const int64_t own_packed = max_seqlen * p.group, pre_packed = T * p.group;
  // Items are counted in 32 bits, on the tile kernel by blocks that step over one another.
  const int64_t most = 0x7fffffff - kSmsB200;
  if (ceil_div(own_packed, 256) * batch * Hkv > most) {
    p.bytes = -1;
    return p;
  }
  int64_t own_units = ceil_div(max_kv_len, 128), pre_units = ceil_div(prefix_len, 128);
  if (own_units == 0 && pre_units == 0) own_units = 1;      // nothing to see: one kernel, for the zeros
  p.own_tile = own_on_tiles(own_packed, own_units);
  if (p.own_tile && prefix_len + max_kv_len < (1 << 30) &&
      prefix_folded(batch * ceil_div(own_packed, 256) * Hkv, ceil_div(pre_packed, 256) * Hkv, pre_units)) {
    p.fold = static_cast<int>(pre_units);
    own_units += pre_units;
    pre_units = 0;
  }
  p.pre_tile = prefix_on_tiles(ceil_div(pre_packed, 16) * Hkv, ceil_div(pre_packed, 256) * Hkv, pre_units);
  // blocks of eight rows where sequences have no more, and a prefix in such blocks costs little next to them
  p.narrow = !p.own_tile && own_packed <= split_block(true) &&
             (p.pre_tile || pre_packed <= split_block(true) ||
              4 * ceil_div(pre_packed, split_block(true)) * pre_units <= batch * own_units);
  const int block = split_block(p.narrow);
  const int64_t own_rows = ceil_div(own_packed, p.own_tile ? 256 : block);
  const int64_t pre_rows = ceil_div(pre_packed, p.pre_tile ? 256 : block);
  p.own_rows = static_cast<int>(own_rows);
  p.pre_rows = static_cast<int>(pre_rows);
  // Split kernel: the pieces that end soonest, as waves of CTAs, each its key tiles and a start and end worth two
  // more, and half a tenth of one for every result that the join reads.  Own lengths are known on the device alone: 0.6
  // of the longest is assumed, and that their CTAs, of all lengths, leave a last wave less empty than the prefix's.
  // Five CTAs per SM whatever the lengths took 13.7 us instead of 10.4 (8 tokens behind 2000 positions) and
  // 16.4 instead of 12.7 (20 sequences of up to 200 tokens behind 1000).
  const int64_t pre_blocks = p.pre_tile ? 0 : pre_rows * Hkv, own_blocks = p.own_tile ? 0 : batch * own_rows * Hkv;
  const int64_t resident = split_resident(d, int8, p.narrow) * kSmsB200;
  int64_t chunk = 1, best = 0;
  // With many own key tiles the lengths alone fill the last waves, and what counts is that the pieces are long: five
  // CTAs per SM (32 sequences of up to 2000 tokens, INT8: 32.0 us, by waves 37.9).
  const bool many = own_blocks * own_units > 13 * kSmsB200;
  if (many) chunk = ceil_div(own_blocks * own_units + pre_blocks * pre_units, 5 * kSmsB200);
  const int64_t longest = own_units > pre_units ? own_units : pre_units;
  if (chunk > longest) chunk = longest;      // below 2^23 key tiles
  for (int64_t c = 1; !many && c <= 64 && (c == 1 || c <= longest); ++c) {
    const int64_t pre_ctas = pre_blocks * ceil_div(pre_units, c);
    const int64_t own_ctas = own_blocks * ceil_div((own_units * 6 + 9) / 10, c);
    const int64_t tenths = 10 * (pre_ctas + own_ctas) / resident;      // of a wave
    const int64_t waves = own_ctas > pre_ctas ? (tenths + 3 > 10 ? tenths + 3 : 10) : (tenths < 10 ? 10 : tenths + 6);
    const int64_t results = (pre_blocks > 0 ? ceil_div(pre_units, c) : 0) + (own_blocks > 0 ? ceil_div(own_units, c) : 0);
    const int64_t cost = waves * (20 + 10 * c) / 10 + results / 2;
    if (best == 0 || cost < best) {
      best = cost;
      chunk = c;
    }
  }
  if (p.pre_tile) {
    // Equal pieces of the line of key tiles, one for each SM; or, where that costs a CTA at most kSplitBlockTiles more
    // key tiles, equal pieces of every row block, so that no CTA pays a second block's start and end.
    const int64_t blocks = Hkv * pre_rows, line = blocks * pre_units;
    if (line >= (1ll << 31)) {
      p.bytes = -1;
      return p;
    }
    const int64_t least = ceil_div(pre_units, kMostSplits);
    int64_t c = ceil_div(line, kSmsB200);
    if (blocks <= kSmsB200) {
      const int64_t whole = ceil_div(pre_units, kSmsB200 / blocks);
      if (whole <= c + kSplitBlockTiles) {
        c = whole;
        p.pre_pieces = 1;
      }
    }
    if (c < least) c = least;
    if (c < 1) c = 1;
    p.pre_tiles = static_cast<int>(pre_units);
    if (p.pre_pieces != 0) {
      p.pre_pieces = static_cast<int>(ceil_div(pre_units, c));
      p.pre_chunk = static_cast<int>(ceil_div(pre_units, p.pre_pieces));
      p.pre_pieces = static_cast<int>(ceil_div(pre_units, p.pre_chunk));
      p.pre_ctas = static_cast<int>(blocks * p.pre_pieces);
      p.pre_splits = p.pre_pieces;
    } else {
      if (c > line) c = line;
      p.pre_chunk = static_cast<int>(c);
      p.pre_ctas = static_cast<int>(ceil_div(line, c));
      p.pre_splits = static_cast<int>(line <= c ? 1 : (pre_units % c == 0 ? pre_units / c : ceil_div(pre_units - 1, c) + 1));
    }
  } else {
    const int64_t c = chunk > ceil_div(pre_units, kMostSplits) ? chunk : ceil_div(pre_units, kMostSplits);
    p.pre_chunk = static_cast<int>((c < 1 ? 1 : c) * 128);
    p.pre_splits = static_cast<int>(ceil_div(pre_units, c < 1 ? 1 : c));
  }
  int64_t c = chunk;
  if (p.own_tile) {
    // as many splits as end soonest: waves of items, each its key tiles and a start worth kItemTiles more
    const int64_t items = batch * own_rows * Hkv;
    int64_t least = 0;
    for (int64_t s = 1; s <= kMostSplits && s <= own_units; ++s) {
      const int64_t cost = ceil_div(items * s, kSmsB200) * (ceil_div(own_units, s) + kItemTiles) + (s > 1 ? kItemTiles : 0);
      if (least == 0 || cost < least) {
        least = cost;
        c = ceil_div(own_units, s);
      }
    }
  }
  if (c < ceil_div(own_units, kMostSplits)) c = ceil_div(own_units, kMostSplits);
  if (c < 1) c = 1;
  p.own_chunk = static_cast<int>(c * 128);
  p.own_splits = static_cast<int>(ceil_div(own_units, c));
  p.slots = p.own_splits + p.pre_splits;
  const int64_t items = own_rows * batch * Hkv * p.own_splits + (p.pre_tile ? 0 : pre_rows * Hkv * p.pre_splits);
  if (items > most) {
    p.bytes = -1;
    return p;
  }
  const int64_t rows = T * Hq;
  p.ml_bytes = (p.slots * rows * 8 + 255) / 256 * 256;
  p.bytes = p.slots > 1 ? p.ml_bytes + p.slots * rows * d * 4 : 0;
  if (p.bytes < 256) p.bytes = 256;
  return p;
}

namespace {

constexpr int kWarps = 4;
constexpr int kStep = 16;     // keys of one warp step: never more than one page
constexpr int kStages = 3;
// 2^kPOffset is the largest weight when the reference is the maximum; scores
// above it leave it alone up to this exponent: 2^15 at most, inside fp16.  (What
// counts is the exponent as it is computed: 2^24 and more from zero, a score
// and a reference have steps of 2 and more.)
constexpr float kTop = 15.0f;

__device__ __forceinline__ void ldsm4(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void ldsm4t(uint32_t a, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(a)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
// An 8 x 8 matrix of fp16, two columns of row lane / 4 in each lane, transposed.
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
__device__ __forceinline__ uint2 lds64(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a) : "memory");
  return v;
}

// Bytes of one 16-key stage of K (V the same), and where the 16-byte piece c
// of key row `row` lies in it: as the TMA copy of 16 rows writes it, 64
// columns (fp16) at a time in the 128-byte swizzle, INT8 rows of 64 bytes in the
// 64-byte one.  The reads below (ldmatrix of eight rows; 16-byte reads of
// codes) meet banks at most twice.
template <int D, bool INT8>
struct Stage {
  static constexpr int ROW = D * (INT8 ? 1 : 2);
  static constexpr int BYTES = kStep * ROW;
  static constexpr int PIECES = ROW / 16;
  __device__ static __forceinline__ uint32_t at(int row, int c) {
    if (INT8 && D == 64) return row * 64 + ((c ^ ((row >> 1) & 3)) << 4);
    return (c >> 3) * (kStep * 128) + row * 128 + (((c & 7) ^ (row & 7)) << 4);
  }
};

template <int D, bool INT8>
struct SplitSmem {
  static constexpr int RING = kWarps * kStages * 2 * Stage<D, INT8>::BYTES;
  static constexpr int OFF_SCALE = RING;                                              // [warp][stage][3][16] floats
  static constexpr int OFF_ML = OFF_SCALE + (INT8 ? kWarps * kStages * 3 * kStep * 4 : 0);   // [warp][16] (m, l)
  static constexpr int OFF_BAR = OFF_ML + kWarps * 16 * 8;                            // [warp][stage], abort flag
  static constexpr int BYTES = OFF_BAR + kWarps * kStages * 8 + 16 + 1024;
};

// Attention of up to 16 packed rows (NARROW: 8) over one range of keys.
//
// Decoding reads far more than it computes (a key's 2 d values serve g rows),
// so this is built around the copies: each warp owns every fourth 16-key step
// and its own three-stage ring, with no barrier between warps until the join at
// the end.  A warp's step is a chain of dependent
// instructions, so it takes several warps to keep up with the copies: at
// d = 128 in fp16 two CTAs (eight warps, 192 KB of rings) fit an SM, else
// three or four.  Measured with 32 single tokens, 32 query heads over 8: behind
// 16000 own tokens each, fp16, 2.1 GB in 299 us (7.0 TB/s, HBM's rate); INT8, 1.07
// GB in 215 us (5.0 TB/s: four warps a scheduler wait for one another's chains of
// dependent instructions, the conversion's among them); behind 200 to 2000,
// where starts, ends and the join weigh, 144 MB in 30 us.  A step's keys lie in one page, so a TMA copy
// brings its K (two at d = 128 in fp16), another its V, for a dozen
// instructions where row copies took over a hundred.  A step that the range
// ends in, or on a bad page, is copied row by row: rows past the end are zeros and
// never read from memory.  The products run on mma.sync m16n8k16: 16 rows
// hold a whole group of query heads, where a 128-row tensor-memory tile would
// be nearly empty.  NARROW, for single tokens with up to eight query heads for a
// K/V head, turns the products over: S^T = K Q^T and O^T = V^T P^T, keys and
// dimensions on the 16 rows and the query rows on the 8 columns, with half the
// MMAs, exponentials and sums (four INT8 CTAs on an SM, not three; behind 4000 own
// tokens 77 -> 65 us in INT8, 83.5 -> 81.7 us in fp16).  P^T is the transpose of
// S^T's fragments, one movmatrix for each 8 x 8.
//
// INT8: K and V stay codes in shared memory and become fp16 in registers
// (exactly).  With t_j = s_j ks_j + log2 vs_j the weights 2^(t_j - m) carry
// the V scale, and the row sum takes 2^(t_j - m) / vs_j: no rounding is added
// and the weights keep fp16's range whatever the scales are.  The code layouts
// follow the fragments: the order of d within the QK^T sum is free, so a
// lane's 16 consecutive codes serve four MMAs; the order of output columns is
// free too, so a lane's n index stands for d / 8 consecutive dimensions.
template <int D, bool INT8, bool NARROW>
__device__ __forceinline__ void split_rows(const SharedArgs& a, const PageMaps& maps, DevErr err) {
  using S = Stage<D, INT8>;
  using L_ = SplitSmem<D, INT8>;
  constexpr int KS = D / 16;
  constexpr int NT = NARROW ? D / 16 : D / 8;      // tiles of O
  constexpr int BR = split_block(NARROW);
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = smem_raw + ((1024u - (smem_u32(smem_raw) & 1023u)) & 1023u);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int quad = lane & 3, r8 = lane >> 2;
  const SharedPlan& p = a.plan;
  const int H = a.pool.H, g = p.group, Hq = H * g;

  // ---- which rows and keys (packed rows and keys stay below 2^31)
  int item = blockIdx.x;
  const int kvh = item % H;
  item /= H;
  const int pre_items = p.pre_tile ? 0 : p.pre_splits * p.pre_rows;
  const bool prefix = item < pre_items;
  int b = 0, slot, row0, start = 0, nrows, k0, k1;
  int hidden = 0;         // own, causal: token i of the sequence sees keys below hidden + i
  if (prefix) {
    slot = item / p.pre_rows;
    row0 = (item - slot * p.pre_rows) * BR;
    nrows = static_cast<int>(a.T) * g;
    k0 = slot * p.pre_chunk;
    k1 = min(k0 + p.pre_chunk, static_cast<int>(a.prefix_len));
  } else {
    item -= pre_items;
    const int per = a.batch * p.own_rows;
    const int split = item / per;
    item -= split * per;
    b = item / p.own_rows;
    row0 = (item - b * p.own_rows) * BR;
    slot = p.pre_splits + split;
    k0 = split * p.own_chunk;
  }
  // the first steps' table entries, before the lengths are known: one latency less
  const int shift = a.pool.page_shift, page_mask = (1 << shift) - 1;
  const int first = k0 + warp * kStep;
  const int key_bound = prefix ? static_cast<int>(a.prefix_len) : static_cast<int>(a.max_kv);
  auto raw_entry = [&](int key) -> int32_t {
    const int col = key >> shift;
    if (key >= key_bound || (!prefix && col >= a.pt.cols)) return -1;
    return __ldg(prefix ? a.prefix_pages + col : a.pt.table + b * a.pt.stride + col);
  };
  int32_t page = raw_entry(first), page1 = raw_entry(first + kWarps * kStep), page2 = raw_entry(first + 2 * kWarps * kStep);
  if (!prefix) {
    int64_t start64, n64;
    seq_rows(a, b, start64, n64);
    const bool outside = rows_outside(a, start64, n64, BR);
    if (outside && threadIdx.x == 0) dev_error(err, TM_DEVERR_SEQLEN);   // offsets that the launch was not sized for
    const int n = static_cast<int>(n64);
    if (outside || row0 >= n * g) return;
    start = static_cast<int>(start64);
    nrows = n * g;
    int lk = __ldg(a.kv_lens + b);
    if (lk > a.max_kv) {
      if (threadIdx.x == 0) dev_error(err, TM_DEVERR_SEQLEN);
      lk = static_cast<int>(a.max_kv);
    }
    lk = max(lk, 0);
    hidden = lk - n + 1;
    k1 = min(k0 + p.own_chunk, lk);
    if (a.causal) k1 = min(k1, hidden + (min(row0 + BR, nrows) - 1) / g);   // keys that the block's last row sees
  }
  const int rows = min(nrows - row0, BR);
  const int64_t total = a.T * Hq;
  const bool direct = p.slots == 1;

  // (token, query head) of packed row r of this block
  auto token_of = [&](int r) { return start + (row0 + r) / g; };
  auto head_of = [&](int r) { return kvh * g + (row0 + r) % g; };

  if (k0 >= k1) {     // nothing visible here
    if (!direct) {
      if (threadIdx.x < rows)
        a.ml[slot * total + static_cast<int64_t>(token_of(threadIdx.x)) * Hq + head_of(threadIdx.x)] =
            make_float2(-INFINITY, 0.f);
    } else {
      for (int i = threadIdx.x; i < rows * (D / 8); i += kWarps * 32) {
        const int r = i / (D / 8);
        if (token_of(r) < rows_in_use(a) && token_of(r) >= first_row(a))
          *reinterpret_cast<uint4*>(a.out + token_of(r) * a.o_t + head_of(r) * a.o_h + (i % (D / 8)) * 8) =
              make_uint4(0, 0, 0, 0);
      }
    }
    return;
  }

  uint8_t* ring = smem + warp * kStages * 2 * S::BYTES;
  const uint32_t ring_s = smem_u32(ring);
  float* scales = reinterpret_cast<float*>(smem + L_::OFF_SCALE) + warp * kStages * 3 * kStep;
  float2* ml_s = reinterpret_cast<float2*>(smem + L_::OFF_ML);
  const uint32_t bar0 = smem_u32(smem + L_::OFF_BAR) + warp * kStages * 8;
  volatile int* abort_flag = reinterpret_cast<volatile int*>(smem + L_::OFF_BAR + kWarps * kStages * 8);
  if (lane == 0) {
    for (int i = 0; i < kStages; ++i) mbar_init(bar0 + 8 * i, 1);
    *abort_flag = 0;
    fence_barrier_init();
  }
  __syncwarp();

  const int steps = first < k1 ? (k1 - first + kWarps * kStep - 1) / (kWarps * kStep) : 0;
  // page of step i as the table has it; -1 where nothing is to be read
  auto entry_at = [&](int i) -> int32_t { return i < steps ? raw_entry(first + i * (kWarps * kStep)) : -1; };
  uint32_t by_tma = 0;      // bit s: stage s is filled by TMA
  const uint64_t policy = keys_policy(prefix ? p.pre_rows : p.own_rows);
  struct Scales {
    __half k, v;      // as loaded: a conversion would wait for the load
  };
  // INT8: a step's scales, as issue() loaded them, into its stage
  auto keep_scales = [&](int st, const Scales& x) {
    if (!INT8 || lane >= kStep) return;
    float* sc = scales + st * 3 * kStep + lane;
    const float v = __half2float(x.v), f = v == 0.f ? 5.9604645e-8f : v;   // a zero scale (codes all 0) counts in the row sum alone
    sc[0] = __half2float(x.k) * a.scale_log2;
    sc[kStep] = __log2f(f);             // within 2^-18 (two units in the last place of up to 24): a weight's relative error
    sc[2 * kStep] = __frcp_rn(f);
  };
  // copies of step i into stage st
  auto issue = [&](int i, int st, int32_t page, Scales& sc) {
    if (i < steps) {
      const int key = first + i * (kWarps * kStep), s = key & page_mask;
      const bool ok = page_ok(page, a.pool.num_pages);
      if (!ok && lane == 0) dev_error(err, TM_DEVERR_SEQLEN);
      const int valid = ok ? min(k1 - key, kStep) : 0;
      if (INT8) {
        const int64_t so = page * a.pool.sstride_page + (s + lane) * a.pool.sstride_t + kvh * a.pool.sstride_h;
        sc.k = sc.v = __float2half(0.f);
        if (lane < valid) {
          sc.k = a.pool.ks[so];
          sc.v = a.pool.vs[so];
        }
      }
      const uint32_t dst = ring_s + st * 2 * S::BYTES;
      if (maps.ok && valid == kStep) {
        by_tma |= 1u << st;
        if (elect_one()) {
          const uint32_t bar = bar0 + 8 * st;
          mbar_arrive_expect_tx(bar, 2 * S::BYTES);
          const int32_t c1 = maps.heads_inner ? kvh : s, c2 = maps.heads_inner ? s : kvh;
#pragma unroll
          for (int hh = 0; hh < (INT8 ? 1 : D / 64); ++hh) {
            tma_load_4d(dst + hh * kStep * 128, &maps.k, bar, hh * 64, c1, c2, page, policy);
            tma_load_4d(dst + S::BYTES + hh * kStep * 128, &maps.v, bar, hh * 64, c1, c2, page, policy);
          }
        }
        __syncwarp();
      } else {
        by_tma &= ~(1u << st);
        constexpr int RPI = 32 / S::PIECES;          // rows of one copy instruction
        const int c = lane % S::PIECES;
        const int64_t off = (valid > 0 ? page * a.pool.stride_page + s * a.pool.stride_t : 0) + kvh * a.pool.stride_h + c * 16;
#pragma unroll 1
        for (int row = lane / S::PIECES; row < kStep; row += RPI) {
          const bool real = row < valid;
          const int64_t at = real ? off + row * a.pool.stride_t : 0;
          cp16(dst + S::at(row, c), a.pool.k + at, real);
          cp16(dst + S::BYTES + S::at(row, c), a.pool.v + at, real);
        }
      }
    }
    cp_commit();
  };
  Scales sc_a{}, sc_b{};
  issue(0, 0, page, sc_a);
  issue(1, 1, page1, sc_b);
  page = page2;

  // ---- this lane's rows: limits and Q fragments, while the first copies are under way
  // In scores, weights and O a lane holds rows r8 and r8 + 8 (NARROW: 2 quad and 2 quad + 1).
  auto row_of = [&](int h) { return NARROW ? 2 * quad + h : r8 + 8 * h; };
  int lim[2];
  uint32_t qf[KS][NARROW ? 2 : 4];      // NARROW: the B operand, row r8
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    lim[i] = k1;
    if (!prefix && a.causal && row_of(i) < rows) lim[i] = min(k1, hidden + (row0 + row_of(i)) / g);
  }
  constexpr int QH = NARROW ? 1 : 2;
#pragma unroll
  for (int i = 0; i < QH; ++i) {
    const int r = r8 + 8 * i;
    const bool real = r < rows;
    const __half* q = real ? a.q + token_of(r) * a.q_t + head_of(r) * a.q_h : a.q;
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      if (INT8) {
        // k-step s takes word s % 4 of the lane's 16-byte piece at 64 (s / 4) + 16 quad
        const int at = (s >> 2) * 64 + quad * 16 + (s & 3) * 4;
        const uint2 v = real ? *reinterpret_cast<const uint2*>(q + at) : make_uint2(0, 0);
        qf[s][i] = v.x;
        qf[s][QH + i] = v.y;
      } else {
        qf[s][i] = real ? *reinterpret_cast<const uint32_t*>(q + 16 * s + 2 * quad) : 0u;
        qf[s][QH + i] = real ? *reinterpret_cast<const uint32_t*>(q + 16 * s + 8 + 2 * quad) : 0u;
      }
    }
  }
  // steps that end at or below this key need no mask
  int open = k1;
  if (!prefix && a.causal) open = min(open, hidden + row0 / g);

  float o[NT][4];
#pragma unroll
  for (int i = 0; i < NT; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};

  if (steps > 0) keep_scales(0, sc_a);
  if (steps > 1) keep_scales(1, sc_b);
  int st = 0;
  uint32_t laps = 0;        // bit s: parity of stage s's next TMA fill
  for (int i = 0; i < steps; ++i) {
    cp_wait<1>();           // this step's row copies, if any
    if (by_tma >> st & 1) {
      mbar_wait(bar0 + 8 * st, laps >> st & 1, err, abort_flag);
      laps ^= 1u << st;
    }
    __syncwarp();
    const int freed = st == 0 ? kStages - 1 : st - 1;        // the stage that step i - 1 used
    issue(i + 2, freed, page, sc_a);
    page = entry_at(i + 3);
    const uint32_t ks_s = ring_s + st * 2 * S::BYTES;
    const uint32_t vs_s = ks_s + S::BYTES;
    const int sc_st = st;
    const int key0 = first + i * (kWarps * kStep);
    st = st == kStages - 1 ? 0 : st + 1;

    // Scores: x[j][2 h + e] is key 8 j + 2 quad + e against row r8 + 8 h; NARROW: x[j][h] key 8 j + r8 against row 2 quad + h
    constexpr int XE = NARROW ? 2 : 4;
    float x[2][XE], iv[2][2];
    const float* sc = scales + sc_st * 3 * kStep + (NARROW ? r8 : 2 * quad);
    if constexpr (NARROW) {
      // K is the A operand; four sums, so that two dependent MMAs are the longest chain at d = 128
      float s[4][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) s[j][0] = s[j][1] = s[j][2] = s[j][3] = 0.f;
      if (!INT8) {
#pragma unroll
        for (int ks = 0; ks < KS; ++ks) {
          uint32_t afr[4];
          ldsm4(ks_s + S::at(lane & 15, 2 * ks + (lane >> 4)), afr);
          mma16816(s[ks & 3], afr, qf[ks][0], qf[ks][1]);
        }
      } else {
#pragma unroll
        for (int c = 0; c < KS / 4; ++c) {
          const uint4 v = lds128(ks_s + S::at(r8, 4 * c + quad)), u = lds128(ks_s + S::at(8 + r8, 4 * c + quad));
          const uint32_t w[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u};
          const uint32_t y[4] = {u.x ^ 0x80808080u, u.y ^ 0x80808080u, u.z ^ 0x80808080u, u.w ^ 0x80808080u};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t afr[4] = {codes2(w[e], 0x4140u), codes2(y[e], 0x4140u), codes2(w[e], 0x4342u),
                                     codes2(y[e], 0x4342u)};
            mma16816(s[e], afr, qf[4 * c + e][0], qf[4 * c + e][1]);
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const float kj = INT8 ? sc[8 * j] : a.scale_log2, vj = INT8 ? sc[kStep + 8 * j] : 0.f;
        iv[j][0] = iv[j][1] = INT8 ? sc[2 * kStep + 8 * j] : 1.f;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          x[j][h] = ((s[0][2 * j + h] + s[1][2 * j + h]) + (s[2][2 * j + h] + s[3][2 * j + h])) * kj + vj;
      }
    } else {
      // even and odd halves of d in sums of their own: half the chain of dependent MMAs
      float s[2][4], s2[2][4];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int e = 0; e < 4; ++e) s[j][e] = s2[j][e] = 0.f;
      }
      if (!INT8) {
#pragma unroll
        for (int ks = 0; ks < KS; ks += 2) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            uint32_t bfr[4];
            ldsm4(ks_s + S::at(8 * j + (lane & 7), 2 * ks + (lane >> 3)), bfr);
            mma16816(s[j], qf[ks], bfr[0], bfr[1]);
            mma16816(s2[j], qf[ks + 1], bfr[2], bfr[3]);
          }
        }
      } else {
#pragma unroll
        for (int c = 0; c < KS / 4; ++c) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 v = lds128(ks_s + S::at(8 * j + r8, 4 * c + quad));
            const uint32_t w[4] = {v.x ^ 0x80808080u, v.y ^ 0x80808080u, v.z ^ 0x80808080u, v.w ^ 0x80808080u};
#pragma unroll
            for (int e = 0; e < 4; ++e)
              mma16816(e & 1 ? s2[j] : s[j], qf[4 * c + e], codes2(w[e], 0x4140u), codes2(w[e], 0x4342u));
          }
        }
      }
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float k0s = a.scale_log2, k1s = a.scale_log2, v0 = 0.f, v1 = 0.f;
        if (INT8) {
          const float2 fk = *reinterpret_cast<const float2*>(sc + 8 * j);
          const float2 fv = *reinterpret_cast<const float2*>(sc + kStep + 8 * j);
          const float2 fi = *reinterpret_cast<const float2*>(sc + 2 * kStep + 8 * j);
          k0s = fk.x;
          k1s = fk.y;
          v0 = fv.x;
          v1 = fv.y;
          iv[j][0] = fi.x;
          iv[j][1] = fi.y;
        }
        x[j][0] = (s[j][0] + s2[j][0]) * k0s + v0;
        x[j][1] = (s[j][1] + s2[j][1]) * k1s + v1;
        x[j][2] = (s[j][2] + s2[j][2]) * k0s + v0;
        x[j][3] = (s[j][3] + s2[j][3]) * k1s + v1;
      }
    }
    // hidden keys to -inf by selection, whatever they hold
    if (key0 + kStep > open) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int e = 0; e < XE; ++e) {
          const int key = key0 + 8 * j + (NARROW ? r8 : 2 * quad + (e & 1));
          if (key >= lim[NARROW ? e : e >> 1]) x[j][e] = -INFINITY;
        }
      }
    }
    // the references are raised (and O and l rescaled) only when a weight would exceed 2^kTop
    float mx[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
      mx[h] = NARROW ? fmaxf(x[0][h], x[1][h])
                     : fmaxf(fmaxf(x[0][XE / 2 * h], x[0][XE / 2 * h + 1]), fmaxf(x[1][XE / 2 * h], x[1][XE / 2 * h + 1]));
    if (__any_sync(0xffffffffu, mx[0] - (m[0] - kPOffset) > kTop || mx[1] - (m[1] - kPOffset) > kTop)) {
      float scale[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        for (int w = NARROW ? 4 : 1; w < (NARROW ? 32 : 4); w *= 2) mx[h] = fmaxf(mx[h], __shfl_xor_sync(0xffffffffu, mx[h], w));
        const float mn = fmaxf(m[h], mx[h]);
        scale[h] = ex2_approx((m[h] - kPOffset) - (mn == -INFINITY ? 0.f : mn - kPOffset));      // as the exponents take them
        m[h] = mn;
        l[h] *= scale[h];
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
#pragma unroll
        for (int e = 0; e < 4; ++e) o[n][e] *= scale[NARROW ? e & 1 : e >> 1];
      }
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float use = (m[h] == -INFINITY ? 0.f : m[h]) - kPOffset;
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
#pragma unroll
        for (int e = 0; e < XE / 2; ++e) {
          const float pr = ex2_approx(x[j][XE / 2 * h + e] - use);
          x[j][XE / 2 * h + e] = pr;
          sum += INT8 ? pr * iv[j][e] : pr;
        }
      }
      l[h] += sum;
    }
    // P as an operand: rows and keys as the scores have them; NARROW: keys 2 quad .. against row r8, so transposed
    uint32_t pf[4];
    if constexpr (NARROW) {
      pf[0] = transpose8(pack_half2(x[0][0], x[0][1]));
      pf[1] = transpose8(pack_half2(x[1][0], x[1][1]));
    } else {
      pf[0] = pack_half2(x[0][0], x[0][1]);
      pf[1] = pack_half2(x[0][XE - 2], x[0][XE - 1]);
      pf[2] = pack_half2(x[1][0], x[1][1]);
      pf[3] = pack_half2(x[1][XE - 2], x[1][XE - 1]);
    }
    if (!INT8) {
      if constexpr (NARROW) {
        // V^T is the A operand: dimensions 16 n + r8 and 8 more, keys 2 quad .. and 8 more
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          uint32_t afr[4];
          ldsm4t(vs_s + S::at((lane >> 4) * 8 + (lane & 7), 2 * n + ((lane >> 3) & 1)), afr);
          mma16816(o[n], afr, pf[0], pf[1]);
        }
      } else {
#pragma unroll
        for (int n = 0; n < NT; n += 2) {
          uint32_t bfr[4];
          ldsm4t(vs_s + S::at(((lane >> 3) & 1) * 8 + (lane & 7), n + (lane >> 4)), bfr);
          mma16816(o[n], pf, bfr[0], bfr[1]);
          mma16816(o[n + 1], pf, bfr[2], bfr[3]);
        }
      }
    } else {
      // keys 2 quad, 2 quad + 1, 2 quad + 8, 2 quad + 9 of the 16; this lane's index r8 stands for dimensions
      // r8 * (D / 8) + n: of n-tile n, or (NARROW) of rows r8 and r8 + 8 of tile n / 2 by turns
      uint32_t w[4][D / 32];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int row = 2 * quad + (e & 1) + 8 * (e >> 1);
        if (D == 128) {
          const uint4 v = lds128(vs_s + S::at(row, r8));
          w[e][0] = v.x ^ 0x80808080u;
          w[e][1] = v.y ^ 0x80808080u;
          w[e][D / 32 - 2] = v.z ^ 0x80808080u;
          w[e][D / 32 - 1] = v.w ^ 0x80808080u;
        } else {
          const uint2 v = lds64(vs_s + S::at(row, r8 >> 1) + (r8 & 1) * 8);
          w[e][0] = v.x ^ 0x80808080u;
          w[e][1] = v.y ^ 0x80808080u;
        }
      }
#pragma unroll
      for (int q = 0; q < D / 32; ++q) {
#pragma unroll
        for (int hlf = 0; hlf < 2; ++hlf) {
          const uint32_t lo = __byte_perm(w[0][q], w[1][q], hlf ? 0x7362u : 0x5140u);
          const uint32_t hi = __byte_perm(w[2][q], w[3][q], hlf ? 0x7362u : 0x5140u);
          const uint32_t v[4] = {codes2(lo, 0x4140u), codes2(lo, 0x4342u), codes2(hi, 0x4140u), codes2(hi, 0x4342u)};
          if constexpr (NARROW) {
            mma16816(o[2 * q + hlf], v, pf[0], pf[1]);
          } else {
            mma16816(o[4 * q + 2 * hlf], pf, v[0], v[2]);
            mma16816(o[4 * q + 2 * hlf + 1], pf, v[1], v[3]);
          }
        }
      }
    }
    if (i + 2 < steps) keep_scales(freed, sc_a);      // the loads have had this step's time
  }
  cp_wait<0>();
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    // a row that saw keys, all of them at -inf (its query is not finite): 0 / 0, not a row that saw nothing
    if (lim[h] > first && m[h] == -INFINITY) l[h] = NAN;
    for (int w = NARROW ? 4 : 1; w < (NARROW ? 32 : 4); w *= 2) l[h] += __shfl_xor_sync(0xffffffffu, l[h], w);
  }

  // ---- join the four warps, in fragment order: register e of n-tile n of lane
  const bool writer = NARROW ? r8 == 0 : quad == 0;      // of its rows' m and l
  if (writer) {
    ml_s[warp * 16 + row_of(0)] = make_float2(m[0] - kPOffset, l[0]);
    ml_s[warp * 16 + row_of(1)] = make_float2(m[1] - kPOffset, l[1]);
  }
  __syncwarp();
  static_assert(NT * 32 * 16 <= kStages * 2 * S::BYTES, "a warp's O fits its ring");
  float* os = reinterpret_cast<float*>(ring);    // this warp's ring, no longer read
#pragma unroll
  for (int n = 0; n < NT; ++n)
    *reinterpret_cast<float4*>(os + (n * 32 + lane) * 4) = make_float4(o[n][0], o[n][1], o[n][2], o[n][3]);
  __syncthreads();
  float wgt[2][kWarps], M[2], L[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    M[h] = -INFINITY;
    L[h] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M[h] = fmaxf(M[h], ml_s[w * 16 + row_of(h)].x);
    const float use = M[h] == -INFINITY ? 0.f : M[h];
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 f = ml_s[w * 16 + row_of(h)];
      wgt[h][w] = ex2_approx(f.x - use);
      L[h] += wgt[h][w] * f.y;
    }
    if (direct) {
      const float inv = L[h] > 0.f ? 1.f / L[h] : (L[h] == 0.f ? 0.f : L[h]);
#pragma unroll
      for (int w = 0; w < kWarps; ++w) wgt[h][w] *= inv;
    }
  }
  constexpr int NW = NT / kWarps;    // n-tiles per warp
  float acc[NW][4];
#pragma unroll
  for (int n = 0; n < NW; ++n) {
    acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float* src = reinterpret_cast<const float*>(smem + w * kStages * 2 * S::BYTES);
      const float4 f = *reinterpret_cast<const float4*>(src + ((warp * NW + n) * 32 + lane) * 4);
      acc[n][0] += wgt[0][w] * f.x;
      acc[n][1] += wgt[NARROW ? 1 : 0][w] * f.y;
      acc[n][2] += wgt[NARROW ? 0 : 1][w] * f.z;
      acc[n][3] += wgt[1][w] * f.w;
    }
  }
  const int64_t used = direct ? rows_in_use(a) : 0, unused = direct ? first_row(a) : 0;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int r = row_of(h);
    if (r >= rows) continue;
    const int64_t t = token_of(r);
    const int64_t idx = slot * total + t * Hq + head_of(r);
    if (!direct && warp == 0 && writer) a.ml[idx] = make_float2(M[h], L[h]);
    if (direct && (t >= used || t < unused)) continue;
    __half* oh = direct ? a.out + t * a.o_t + head_of(r) * a.o_h : nullptr;
    float* of = direct ? nullptr : a.o + idx * D;
    if (NARROW && INT8) {
      // tiles warp * NW ..: 2 NW consecutive dimensions
#pragma unroll
      for (int n = 0; n < NW; ++n) {
        const int at = r8 * (D / 8) + 2 * (warp * NW + n);
        if (direct)
          *reinterpret_cast<uint32_t*>(oh + at) = pack_half2(acc[n][h], acc[n][2 + h]);
        else
          *reinterpret_cast<float2*>(of + at) = make_float2(acc[n][h], acc[n][2 + h]);
      }
    } else if (NARROW) {
#pragma unroll
      for (int n = 0; n < NW; ++n) {
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int at = (warp * NW + n) * 16 + 8 * e + r8;
          if (direct)
            oh[at] = __float2half_rn(acc[n][2 * e + h]);
          else
            of[at] = acc[n][2 * e + h];
        }
      }
    } else if (INT8) {
      // n-tiles warp * NW ..: consecutive dimensions for each of the lane's two columns
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        const int at = (2 * quad + e) * (D / 8) + warp * NW;
#pragma unroll
        for (int n = 0; n < NW; n += 2) {
          if (direct)
            *reinterpret_cast<uint32_t*>(oh + at + n) = pack_half2(acc[n][2 * h + e], acc[n + 1 < NW ? n + 1 : n][2 * h + e]);
          else
            *reinterpret_cast<float2*>(of + at + n) = make_float2(acc[n][2 * h + e], acc[n + 1 < NW ? n + 1 : n][2 * h + e]);
        }
      }
    } else {
#pragma unroll
      for (int n = 0; n < NW; ++n) {
        const int at = (warp * NW + n) * 8 + 2 * quad;
        if (direct)
          *reinterpret_cast<uint32_t*>(oh + at) = pack_half2(acc[n][2 * h], acc[n][2 * h + 1]);
        else
          *reinterpret_cast<float2*>(of + at) = make_float2(acc[n][2 * h], acc[n][2 * h + 1]);
      }
    }
  }
}

template <int D, bool INT8, bool NARROW>
__global__ void __launch_bounds__(kWarps * 32, split_resident(D, INT8, NARROW))
    split_kernel(const __grid_constant__ SharedArgs a, const __grid_constant__ PageMaps maps, DevErr err) {
  pdl_launch_dependents();
  split_rows<D, INT8, NARROW>(a, maps, err);
  pdl_wait();      // whoever waits for this kernel has waited for the one before it
}

// Results of one row (token t, query head h): prefix results lie in slots 0 ..
// pre - 1, the pieces of the line that the row block's key tiles lie in.
__device__ __forceinline__ int prefix_results(const SharedPlan& p, int t, int h) {
  if (!p.pre_tile || p.pre_pieces > 0) return p.pre_splits;
  const int kvh = h / p.group;
  const int packed = t * p.group + h - kvh * p.group;
  const int first = (kvh * p.pre_rows + packed / 256) * p.pre_tiles;
  return (first + p.pre_tiles - 1) / p.pre_chunk - first / p.pre_chunk + 1;
}

// Joins the results of many rows: eight lanes per row, four results at a time
// (their weights first, then the O rows that carry one).  Bound by the O rows,
// 512 bytes of each result at d = 128.
template <int D>
__global__ void __launch_bounds__(256) join_rows_kernel(const __grid_constant__ SharedArgs a) {
  constexpr int V = D / 32;      // 16-byte pieces of a lane
  const SharedPlan& p = a.plan;
  const int Hq = a.pool.H * p.group;
  const int64_t total = a.T * Hq;
  const int row = static_cast<int>(blockIdx.x) * 32 + (threadIdx.x >> 3);
  const int lane = threadIdx.x & 7;
  const int t = row / Hq, h = row - t * Hq;
  const bool live_row = row < total && t < rows_in_use(a) && t >= first_row(a);
  const int pre = prefix_results(p, t, h);
  const int count = live_row ? pre + p.own_splits : 0;
  const int own_at = p.pre_splits - pre;      // result i lies in slot i, or i + own_at from `pre` on
  pdl_wait();
  float M = -INFINITY, L = 0.f;
  float4 acc[V];
#pragma unroll
  for (int v = 0; v < V; ++v) acc[v] = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int i0 = 0; i0 < count; i0 += 4) {
    float2 ml[4];
    float4 f[4][V];
    float mx = M;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k;
      ml[k] = make_float2(-INFINITY, 0.f);
      if (i < count) ml[k] = a.ml[(i + (i < pre ? 0 : own_at)) * total + row];
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int i = i0 + k;
      mx = fmaxf(mx, ml[k].x);
#pragma unroll
      for (int v = 0; v < V; ++v) f[k][v] = make_float4(0.f, 0.f, 0.f, 0.f);
      if (ml[k].y != 0.f) {      // NaN counts
        const float4* src = reinterpret_cast<const float4*>(a.o + ((i + (i < pre ? 0 : own_at)) * total + row) * D) + lane;
#pragma unroll
        for (int v = 0; v < V; ++v) f[k][v] = __ldcs(src + 8 * v);
      }
    }
    const float use = mx == -INFINITY ? 0.f : mx;
    const float keep = ex2_approx(M - use);
    M = mx;
    L *= keep;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      acc[v].x *= keep;
      acc[v].y *= keep;
      acc[v].z *= keep;
      acc[v].w *= keep;
    }
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float w = ml[k].y == 0.f ? 0.f : ex2_approx(ml[k].x - use);
      L += w * ml[k].y;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        acc[v].x += w * f[k][v].x;
        acc[v].y += w * f[k][v].y;
        acc[v].z += w * f[k][v].z;
        acc[v].w += w * f[k][v].w;
      }
    }
  }
  if (!live_row) return;
  const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
  __half* dst = a.out + t * a.o_t + h * a.o_h + lane * 4;
#pragma unroll
  for (int v = 0; v < V; ++v)
    *reinterpret_cast<uint2*>(dst + 32 * v) = make_uint2(pack_half2(acc[v].x * inv, acc[v].y * inv),
                                                         pack_half2(acc[v].z * inv, acc[v].w * inv));
}

// Joins a row's results: W warps per (token, query head).  Every warp weighs
// all slots (one or two per lane); warp w adds the O rows of slots w, w + W, ..,
// eight loads in flight, and the warps' sums meet in shared memory.  Moves
// count * d * 4 bytes a row, mostly out of L2; with few rows it is bound by
// latency: W is as large as leaves one wave of blocks.
template <int D, int W>
__global__ void __launch_bounds__(256, 4) join_kernel(const __grid_constant__ SharedArgs a) {
  constexpr int V = D / 32;
  __shared__ float sums[8][D];
  const int Hq = a.pool.H * a.plan.group;
  const int64_t total = a.T * Hq;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * (8 / W) + warp / W;
  const int part = warp % W;
  const int t = static_cast<int>(static_cast<uint32_t>(row) / static_cast<uint32_t>(Hq));     // rows stay below 2^30
  const bool live_row = row < total && t < rows_in_use(a) && t >= first_row(a);
  const SharedPlan& p = a.plan;
  const int pre = prefix_results(p, t, static_cast<int>(row) - t * Hq);
  const int count = live_row ? pre + p.own_splits : 0;
  const int own_at = p.pre_splits - pre;      // result i lies in slot i, or i + own_at from `pre` on
  pdl_wait();
  float m[2], wgt[2], M = -INFINITY, L = 0.f;
  static_assert(2 * (kMostSplits + 2) <= 64, "two slots per lane");
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = lane + 32 * k;
    float2 ml = make_float2(-INFINITY, 0.f);
    if (i < count) ml = a.ml[(i + (i < pre ? 0 : own_at)) * total + row];
    m[k] = ml.x;
    wgt[k] = ml.y;
    M = fmaxf(M, ml.x);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xffffffffu, M, o));
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const float l = wgt[k];
    wgt[k] = l == 0.f ? 0.f : ex2_approx(m[k] - (M == -INFINITY ? 0.f : M));
    L += wgt[k] * l;
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) L += __shfl_xor_sync(0xffffffffu, L, o);
  float acc[V] = {};
  constexpr int U = 8;
  for (int i0 = part; i0 < count; i0 += U * W) {
    float w[U], f[U][V];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = i0 + k * W;
      w[k] = __shfl_sync(0xffffffffu, i < 32 ? wgt[0] : wgt[1], i & 31);
      if (i >= count) w[k] = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) f[k][v] = 0.f;
      if (w[k] != 0.f) {      // NaN counts
        const float* src = a.o + ((i + (i < pre ? 0 : own_at)) * total + row) * D + lane * V;
        if (V == 4) {
          const float4 q = __ldcs(reinterpret_cast<const float4*>(src));
          f[k][0] = q.x;
          f[k][1] = q.y;
          f[k][V - 2] = q.z;
          f[k][V - 1] = q.w;
        } else {
          const float2 q = __ldcs(reinterpret_cast<const float2*>(src));
          f[k][0] = q.x;
          f[k][1] = q.y;
        }
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
#pragma unroll
      for (int v = 0; v < V; ++v) acc[v] += w[k] * f[k][v];
    }
  }
#pragma unroll
  for (int v = 0; v < V; ++v) sums[warp][lane * V + v] = acc[v];
  __syncthreads();
  if (part != 0) return;
#pragma unroll
  for (int w = 1; w < W; ++w) {
#pragma unroll
    for (int v = 0; v < V; ++v) acc[v] += sums[warp + w][lane * V + v];
  }
  if (!live_row) return;
  const float inv = L > 0.f ? 1.f / L : (L == 0.f ? 0.f : L);
  __half* dst = a.out + t * a.o_t + (static_cast<int>(row) - t * Hq) * a.o_h + lane * V;
  if (V == 4)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_half2(acc[0] * inv, acc[1] * inv),
                                                pack_half2(acc[V - 2] * inv, acc[V - 1] * inv));
  else
    *reinterpret_cast<uint32_t*>(dst) = pack_half2(acc[0] * inv, acc[1] * inv);
}

// Without room for own tokens (max_kv = 0) only the prefix's kernel runs; this one makes the tests that theirs would.
__global__ void __launch_bounds__(256) check_kernel(const __grid_constant__ SharedArgs a, DevErr err) {
  const int64_t b = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (b < a.batch) {
    int64_t start, n;
    seq_rows(a, static_cast<int>(b), start, n);
    if (rows_outside(a, start, n, a.plan.own_tile ? 256 : split_block(a.plan.narrow)) ||
        (n > 0 && __ldg(a.kv_lens + b) > a.max_kv))
      dev_error(err, TM_DEVERR_SEQLEN);
  }
  pdl_launch_dependents();
  pdl_wait();
}

template <int D, bool INT8, bool NARROW>
tm_status launch_split(const SharedArgs& a, bool overlap, DevErr err, cudaStream_t stream) {
  constexpr int smem = SplitSmem<D, INT8>::BYTES;
  static std::atomic<uint64_t> prepared{0};
  const tm_status st = prepare_smem(split_kernel<D, INT8, NARROW>, smem, prepared);
  if (st != TM_OK) return st;
  const SharedPlan& p = a.plan;
  const int64_t items = ((p.pre_tile ? 0 : static_cast<int64_t>(p.pre_splits) * p.pre_rows) +
                         (p.own_tile ? 0 : static_cast<int64_t>(p.own_splits) * a.batch * p.own_rows)) * a.pool.H;
  return launch_kernel(split_kernel<D, INT8, NARROW>, items, kWarps * 32, smem, overlap, stream, a,
                       page_maps(a.pool, D, INT8, kStep), err);
}

// Up to three kernels, each allowed to start while the one before it drains:
// none but the join reads what another writes, and the join waits for all.
tm_status launch(const SharedArgs& a, int d, bool int8, DevErr err, cudaStream_t stream) {
  const SharedPlan& p = a.plan;
  bool after = false;
  tm_status st = TM_OK;
  if (p.own_splits == 0) {
    st = launch_kernel(check_kernel, ceil_div(a.batch, 256), 256, 0, after, stream, a, err);
    after = true;
  }
  if (st == TM_OK && p.pre_tile) {
    st = shared_tile(a, d, int8, true, after, err, stream);
    after = true;
  }
  if (st == TM_OK && p.own_tile && p.own_splits > 0) {
    st = shared_tile(a, d, int8, false, after, err, stream);
    after = true;
  }
  if (st == TM_OK && ((!p.pre_tile && p.pre_splits > 0) || (!p.own_tile && p.own_splits > 0))) {
    auto split = p.narrow ? (d == 128 ? (int8 ? launch_split<128, true, true> : launch_split<128, false, true>)
                                      : (int8 ? launch_split<64, true, true> : launch_split<64, false, true>))
                          : (d == 128 ? (int8 ? launch_split<128, true, false> : launch_split<128, false, false>)
                                      : (int8 ? launch_split<64, true, false> : launch_split<64, false, false>));
    st = split(a, after, err, stream);
    after = true;
  }
  if (st != TM_OK || p.slots == 1) return st;
  const int64_t rows = a.T * a.pool.H * p.group;
  if (rows >= 8192 || p.slots <= 2)
    return launch_kernel(d == 128 ? join_rows_kernel<128> : join_rows_kernel<64>, ceil_div(rows, 32), 256, 0, after, stream, a);
  constexpr int64_t kResident = 4 * kSmsB200;       // blocks of 256 threads at 64 registers
  const int W = rows <= kResident ? 8 : (rows <= 2 * kResident ? 4 : (rows <= 4 * kResident ? 2 : 1));
  auto join = d == 128 ? (W == 8 ? join_kernel<128, 8> : W == 4 ? join_kernel<128, 4> : W == 2 ? join_kernel<128, 2> : join_kernel<128, 1>)
                       : (W == 8 ? join_kernel<64, 8> : W == 4 ? join_kernel<64, 4> : W == 2 ? join_kernel<64, 2> : join_kernel<64, 1>);
  return launch_kernel(join, ceil_div(rows, 8 / W), 256, 0, after, stream, a);
}

bool plan_args_ok(int64_t T, int32_t Hq, int32_t Hkv, int32_t batch, int64_t max_seqlen, int64_t prefix_len,
                  int64_t max_kv_len) {
  return T >= 0 && Hq > 0 && Hkv > 0 && Hq % Hkv == 0 && batch > 0 && max_seqlen >= 0 && prefix_len >= 0 &&
         max_kv_len >= 0 && prefix_len <= (1ll << 30) && max_kv_len <= (1ll << 30) && T <= (1ll << 24) &&
         static_cast<int64_t>(Hq) * T <= (1ll << 30) && Hq <= 65536;
}

}  // namespace
}  // namespace tmk

extern "C" int64_t tm_attn_shared_prefix_workspace(int64_t T, int32_t Hq, int32_t Hkv, int32_t d, int32_t batch,
                                                   int32_t max_seqlen, int64_t prefix_len, int64_t max_kv_len) {
  if (!tmk::plan_args_ok(T, Hq, Hkv, batch, max_seqlen, prefix_len, max_kv_len) || (d != 64 && d != 128)) return -1;
  // for pages of either type
  const int64_t f16 = tmk::shared_plan(T, Hq, Hkv, d, false, batch, max_seqlen, prefix_len, max_kv_len).bytes;
  const int64_t i8 = tmk::shared_plan(T, Hq, Hkv, d, true, batch, max_seqlen, prefix_len, max_kv_len).bytes;
  return f16 < 0 || i8 < 0 ? -1 : (f16 > i8 ? f16 : i8);
}

extern "C" tm_status tm_attn_shared_prefix(const tm_tensor* q, const tm_paged_kv* cache, tm_tensor* out,
                                           const int32_t* table, int64_t table_stride, int32_t table_cols,
                                           const int32_t* kv_lens, const int32_t* cu_seqlens, int32_t batch,
                                           int32_t max_seqlen, const int32_t* prefix_pages, int64_t prefix_len,
                                           int64_t max_kv_len, int32_t causal, void* workspace,
                                           int64_t workspace_bytes, void* stream) {
  using namespace tmk;
  SharedArgs a{};
  bool int8 = false;
  tm_status st = paged_pool(cache, &a.pool, &int8);
  if (st != TM_OK) return st;
  st = page_table(a.pool, table, table_stride, table_cols, &a.pt);
  if (st != TM_OK) return st;
  if (q == nullptr || out == nullptr || kv_lens == nullptr || batch <= 0) return TM_ERR_INVALID_ARG;
  const int64_t T = q->T, d = cache->d;
  if (T < 0 || !thd_ok(q, T, q->H, d) || !thd_out_ok(out, T, q->H, d)) return TM_ERR_INVALID_ARG;
  if (cu_seqlens == nullptr) {
    if (T % batch != 0) return TM_ERR_INVALID_ARG;
    if (T / batch > 0x7fffffff) return TM_ERR_UNSUPPORTED;
    max_seqlen = static_cast<int32_t>(T / batch);
  }
  if (q->H > 65536 || !plan_args_ok(T, static_cast<int32_t>(q->H), cache->H, batch, max_seqlen, prefix_len, max_kv_len))
    return TM_ERR_INVALID_ARG;
  if (prefix_len > 0 && prefix_pages == nullptr) return TM_ERR_INVALID_ARG;
  if (max_kv_len > static_cast<int64_t>(table_cols) * cache->page_size) return TM_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(kv_lens) | reinterpret_cast<uintptr_t>(cu_seqlens) |
       reinterpret_cast<uintptr_t>(prefix_pages)) & 3u)
    return TM_ERR_INVALID_ARG;
  a.plan = shared_plan(T, static_cast<int32_t>(q->H), cache->H, cache->d, int8, batch, max_seqlen, prefix_len, max_kv_len);
  if (a.plan.bytes < 0) return TM_ERR_UNSUPPORTED;
  if (workspace == nullptr || (reinterpret_cast<uintptr_t>(workspace) & 255u) || workspace_bytes < a.plan.bytes)
    return TM_ERR_INVALID_ARG;
  if (T == 0) return TM_OK;
  a.q = static_cast<const __half*>(q->data);
  a.q_t = q->stride_t;
  a.q_h = q->stride_h;
  a.out = static_cast<__half*>(out->data);
  a.o_t = out->stride_t;
  a.o_h = out->stride_h;
  a.kv_lens = kv_lens;
  a.cu = cu_seqlens;
  a.prefix_pages = prefix_pages;
  a.T = T;
  a.per_seq = T / batch;
  a.prefix_len = prefix_len;
  a.max_kv = max_kv_len;
  a.batch = batch;
  a.causal = causal != 0;
  a.ml = static_cast<float2*>(workspace);
  a.o = reinterpret_cast<float*>(static_cast<uint8_t*>(workspace) + a.plan.ml_bytes);
  a.scale_log2 = static_cast<float>(1.4426950408889634 / sqrt(static_cast<double>(d)));
  const DevErr err{device_error_word()};
  if (err.word == nullptr) return cuda_fail(static_cast<int>(cudaErrorInvalidSymbol));
  cudaStream_t s = as_stream(stream);
  return launch(a, static_cast<int>(d), int8, err, s);
}
