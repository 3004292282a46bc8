// tm_rope.cu -- rotary positions, norms of queries and keys, and appending
// rotated keys and values to a paged cache: one kernel over the rows of the
// new tokens.
//
// For each (token, head) row x of d values:
//   n = x / sqrt(mean(x^2) + eps) * w               (norm, optional)
//   y_a = m (n_a cos - n_b sin), y_b = m (n_a sin + n_b cos) with the pair's
//   angle p f_i                                     (rotation, optional)
// in fp32 from the fp16 input to one rounding (or one quantisation) at the end.
// Every byte is read once and written once, so long prompts are bound by HBM
// and single steps by latency.
//
// Angles: a frequency is a 64-bit binary fraction F of a turn per position, so
// p * F mod 2^64 is the angle as a fraction of a turn without range reduction
// and without loss at far positions; its top 32 bits, as a signed number of
// half turns, go to sincospif.  A warp computes the (up to 64) sines and
// cosines of its token once, two per lane, into its own 512 bytes of shared
// memory, and uses them for all the heads it handles.
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <math.h>

#include "tm_device.cuh"
#include "tm_host.h"
#include "tm_paged.cuh"

namespace tmk {
namespace {

constexpr int kTokenWarps = 4;
constexpr int kSms = 148;

struct Rows {
  const __half* in;
  __half* out;
  int64_t in_t, in_h, out_t, out_h;
  const __half* weight;   // norm weight or null
};

struct TokenArgs {
  Rows q, k, v;                       // v: append only
  int hq, hk, hv;                     // heads of each (0: none)
  int64_t T;
  int parts;                          // warps per token
  float eps;
  int rope, interleaved, rot;
  float mscale;
  const int32_t* positions;           // rope / norm
  int64_t pos_offset;
  const int32_t* kv_lens;             // append
  const int32_t* cu;
  int batch;
  int64_t per_seq;                    // rows per sequence when cu is null
  PagedPool pool;
  PageTable pt;
  uint64_t turns[64];
};

__device__ __forceinline__ void unpack8(uint4 v, float (&x)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
    x[2 * i] = f.x;
    x[2 * i + 1] = f.y;
  }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
  return make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
}

enum { kNoCache = 0, kCacheF16 = 1, kCacheI8 = 2 };

// A warp takes one token and every `parts`-th group of 32 / (D / 8) heads; a
// lane holds 8 consecutive values of a head (one 16-byte load).  U groups are
// loaded before the first is used, to keep several loads in flight.
template <int D, int CACHE>
__global__ void __launch_bounds__(kTokenWarps * 32) token_kernel(const __grid_constant__ TokenArgs a, DevErr err) {
  constexpr int LPR = D / 8;          // lanes of a row
  constexpr int RPW = 32 / LPR;       // rows of a warp
  constexpr int U = 4;
  __shared__ __align__(16) float2 trig[kTokenWarps][64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t job = static_cast<int64_t>(blockIdx.x) * kTokenWarps + warp;
  const int64_t t = job / a.parts;
  const int part = static_cast<int>(job - t * a.parts);
  if (t >= a.T) return;

  int64_t pos;
  int64_t slot_row = -1, slot_scale = 0;   // where the token's K and V go (CACHE)
  if (CACHE == kNoCache) {
    pos = (a.positions != nullptr ? static_cast<int64_t>(__ldg(a.positions + t)) : t) + a.pos_offset;
  } else {
    int b;
    int64_t i, n;
    if (a.cu != nullptr) {
      b = sequence_of(a.cu, a.batch, t);
      if (b >= a.batch) return;            // behind the last sequence
      const int32_t s = __ldg(a.cu + b);
      n = __ldg(a.cu + b + 1) - s;
      i = t - s;
    } else {
      b = static_cast<int>(t / a.per_seq);
      n = a.per_seq;
      i = t - b * n;
    }
    const int64_t j = __ldg(a.kv_lens + b) - n + i;
    pos = j + a.pos_offset;
    if (j >= 0) {
      const int32_t page = page_of(a.pt, b, j);
      if (page < 0) {
        if (lane == 0) dev_error(err, TM_DEVERR_SEQLEN);
      } else {
        const int64_t s = j & ((1 << a.pt.page_shift) - 1);
        slot_row = page * a.pool.stride_page + s * a.pool.stride_t;
        slot_scale = page * a.pool.sstride_page + s * a.pool.sstride_t;
      }
    }
  }

  const int half_rot = a.rot >> 1;
  if (a.rope) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = lane + 32 * r;
      if (i < half_rot) {
        const uint64_t turn = static_cast<uint64_t>(pos) * a.turns[i];
        const int32_t top = static_cast<int32_t>(static_cast<uint32_t>(turn >> 32));
        float sn, cs;
        sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &sn, &cs);   // 2^-31: half turns
        trig[warp][i] = make_float2(cs * a.mscale, sn * a.mscale);
      }
    }
    __syncwarp();
  }

  // this lane's place in a row and its eight (cos, sin): in the half layout
  // its values are the first or second members of pairs i0 .. i0 + 7, and the
  // partner values sit `half_rot` away, half_rot / 8 lanes off; in the
  // interleaved one it holds the whole pairs i0 .. i0 + 3.
  const int l = lane & (LPR - 1);
  const int sub = lane / LPR;
  const int rot_lanes = a.rot >> 3, half_lanes = a.rot >> 4;
  const bool turned = a.rope && l < rot_lanes;
  const bool second = !a.interleaved && l >= half_lanes;
  const int partner = a.interleaved ? lane : (turned ? (second ? lane - half_lanes : lane + half_lanes) : lane);
  float cs[8], sn[8];
  if (turned) {
    if (a.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 f = trig[warp][4 * l + e];
        cs[e] = f.x;
        sn[e] = f.y;
      }
    } else {
      const int i0 = 8 * (second ? l - half_lanes : l);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float2 f = trig[warp][i0 + e];
        cs[e] = f.x;
        sn[e] = second ? f.y : -f.y;
      }
    }
  }

  const int heads = a.hq + a.hk + a.hv;
  const int groups = (heads + RPW - 1) / RPW;
  for (int g0 = part; g0 < groups; g0 += a.parts * U) {
    uint4 raw[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = (g0 + u * a.parts) * RPW + sub;
      raw[u] = make_uint4(0, 0, 0, 0);
      if (h < heads) {
        const bool isq = h < a.hq, isk = h < a.hq + a.hk;
        const Rows& r = isq ? a.q : (isk ? a.k : a.v);
        const int hh = isq ? h : (isk ? h - a.hq : h - a.hq - a.hk);
        raw[u] = *(reinterpret_cast<const uint4*>(r.in + t * r.in_t + hh * r.in_h) + l);   // in place: not ld.nc
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int g = g0 + u * a.parts;
      if (g >= groups) break;              // the same for the whole warp
      const int h = g * RPW + sub;
      const bool isq = h < a.hq, isk = !isq && h < a.hq + a.hk;
      const bool isv = !isq && !isk;
      const int hh = isq ? h : (isk ? h - a.hq : h - a.hq - a.hk);
      const __half* w = isq ? a.q.weight : (isk ? a.k.weight : nullptr);
      float x[8];
      unpack8(raw[u], x);
      // the norm's sum runs over the row's lanes; all lanes take part in the
      // shuffles whatever their row
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) ss += x[e] * x[e];
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
      if (w != nullptr) {
        const float inv = 1.0f / sqrtf(ss * (1.0f / D) + a.eps);
        float wf[8];
        unpack8(__ldg(reinterpret_cast<const uint4*>(w) + l), wf);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = x[e] * inv * wf[e];
      }
      if (a.rope) {
        if (a.interleaved) {
          if (turned && !isv) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float p = x[2 * e], q = x[2 * e + 1];
              x[2 * e] = p * cs[e] - q * sn[e];
              x[2 * e + 1] = p * sn[e] + q * cs[e];
            }
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float y = __shfl_sync(0xffffffffu, x[e], partner);
            if (turned && !isv) x[e] = x[e] * cs[e] + y * sn[e];
          }
        }
      }
      if (CACHE == kCacheI8) {
        // absmax as integer bits: a NaN compares above everything and so
        // reaches the scale
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) m = max(m, __float_as_uint(x[e]) & 0x7fffffffu);
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (!isq && h < heads && slot_row >= 0) {
          const __half s16 = __float2half_rn(__fdiv_rn(__uint_as_float(m), 127.0f));
          const float s = __half2float(s16);
          uint32_t c[2] = {0, 0};
          if (s != 0.f) {
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              int v = __float2int_rn(__fdiv_rn(x[e], s));
              v = max(-127, min(127, v));
              c[e >> 2] |= static_cast<uint32_t>(v & 255) << (8 * (e & 3));
            }
          }
          uint8_t* base = isk ? a.pool.k : a.pool.v;
          *reinterpret_cast<uint2*>(base + slot_row + hh * a.pool.stride_h + 8 * l) = make_uint2(c[0], c[1]);
          if (l == 0) (isk ? a.pool.ks : a.pool.vs)[slot_scale + hh * a.pool.sstride_h] = s16;
        }
      }
      if (h >= heads) continue;
      if (CACHE == kNoCache || isq) {
        const Rows& r = isq ? a.q : a.k;
        *(reinterpret_cast<uint4*>(r.out + t * r.out_t + hh * r.out_h) + l) = pack8(x);
      } else if (CACHE == kCacheF16 && slot_row >= 0) {
        uint8_t* base = isk ? a.pool.k : a.pool.v;
        *reinterpret_cast<uint4*>(base + slot_row + hh * a.pool.stride_h + 16 * l) = pack8(x);
      }
    }
  }
}

// Warps per token: enough of them for every SM to hold about 32 while a token
// has heads to share out, else at least eight groups of heads each, so that
// the token's sines and cosines are computed few times.
int token_parts(int64_t T, int groups) {
  const int64_t want = (static_cast<int64_t>(kSms) * 32 + T - 1) / T;
  const int64_t least = (groups + 7) / 8;
  int64_t p = want > least ? want : least;
  return static_cast<int>(p < groups ? p : groups);
}

Rows rows_of(const tm_tensor* in, const tm_tensor* out, const void* w) {
  Rows r{};
  if (in != nullptr) {
    r.in = static_cast<const __half*>(in->data);
    r.in_t = in->stride_t;
    r.in_h = in->stride_h;
  }
  if (out != nullptr) {
    r.out = static_cast<__half*>(out->data);
    r.out_t = out->stride_t;
    r.out_h = out->stride_h;
  }
  r.weight = static_cast<const __half*>(w);
  return r;
}

bool rope_ok(const tm_rope_freqs* r, int64_t d) {
  return r->d == d && r->rot_dim >= 16 && r->rot_dim <= d && r->rot_dim % 16 == 0;
}

void set_rope(TokenArgs* a, const tm_rope_freqs* r) {
  if (r == nullptr) return;
  a->rope = 1;
  a->interleaved = r->interleaved != 0;
  a->rot = r->rot_dim;
  a->mscale = r->mscale;
  for (int i = 0; i < 64; ++i) a->turns[i] = r->turns[i];
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

tm_status launch_tokens(TokenArgs& a, int d, int cache, cudaStream_t stream) {
  const int rpw = 256 / d;
  const int groups = (a.hq + a.hk + a.hv + rpw - 1) / rpw;
  a.parts = token_parts(a.T, groups);
  const int64_t blocks = (a.T * a.parts + kTokenWarps - 1) / kTokenWarps;
  if (blocks > 0x7fffffff) return TM_ERR_UNSUPPORTED;
  const DevErr err{device_error_word()};
  if (err.word == nullptr) return cuda_fail(static_cast<int>(cudaErrorInvalidSymbol));
  auto kernel = cache == kCacheI8 ? (d == 128 ? token_kernel<128, kCacheI8> : token_kernel<64, kCacheI8>)
                : cache == kCacheF16 ? (d == 128 ? token_kernel<128, kCacheF16> : token_kernel<64, kCacheF16>)
                                     : (d == 128 ? token_kernel<128, kNoCache> : token_kernel<64, kNoCache>);
  kernel<<<static_cast<unsigned>(blocks), kTokenWarps * 32, 0, stream>>>(a, err);
  return check_cuda(cudaGetLastError());
}

// tm_rope and tm_qk_norm_rope: the checks they share, and the launch.
tm_status rope_rows(const tm_tensor* q, const tm_tensor* k, tm_tensor* q_out, tm_tensor* k_out, const void* q_weight,
                    const void* k_weight, float eps, const tm_rope_freqs* rope, const int32_t* positions,
                    int64_t pos_offset, void* stream) {
  if (q == nullptr || (k == nullptr) != (k_out == nullptr)) return TM_ERR_INVALID_ARG;
  const int64_t T = q->T, d = q->d;
  if (T < 0 || !thd_ok(q, T, q->H, d) || !thd_out_ok(q_out, T, q->H, d)) return TM_ERR_INVALID_ARG;
  if (k != nullptr && (!thd_ok(k, T, k->H, d) || !thd_out_ok(k_out, T, k->H, d))) return TM_ERR_INVALID_ARG;
  if (d != 64 && d != 128) return TM_ERR_UNSUPPORTED;
  if (rope != nullptr && !rope_ok(rope, d)) return TM_ERR_INVALID_ARG;
  if (!aligned(positions, 4) || !aligned(q_weight, 16) || !aligned(k_weight, 16)) return TM_ERR_INVALID_ARG;
  if (q->H > 65536 || (k != nullptr && k->H > 65536)) return TM_ERR_UNSUPPORTED;
  if (T == 0) return TM_OK;
  TokenArgs a{};
  a.q = rows_of(q, q_out, q_weight);
  a.k = rows_of(k, k_out, k_weight);
  a.hq = static_cast<int>(q->H);
  a.hk = k != nullptr ? static_cast<int>(k->H) : 0;
  a.T = T;
  a.eps = eps;
  a.positions = positions;
  a.pos_offset = pos_offset;
  set_rope(&a, rope);
  return launch_tokens(a, static_cast<int>(d), kNoCache, as_stream(stream));
}

}  // namespace
}  // namespace tmk

extern "C" tm_status tm_rope_init(tm_rope_freqs* rope, int32_t d, int32_t rot_dim, int32_t interleaved, double theta,
                                  int32_t scaling, double factor, double original_max, double fast, double slow) {
  if (rope == nullptr || (d != 64 && d != 128) || rot_dim < 16 || rot_dim > d || rot_dim % 16) return TM_ERR_INVALID_ARG;
  if (!(theta > 1.0) || !isfinite(theta) || scaling < TM_ROPE_PLAIN || scaling > TM_ROPE_BANDS)
    return TM_ERR_INVALID_ARG;
  const bool bands = scaling == TM_ROPE_YARN || scaling == TM_ROPE_BANDS;
  if (scaling != TM_ROPE_PLAIN && (!(factor >= 1.0) || !isfinite(factor))) return TM_ERR_INVALID_ARG;
  if (bands && (!(original_max > 0.0) || !isfinite(original_max) || !(slow > 0.0) || !(fast > slow) || !isfinite(fast)))
    return TM_ERR_INVALID_ARG;
  const double two_pi = 6.283185307179586476925;
  rope->d = d;
  rope->rot_dim = rot_dim;
  rope->interleaved = interleaved != 0;
  rope->mscale = scaling == TM_ROPE_YARN ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.0f;
  if (scaling == TM_ROPE_NTK) theta *= pow(factor, static_cast<double>(rot_dim) / (rot_dim - 2));
  double lo = 0.0, hi = 0.0;
  if (scaling == TM_ROPE_YARN) {
    lo = floor(rot_dim * log(original_max / (fast * two_pi)) / (2.0 * log(theta)));
    hi = ceil(rot_dim * log(original_max / (slow * two_pi)) / (2.0 * log(theta)));
    lo = lo > 0.0 ? lo : 0.0;
    hi = hi < rot_dim - 1 ? hi : rot_dim - 1;
  }
  for (int i = 0; i < 64; ++i) {
    rope->turns[i] = 0;
    if (i >= rot_dim / 2) continue;
    double f = pow(theta, -2.0 * i / rot_dim);
    if (scaling == TM_ROPE_LINEAR) f /= factor;
    if (scaling == TM_ROPE_YARN) {
      double r = (i - lo) / (hi - lo > 0.001 ? hi - lo : 0.001);
      r = r < 0.0 ? 0.0 : (r > 1.0 ? 1.0 : r);
      f = f * (1.0 - r) + f / factor * r;
    }
    if (scaling == TM_ROPE_BANDS) {
      double s = (original_max * f / two_pi - slow) / (fast - slow);
      s = s < 0.0 ? 0.0 : (s > 1.0 ? 1.0 : s);
      f = f * s + f / factor * (1.0 - s);
    }
    // f <= 1, so f / 2 pi is below 1/4 turn: the product stays below 2^62
    rope->turns[i] = static_cast<uint64_t>(llrint(f / two_pi * 18446744073709551616.0));
  }
  return TM_OK;
}

extern "C" tm_status tm_rope(const tm_tensor* q, const tm_tensor* k, tm_tensor* q_out, tm_tensor* k_out,
                             const tm_rope_freqs* rope, const int32_t* positions, int64_t pos_offset, void* stream) {
  if (rope == nullptr) return TM_ERR_INVALID_ARG;
  return tmk::rope_rows(q, k, q_out, k_out, nullptr, nullptr, 0.f, rope, positions, pos_offset, stream);
}

extern "C" tm_status tm_qk_norm_rope(const tm_tensor* q, const tm_tensor* k, tm_tensor* q_out, tm_tensor* k_out,
                                     const void* q_weight, const void* k_weight, float eps, const tm_rope_freqs* rope,
                                     const int32_t* positions, int64_t pos_offset, void* stream) {
  if (q_weight == nullptr || (k != nullptr && k_weight == nullptr) || !(eps >= 0.f) || !isfinite(eps))
    return TM_ERR_INVALID_ARG;
  return tmk::rope_rows(q, k, q_out, k_out, q_weight, k != nullptr ? k_weight : nullptr, eps, rope, positions,
                        pos_offset, stream);
}

extern "C" tm_status tm_kv_append(const tm_tensor* k, const tm_tensor* v, const tm_paged_kv* cache,
                                  const int32_t* table, int64_t table_stride, int32_t table_cols,
                                  const int32_t* kv_lens, const int32_t* cu_seqlens, int32_t batch,
                                  const tm_rope_freqs* rope, int64_t pos_offset, const tm_tensor* q, tm_tensor* q_out,
                                  const void* q_weight, const void* k_weight, float eps, void* stream) {
  using namespace tmk;
  TokenArgs a{};
  bool int8 = false;
  tm_status st = paged_pool(cache, &a.pool, &int8);
  if (st != TM_OK) return st;
  st = page_table(a.pool, table, table_stride, table_cols, &a.pt);
  if (st != TM_OK) return st;
  if (k == nullptr || kv_lens == nullptr || batch <= 0 || (q == nullptr) != (q_out == nullptr)) return TM_ERR_INVALID_ARG;
  const int64_t T = k->T, d = cache->d;
  if (T < 0 || !thd_ok(k, T, cache->H, d) || !thd_ok(v, T, cache->H, d)) return TM_ERR_INVALID_ARG;
  if (q != nullptr && (!thd_ok(q, T, q->H, d) || !thd_out_ok(q_out, T, q->H, d))) return TM_ERR_INVALID_ARG;
  if (cu_seqlens == nullptr && T % batch != 0) return TM_ERR_INVALID_ARG;
  if (!aligned(kv_lens, 4) || !aligned(cu_seqlens, 4) || !aligned(q_weight, 16) || !aligned(k_weight, 16))
    return TM_ERR_INVALID_ARG;
  if ((q_weight != nullptr || k_weight != nullptr) && (!(eps >= 0.f) || !isfinite(eps))) return TM_ERR_INVALID_ARG;
  if (rope != nullptr && !rope_ok(rope, d)) return TM_ERR_INVALID_ARG;
  if (cache->H > 65536 || (q != nullptr && q->H > 65536)) return TM_ERR_UNSUPPORTED;
  if (T == 0) return TM_OK;
  a.q = rows_of(q, q_out, q_weight);
  a.k = rows_of(k, nullptr, k_weight);
  a.v = rows_of(v, nullptr, nullptr);
  a.hq = q != nullptr ? static_cast<int>(q->H) : 0;
  a.hk = a.hv = cache->H;
  a.T = T;
  a.eps = eps;
  a.pos_offset = pos_offset;
  a.kv_lens = kv_lens;
  a.cu = cu_seqlens;
  a.batch = batch;
  a.per_seq = T / batch;
  set_rope(&a, rope);
  return launch_tokens(a, static_cast<int>(d), int8 ? kCacheI8 : kCacheF16, as_stream(stream));
}
