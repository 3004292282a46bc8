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
// and single steps by latency.  Rotation of 16384 tokens, 32 + 8 heads of 128
// (336 MB): 53.5 us, 0.96 of the measured copy bandwidth.  Norm and rotation of 8191
// tokens, 32 + 8 heads of 64 (84 MB): 16.3 us, 0.79 of it.  Appending 9616 tokens to
// INT8 pages, 4 heads of 128 with 32 query heads rotated (187 MB): 41 us, 0.70 of it:
// a third of the warps fit, and wait for loads first (issue slots 55 % used).  64 tokens:
// 3.5 us, a chain of loads.
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

// A warp takes one token and every `parts`-th item: 512 / D heads of Q, K or V.
// A lane holds 16 values of a head, in two 16-byte pieces chosen so that both
// members of every pair are its own: pieces l and l + rot / 16 in the half
// layout (and the unrotated rest two by two), neighbours in the interleaved
// one.  So the rotation needs no shuffles; the norm's sum takes log2(D / 16).
// U items are loaded before the first is used, to keep loads in flight.
//
// Loads in flight against warps, in registers: one item ahead and seven blocks on
// an SM for norms and for heads of 64 (norms of 4000 tokens, 32 + 8 heads of 128: 16.4
// us, with two and six 19.8; 8191 of 64: 16.3 and 17.6), two and six for rotation alone
// of heads of 128 (16384 tokens: 53.7 us, with one and seven 56.0) and for appending
// (with three and five 59.5 to 60.1 us in one case, 73.1 to 70.4 in another).
__host__ __device__ constexpr int items_ahead(int d, int cache, bool norm) {
  return cache == kNoCache && (norm || d == 64) ? 1 : 2;
}
__host__ __device__ constexpr int blocks_held(int d, int cache, bool norm) { return 8 - items_ahead(d, cache, norm); }

template <int D, int CACHE, bool NORM>
__global__ void __launch_bounds__(kTokenWarps * 32, blocks_held(D, CACHE, NORM)) token_kernel(const __grid_constant__ TokenArgs a, DevErr err) {
  constexpr int LPR = D / 16;         // lanes of a head
  constexpr int RPW = 32 / LPR;       // heads of an item
  constexpr int U = items_ahead(D, CACHE, NORM);
  __shared__ __align__(16) float2 trig[kTokenWarps][64];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t job = static_cast<int64_t>(blockIdx.x) * kTokenWarps + warp;
  int64_t t = job;
  int part = 0;
  if (a.parts > 1) {                  // then a.T * a.parts stays below 2^31
    t = static_cast<uint32_t>(job) / static_cast<uint32_t>(a.parts);
    part = static_cast<int>(job - t * a.parts);
  }
  if (t >= a.T) return;

  // this lane's head of an item, and its two pieces
  const int l = lane & (LPR - 1), sub = lane / LPR;
  const int pairs = a.rot >> 4;       // lanes of a head that rotate
  const bool turned = a.rope && l < pairs;
  int pa = 2 * l, pb = 2 * l + 1;     // unrotated: rot / 8 + 2 (l - rot / 16) = 2 l
  if (turned && !a.interleaved) {
    pa = l;
    pb = l + pairs;
  }

  const int iq = (a.hq + RPW - 1) / RPW, ik = (a.hk + RPW - 1) / RPW, iv = (a.hv + RPW - 1) / RPW;
  const int items = iq + ik + iv;
  uint4 raw[U][2];
  auto load = [&](int it, uint4 (&x)[2]) {
    const bool isq = it < iq, isk = it < iq + ik;        // the same for the whole warp
    const Rows& r = isq ? a.q : (isk ? a.k : a.v);
    const int h = (it - (isq ? 0 : (isk ? iq : iq + ik))) * RPW + sub;
    x[0] = x[1] = make_uint4(0, 0, 0, 0);
    if (it < items && h < (isq ? a.hq : (isk ? a.hk : a.hv))) {
      const uint4* src = reinterpret_cast<const uint4*>(r.in + t * r.in_t + h * r.in_h);      // in place: not ld.nc
      x[0] = src[pa];
      x[1] = src[pb];
    }
  };
  // before the token's sequence, place and page are looked up, a chain of loads of its own
#pragma unroll
  for (int u = 0; u < U; ++u) load(part + u * a.parts, raw[u]);

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
      if (i < 0) return;                   // before the first
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

  // sines and cosines of the token, up to two pairs per lane, while the loads are under way
  float cs[8], sn[8];
  if (a.rope) {
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int i = lane + 32 * r;
      if (i < (a.rot >> 1)) {
        const uint64_t turn = static_cast<uint64_t>(pos) * a.turns[i];
        const int32_t top = static_cast<int32_t>(static_cast<uint32_t>(turn >> 32));
        float s, c;
        sincospif(static_cast<float>(top) * 4.656612873077393e-10f, &s, &c);   // 2^-31: half turns
        trig[warp][i] = make_float2(c * a.mscale, s * a.mscale);
      }
    }
    __syncwarp();
    if (turned) {
#pragma unroll
      for (int e = 0; e < 8; e += 2) {
        const float4 f = *reinterpret_cast<const float4*>(&trig[warp][8 * l + e]);
        cs[e] = f.x;
        sn[e] = f.y;
        cs[e + 1] = f.z;
        sn[e + 1] = f.w;
      }
    }
  }

  for (int it0 = part; it0 < items; it0 += a.parts * U) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int it = it0 + u * a.parts;
      if (it >= items) break;                            // the same for the whole warp
      const bool isq = it < iq, isk = !isq && it < iq + ik, isv = !isq && !isk;
      const int h = (it - (isq ? 0 : (isk ? iq : iq + ik))) * RPW + sub;
      const bool real = h < (isq ? a.hq : (isk ? a.hk : a.hv));
      float x[2][8];
      unpack8(raw[u][0], x[0]);
      unpack8(raw[u][1], x[1]);
      load(it + a.parts * U, raw[u]);                    // the item after the next ones, into the registers just freed
      if (NORM && !isv) {
        const __half* w = isq ? a.q.weight : a.k.weight;
        if (w != nullptr) {
          float ss = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) ss += x[0][e] * x[0][e] + x[1][e] * x[1][e];
#pragma unroll
          for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
          const float inv = rsqrtf(ss * (1.0f / D) + a.eps);      // within 2^-22
          float wf[8];
          unpack8(__ldg(reinterpret_cast<const uint4*>(w) + pa), wf);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[0][e] = x[0][e] * inv * wf[e];
          unpack8(__ldg(reinterpret_cast<const uint4*>(w) + pb), wf);
#pragma unroll
          for (int e = 0; e < 8; ++e) x[1][e] = x[1][e] * inv * wf[e];
        }
      }
      if (turned && !isv) {
        if (a.interleaved) {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            float& p = x[e >> 2][2 * (e & 3)];
            float& q = x[e >> 2][2 * (e & 3) + 1];
            const float y = p * cs[e] - q * sn[e];
            q = p * sn[e] + q * cs[e];
            p = y;
          }
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float y = x[0][e] * cs[e] - x[1][e] * sn[e];
            x[1][e] = x[0][e] * sn[e] + x[1][e] * cs[e];
            x[0][e] = y;
          }
        }
      }
      if (CACHE == kCacheI8 && !isq) {
        // absmax as integer bits: a NaN compares above everything and so
        // reaches the scale
        uint32_t m = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          m = max(m, max(__float_as_uint(x[0][e]) & 0x7fffffffu, __float_as_uint(x[1][e]) & 0x7fffffffu));
#pragma unroll
        for (int o = LPR / 2; o > 0; o >>= 1) m = max(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (real && slot_row >= 0) {
          const __half s16 = __float2half_rn(__fdiv_rn(__uint_as_float(m), 127.0f));
          const float s = __half2float(s16);
          uint32_t c[2][2] = {{0, 0}, {0, 0}};
          if (s != 0.f) {
            // x * (1 / s) is within 2^-22 of the quotient, relative, so its nearest integer is the quotient's
            // unless it lies that close to the middle between two: then divide
            const float by = __frcp_rn(s);
            bool near = false;
#pragma unroll
            for (int p = 0; p < 2; ++p) {
              uint32_t n[8];
#pragma unroll
              for (int e = 0; e < 8; ++e) {
                const float r = fminf(fmaxf(x[p][e] * by, -127.0f), 127.0f);
                const float t = r + 12582912.0f;      // 1.5 * 2^23: the nearest integer, ties to even, in the low bits
                near = near || fabsf(r - (t - 12582912.0f)) > 0.4999f;
                n[e] = __float_as_uint(t);
              }
#pragma unroll
              for (int e = 0; e < 8; e += 4)
                c[p][e >> 2] = __byte_perm(__byte_perm(n[e], n[e + 1], 0x0040), __byte_perm(n[e + 2], n[e + 3], 0x0040),
                                           0x5410);
            }
            if (near) {
#pragma unroll
              for (int p = 0; p < 2; ++p) {
                c[p][0] = c[p][1] = 0;
#pragma unroll
                for (int e = 0; e < 8; ++e) {
                  const int v = max(-127, min(127, __float2int_rn(__fdiv_rn(x[p][e], s))));
                  c[p][e >> 2] |= static_cast<uint32_t>(v & 255) << (8 * (e & 3));
                }
              }
            }
          }
          uint8_t* row = (isk ? a.pool.k : a.pool.v) + slot_row + h * a.pool.stride_h;
          *reinterpret_cast<uint2*>(row + 8 * pa) = make_uint2(c[0][0], c[0][1]);
          *reinterpret_cast<uint2*>(row + 8 * pb) = make_uint2(c[1][0], c[1][1]);
          if (l == 0) (isk ? a.pool.ks : a.pool.vs)[slot_scale + h * a.pool.sstride_h] = s16;
        }
        continue;
      }
      if (!real) continue;
      uint4* dst;
      if (CACHE == kNoCache || isq) {
        const Rows& r = isq ? a.q : a.k;
        dst = reinterpret_cast<uint4*>(r.out + t * r.out_t + h * r.out_h);
      } else {
        if (slot_row < 0) continue;
        dst = reinterpret_cast<uint4*>((isk ? a.pool.k : a.pool.v) + slot_row + h * a.pool.stride_h);
      }
      dst[pa] = pack8(x[0]);
      dst[pb] = pack8(x[1]);
    }
  }
}

// Warps per token: enough of them for every SM to hold ten while a token has
// items to share out; with many tokens one warp takes a token whole, so that its
// sines and cosines are computed once.  An SM holds 24 or 28; with 28 each wave paid the
// chain before the first item again (1000 tokens, 32 + 8 heads of 128, with norms:
// 9.3 us instead of 7.6; 2000 tokens, 16 + 4 heads, rotation alone: 7.9 and 5.6 us).
int token_parts(int64_t T, int items) {
  const int64_t p = (static_cast<int64_t>(kSms) * 10 + T - 1) / T;
  return static_cast<int>(p < items ? p : items);
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
  const int rpw = 512 / d;
  a.parts = token_parts(a.T, (a.hq + rpw - 1) / rpw + (a.hk + rpw - 1) / rpw + (a.hv + rpw - 1) / rpw);
  const int64_t blocks = (a.T * a.parts + kTokenWarps - 1) / kTokenWarps;
  if (blocks > 0x7fffffff) return TM_ERR_UNSUPPORTED;
  const DevErr err{device_error_word()};
  if (err.word == nullptr) return cuda_fail(static_cast<int>(cudaErrorInvalidSymbol));
  const bool norm = a.q.weight != nullptr || a.k.weight != nullptr;
  auto kernel = norm ? (cache == kCacheI8 ? (d == 128 ? token_kernel<128, kCacheI8, true> : token_kernel<64, kCacheI8, true>)
                        : cache == kCacheF16 ? (d == 128 ? token_kernel<128, kCacheF16, true> : token_kernel<64, kCacheF16, true>)
                                             : (d == 128 ? token_kernel<128, kNoCache, true> : token_kernel<64, kNoCache, true>))
                     : (cache == kCacheI8 ? (d == 128 ? token_kernel<128, kCacheI8, false> : token_kernel<64, kCacheI8, false>)
                        : cache == kCacheF16 ? (d == 128 ? token_kernel<128, kCacheF16, false> : token_kernel<64, kCacheF16, false>)
                                             : (d == 128 ? token_kernel<128, kNoCache, false> : token_kernel<64, kNoCache, false>));
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
