// Per-head RMS norm and position rotation of queries and keys, alone
// (duo_qk_norm_rope) or on the way into the cache (duo_append_rope), and the
// append of the 8-bit cache.
//
// For a head vector x of D channels with norm weight w:
//   y = x * rsqrt(mean(x^2) + eps) * w                        (w null: y = x)
//   (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s) for every rotated pair (a, b),
//   c + i s = mscale * e^(i * position * inv_freq[pair]).
// All of it in fp32, rounded once to the input's type.  The angle is formed in
// 64 bits: at position 10^6 a 32-bit product is off by up to 0.06 radian.  As
// a fraction of a turn it is then reduced exactly to [-1/2, 1/2] and only
// that is rounded to fp32 (off by at most 2^-25 of a turn).  Pages: "What is
// DuoAttention" (nav.superapi.store), section "Technical principles of
// DuoAttention" (what each kind of head keeps); the pages leave positions to
// the model.
//
// A warp takes one token and a group of its head vectors: the angles and
// their sines depend on the token only, so they are computed once per group
// and reused for every head.  CPL channels per lane; the partner of a rotated
// channel is in the same lane (interleaved pairs) or CPL-aligned in another
// lane of the same vector, one shuffle per channel.
//
// 8-bit cache: a CTA takes one scale block (32 tokens) of one or more
// retrieval heads.  A block that the call completes is coded as a whole, its
// older tokens read from the bf16 tail; tokens of a block that stays open go
// to the tail.  scale = 2^e, the smallest e >= -120 with max|x| <= 448 * 2^e
// (finite values), code = x / scale rounded to nearest even e4m3, saturating
// (an infinity takes the largest code, a NaN stays one).  A power of two makes
// the division and the expansion to bf16 exact.
#include <algorithm>

#include "common.cuh"
#include "kv8.h"
#include "quant_int4.cuh"

namespace duo {
namespace ra {

enum Mode : int { kAlone = 0, kRaw = 1, kInt4 = 2, kFp8Mode = 3 };

template <typename T, int CPL>
struct Lane {  // CPL channels of one lane, as fp32
  __device__ __forceinline__ static void load(const T *p, float (&x)[CPL]) {
    if constexpr (sizeof(T) == 4) {
      if constexpr (CPL >= 4) {
#pragma unroll
        for (int i = 0; i < CPL / 4; ++i) {
          const float4 v = reinterpret_cast<const float4 *>(p)[i];
          x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
        }
      } else {
#pragma unroll
        for (int i = 0; i < CPL; ++i) x[i] = p[i];
      }
    } else {
      uint32_t w[CPL / 2];
      if constexpr (CPL == 8) {
        const uint4 v = *reinterpret_cast<const uint4 *>(p);
        w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
      } else if constexpr (CPL == 4) {
        const uint2 v = *reinterpret_cast<const uint2 *>(p);
        w[0] = v.x, w[1] = v.y;
      } else {
        w[0] = *reinterpret_cast<const uint32_t *>(p);
      }
#pragma unroll
      for (int i = 0; i < CPL / 2; ++i) {
        const float2 f = bf16x2_to_f2(w[i]);
        x[2 * i] = f.x, x[2 * i + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ static void store(T *p, const float (&x)[CPL]) {
    if constexpr (sizeof(T) == 4) {
      if constexpr (CPL >= 4) {
#pragma unroll
        for (int i = 0; i < CPL / 4; ++i)
          reinterpret_cast<float4 *>(p)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
      } else {
#pragma unroll
        for (int i = 0; i < CPL; ++i) p[i] = x[i];
      }
    } else {
      uint32_t w[CPL / 2];
#pragma unroll
      for (int i = 0; i < CPL / 2; ++i) {
        const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
        w[i] = *reinterpret_cast<const uint32_t *>(&h);
      }
      if constexpr (CPL == 8) *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
      else if constexpr (CPL == 4) *reinterpret_cast<uint2 *>(p) = make_uint2(w[0], w[1]);
      else *reinterpret_cast<uint32_t *>(p) = w[0];
    }
  }
};

// cos and sin (times mscale) of this lane's channels at one position.  sn
// carries the sign of the channel's own side of its pair: out = x * cs +
// partner * sn.  Channels past rot_dim get (1, 0).
template <typename T, int CPL>
__device__ __forceinline__ void rotation(const RopeParams &r, int64_t pos, int c0, float (&cs)[CPL],
                                         float (&sn)[CPL]) {
  constexpr double kPerTurn = 0.15915494309189533576888;  // 1 / (2 pi)
  const int half = r.rot_dim >> 1;
  const double p = (double)pos * kPerTurn;
#pragma unroll
  for (int j = 0; j < CPL; ++j) {
    const int c = c0 + j;
    if (c >= r.rot_dim) {
      cs[j] = 1.f;
      sn[j] = 0.f;
      continue;
    }
    const int pair = r.interleaved ? c >> 1 : (c < half ? c : c - half);
    const double turns = p * (double)r.inv_freq[pair];
    const float f = (float)(turns - rint(turns));  // [-1/2, 1/2]
    float s, k;
    if constexpr (sizeof(T) == 4) {
      sincospif(2.f * f, &s, &k);
    } else {
      // the hardware's sine and cosine are off by about 2^-21 on [-pi, pi],
      // far below the half step 2^-8 of the bf16 result
      __sincosf(6.283185307179586f * f, &s, &k);
    }
    const bool second = r.interleaved ? (c & 1) : (c >= half);
    cs[j] = k * r.mscale;
    sn[j] = (second ? s : -s) * r.mscale;
  }
}

// Sum of squares over a vector: one tree over its channel pairs, in the same
// order whatever the lanes hold, so that every kernel here gives the same bits.
template <int LPR, int CPL>
__device__ __forceinline__ float sum_squares(const float (&x)[CPL]) {
  float s[CPL / 2];
#pragma unroll
  for (int i = 0; i < CPL / 2; ++i) s[i] = fmaf(x[2 * i + 1], x[2 * i + 1], x[2 * i] * x[2 * i]);
#pragma unroll
  for (int n = CPL / 4; n > 0; n >>= 1)
#pragma unroll
    for (int i = 0; i < n; ++i) s[i] = s[2 * i] + s[2 * i + 1];
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) s[0] += __shfl_xor_sync(0xffffffffu, s[0], o);
  return s[0];
}

// Norm (w non-null) and rotation of one vector; every lane of the warp calls.
template <typename T, int D, int CPL>
__device__ __forceinline__ void norm_rotate(const RopeParams &r, const void *w, int sl,
                                            const float (&cs)[CPL], const float (&sn)[CPL],
                                            float (&x)[CPL]) {
  constexpr int LPR = D / CPL;
  if (w) {
    const float inv = rsqrtf(sum_squares<LPR, CPL>(x) * (1.f / D) + r.eps);
    float wv[CPL];
    Lane<T, CPL>::load(static_cast<const T *>(w) + sl * CPL, wv);
#pragma unroll
    for (int j = 0; j < CPL; ++j) x[j] = x[j] * inv * wv[j];
  }
  if (r.rot_dim == 0) return;
  if (r.interleaved) {
#pragma unroll
    for (int j = 0; j < CPL; j += 2) {
      const float a = x[j], b = x[j + 1];
      x[j] = fmaf(a, cs[j], b * sn[j]);
      x[j + 1] = fmaf(b, cs[j + 1], a * sn[j + 1]);
    }
  } else {
    // the partner channels are half / CPL lanes further (first half) or back
    const int lanes = (r.rot_dim >> 1) / CPL;
    const int from = (threadIdx.x & 31) + (sl < lanes ? lanes : (sl < 2 * lanes ? -lanes : 0));
#pragma unroll
    for (int j = 0; j < CPL; ++j) {
      const float partner = __shfl_sync(0xffffffffu, x[j], from);
      x[j] = fmaf(x[j], cs[j], partner * sn[j]);
    }
  }
}

// ------------------------------------------------------------ 8-bit blocks

// The scale's exponent of a block whose largest finite |x| is amax (a bf16
// value): 448 = 1.75 * 2^8, so e = exponent(amax) - 8, one more past 1.75.
__device__ __forceinline__ int scale_exp(float amax) {
  const uint32_t u = __float_as_uint(amax);
  const int e = (int)(u >> 23) - 127 - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return max(e, -120);
}

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }

__device__ __forceinline__ uint16_t e4m3x2(float lo, float hi) {
  uint16_t d;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(d) : "f"(hi), "f"(lo));
  return d;
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;  // infinities and NaN do not set the scale
}

constexpr int kThreads = 256;

// One scale-block CTA: launch row r, heads [h0, h1), item `item` (see the
// launch).  256 threads = 16 half-warps of 16 lanes, 2 tokens each.
template <int D>
__device__ __forceinline__ void block_cta(const RopeRowsParams &P, int r, int h0, int h1, int item) {
  static_assert(D == 128, "the 8-bit cache has head_dim 128");
  using bf = __nv_bfloat16;
  constexpr int CPL = 8;
  __shared__ float s_max[2][2][kThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5;
  const int hw = tid >> 4, sl = tid & 15;  // half-warp, lane in the vector
  const AppendParams &a = P.a;
  const int b = a.rows.row[r];
  const int64_t len = a.rows.len[r];
  // local retrieval rows before and after the call (a sequence shard keeps
  // positions [shard_lo, shard_hi) at row position - shard_lo)
  const int64_t l0 = max((int64_t)0, min(len, a.shard_hi) - a.shard_lo);
  const int64_t l1 = max((int64_t)0, min(len + a.n_tok, a.shard_hi) - a.shard_lo);
  if (l1 <= l0) return;
  const int64_t fb = l0 >> kScaleShift, done = l1 >> kScaleShift;  // blocks [fb, done) become full
  const bool open = (l1 & (kScaleBlock - 1)) != 0;
  const int n_items = (int)max((int64_t)1, done - fb);
  if (item >= n_items) return;
  int buf = 0;
  // Item 0 also writes the block that stays open, after the first block's
  // older tokens have been read from the same tail rows.
  for (int part = 0; part < 2; ++part) {
    const int64_t blk = part == 0 ? fb + item : done;
    const bool full = part == 0;
    if (part == 0 && blk >= done) continue;
    if (part == 1 && (item != 0 || !open)) break;
    if (part == 1) __syncthreads();
    float cs[2][CPL] = {}, sn[2][CPL] = {};
    const bf *src_k[2], *src_v[2];
    bool fresh[2], have[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t l = (blk << kScaleShift) + hw * 2 + i;  // local row
      fresh[i] = l >= l0 && l < l1;
      have[i] = full || fresh[i];
      const int64_t t = l + a.shard_lo - len;               // token of the call
      const int64_t tok = (int64_t)r * a.n_tok + t;
      src_k[i] = static_cast<const bf *>(P.k.p) + tok * P.k.tok;
      src_v[i] = static_cast<const bf *>(P.v.p) + tok * P.v.tok;
      if (fresh[i] && P.rope.rot_dim)
        rotation<bf, CPL>(P.rope, P.positions ? P.positions[tok] : len + t, sl * CPL, cs[i], sn[i]);
    }
    for (int h = h0; h < h1; ++h) {
      const int kvh = a.h.ret_heads[h];
      bf *tk = reinterpret_cast<bf *>(P.tail.k) + ((int64_t)b * a.n_ret + h) * kScaleBlock * D;
      bf *tv = reinterpret_cast<bf *>(P.tail.v) + ((int64_t)b * a.n_ret + h) * kScaleBlock * D;
      float k[2][CPL], v[2][CPL];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int slot = hw * 2 + i;
        const bf *pk = fresh[i] ? src_k[i] + (int64_t)kvh * P.k.head : tk + slot * D;
        const bf *pv = fresh[i] ? src_v[i] + (int64_t)kvh * P.v.head : tv + slot * D;
        if (have[i]) {
          Lane<bf, CPL>::load(pk + sl * CPL, k[i]);
          Lane<bf, CPL>::load(pv + sl * CPL, v[i]);
        } else {
#pragma unroll
          for (int j = 0; j < CPL; ++j) k[i][j] = v[i][j] = 0.f;
        }
      }
      float mk = 0.f, mv = 0.f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        // the two vectors of a warp's halves may differ in kind (tail or
        // new): all lanes rotate, the tail's keep what they had
        float x[CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j) x[j] = k[i][j];
        norm_rotate<bf, D, CPL>(P.rope, P.rope.k_norm, sl, cs[i], sn[i], x);
#pragma unroll
        for (int j = 0; j < CPL; ++j) {
          // rounded to bf16 first: what the rotated keys are everywhere else
          if (fresh[i]) k[i][j] = __bfloat162float(__float2bfloat16_rn(x[j]));
          mk = fmaxf(mk, finite_abs(k[i][j]));
          mv = fmaxf(mv, finite_abs(v[i][j]));
        }
      }
      if (!full) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (!fresh[i]) continue;
          const int slot = hw * 2 + i;
          Lane<bf, CPL>::store(tk + slot * D + sl * CPL, k[i]);
          Lane<bf, CPL>::store(tv + slot * D + sl * CPL, v[i]);
        }
        continue;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        mk = fmaxf(mk, __shfl_xor_sync(0xffffffffu, mk, o));
        mv = fmaxf(mv, __shfl_xor_sync(0xffffffffu, mv, o));
      }
      // two sets of slots in turn: one barrier a head
      if ((tid & 31) == 0) {
        s_max[buf][0][warp] = mk;
        s_max[buf][1][warp] = mv;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < kThreads / 32; ++i) {
        mk = fmaxf(mk, s_max[buf][0][i]);
        mv = fmaxf(mv, s_max[buf][1][i]);
      }
      buf ^= 1;
      const int ek = scale_exp(mk), ev = scale_exp(mv);
      const float ik = pow2i(-ek), iv = pow2i(-ev);
      const int64_t row = ret_row(a.ret, b, h, blk << kScaleShift);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint16_t ck[CPL / 2], cv[CPL / 2];
#pragma unroll
        for (int j = 0; j < CPL / 2; ++j) {
          ck[j] = e4m3x2(k[i][2 * j] * ik, k[i][2 * j + 1] * ik);
          cv[j] = e4m3x2(v[i][2 * j] * iv, v[i][2 * j + 1] * iv);
        }
        const int64_t at = (row + hw * 2 + i) * D + sl * CPL;
        *reinterpret_cast<uint2 *>(a.p.ret_k + at) =
            make_uint2(ck[0] | (uint32_t)ck[1] << 16, ck[2] | (uint32_t)ck[3] << 16);
        *reinterpret_cast<uint2 *>(a.p.ret_v + at) =
            make_uint2(cv[0] | (uint32_t)cv[1] << 16, cv[2] | (uint32_t)cv[3] << 16);
      }
      if (tid == 0) {
        reinterpret_cast<float *>(a.p.ret_k_sz)[row >> kScaleShift] = pow2i(ek);
        reinterpret_cast<float *>(a.p.ret_v_sz)[row >> kScaleShift] = pow2i(ev);
      }
    }
  }
}

// ------------------------------------------------------------ vectors

// Work of the row CTAs: (token, group of RPW * NIT head vectors) per warp.
// Head vectors of a token: the Hq queries (when given), then the K heads and,
// for an append, the V heads; 8-bit caches list their streaming heads only.
template <typename T, int D, int MODE, int NIT>
__global__ void __launch_bounds__(kThreads) rope_rows_kernel(const __grid_constant__ RopeRowsParams P,
                                                             int block_ctas) {
  // 4-bit codes are made by a whole warp per vector (quantize_row_int4)
  constexpr int CPL = MODE == kInt4 ? D / 32 : 8;
  constexpr int LPR = D / CPL, RPW = 32 / LPR;
  const AppendParams &a = P.a;
  if constexpr (MODE == kFp8Mode) {
    if ((int)blockIdx.x < block_ctas) {
      const int groups = (a.n_ret + P.heads_per_cta - 1) / P.heads_per_cta;
      const int item = blockIdx.x % P.block_items;
      const int y = blockIdx.x / P.block_items;
      const int h0 = (y % groups) * P.heads_per_cta;
      block_cta<D>(P, y / groups, h0, min(a.n_ret, h0 + P.heads_per_cta), item);
      return;
    }
  }
  const int lane = threadIdx.x & 31, sl = lane % LPR, sub = lane / LPR;
  const int nq = P.q.p ? P.Hq : 0;
  const int nk = MODE == kFp8Mode ? a.n_str : P.Hkv;
  const int vecs = nq + (MODE == kAlone ? nk : 2 * nk);
  if (vecs == 0) return;
  const int groups = (vecs + RPW * NIT - 1) / (RPW * NIT);
  const int64_t warps = P.tokens * groups;
  const int64_t stride = (int64_t)(gridDim.x - block_ctas) * (kThreads / 32);
  for (int64_t w = (int64_t)(blockIdx.x - block_ctas) * (kThreads / 32) + (threadIdx.x >> 5); w < warps;
       w += stride) {
    const int64_t tok = w / groups;
    const int v0 = (int)(w % groups) * RPW * NIT;
    // where the token goes in the cache
    int lr = 0, b = 0;
    int64_t p = 0, end = 0;
    if constexpr (MODE != kAlone) {
      lr = (int)(tok / a.n_tok);
      b = a.rows.row[lr];
      p = a.rows.len[lr] + (tok - lr * a.n_tok);
      end = a.rows.len[lr] + a.n_tok;
    }
    const bool kept_ret = MODE == kAlone || (p >= a.shard_lo && p < a.shard_hi);
    const bool kept_str = MODE == kAlone || p < a.S || p >= end - a.R;
    float x[NIT][CPL];
    int vec[NIT];   // this lane's vector, -1: none
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
      int vi = v0 + i * RPW + sub;
      const T *src = nullptr;
      if (vi < nq) {
        src = static_cast<const T *>(P.q.p) + tok * P.q.tok + (int64_t)vi * P.q.head;
      } else if (vi < vecs) {
        const bool isv = vi >= nq + nk;
        const int h = vi - nq - (isv ? nk : 0);
        const int kvh = MODE == kFp8Mode ? a.h.str_heads[h] : h;
        const HeadView &in = isv ? P.v : P.k;
        if (MODE == kAlone || (a.h.kind[kvh] ? kept_ret : kept_str))
          src = static_cast<const T *>(in.p) + tok * in.tok + (int64_t)kvh * in.head;
      }
      if (src) {
        Lane<T, CPL>::load(src + sl * CPL, x[i]);
      } else {
        vi = -1;
#pragma unroll
        for (int j = 0; j < CPL; ++j) x[i][j] = 0.f;
      }
      vec[i] = vi;
    }
    float cs[CPL], sn[CPL];
    if (P.rope.rot_dim && v0 < nq + nk)
      rotation<T, CPL>(P.rope, P.positions ? P.positions[tok] : p, sl * CPL, cs, sn);
#pragma unroll
    for (int i = 0; i < NIT; ++i) {
      // queries and keys; a warp may hold both and values too, so the norm's
      // weight is chosen per half and values keep what was loaded
      const int base = v0 + i * RPW;  // the warp's first vector of this step
      if (base < nq + nk) {
        float y[CPL];
#pragma unroll
        for (int j = 0; j < CPL; ++j) y[j] = x[i][j];
        const int vi = base + sub;
        const void *wq = P.rope.q_norm, *wk = P.rope.k_norm;
        const bool mixed = base < nq && base + RPW > nq;
        const void *w = vi < nq ? wq : wk;
        if (!mixed || (wq != nullptr) == (wk != nullptr)) {
          norm_rotate<T, D, CPL>(P.rope, w, sl, cs, sn, y);
        } else {
          // only one of the two is normed: the other half's result is replaced
          float z[CPL];
#pragma unroll
          for (int j = 0; j < CPL; ++j) z[j] = y[j];
          norm_rotate<T, D, CPL>(P.rope, wq ? wq : wk, sl, cs, sn, y);
          norm_rotate<T, D, CPL>(P.rope, nullptr, sl, cs, sn, z);
#pragma unroll
          for (int j = 0; j < CPL; ++j) y[j] = w ? y[j] : z[j];
        }
        if (vi < nq + nk) {
#pragma unroll
          for (int j = 0; j < CPL; ++j) x[i][j] = y[j];
        }
      }
      const int vi = vec[i];
      if constexpr (MODE == kInt4) {
        // one vector a warp: vi is uniform
        if (vi < 0) continue;
        if (vi < nq) {
          Lane<T, CPL>::store(static_cast<T *>(P.q_out) + (tok * P.Hq + vi) * D + sl * CPL, x[i]);
          continue;
        }
        const bool isv = vi >= nq + nk;
        const int kvh = vi - nq - (isv ? nk : 0);
        const int idx = a.h.index[kvh];
        const bool ret = a.h.kind[kvh];
        const int64_t row = ret ? ret_row(a.ret, b, idx, p - a.shard_lo)
                                : ((int64_t)b * a.n_str + idx) * a.Ws + ring_slot(p, a.S, a.R);
        uint8_t *codes = ret ? (isv ? a.p.ret_v : a.p.ret_k) : (isv ? a.p.str_v : a.p.str_k);
        uint8_t *sz = ret ? (isv ? a.p.ret_v_sz : a.p.ret_k_sz) : (isv ? a.p.str_v_sz : a.p.str_k_sz);
        // rounded to bf16 first, so that the codes are those of appending
        // the rotated keys
#pragma unroll
        for (int j = 0; j < CPL; ++j) x[i][j] = __bfloat162float(__float2bfloat16_rn(x[i][j]));
        __half sch, zph;
        const uint32_t packed = quantize_row_int4<CPL>(x[i], &sch, &zph);
        uint8_t *dst = codes + row * (D / 2) + lane * (CPL / 2);
        if constexpr (CPL == 4) *reinterpret_cast<uint16_t *>(dst) = (uint16_t)packed;
        else *dst = (uint8_t)packed;
        if (lane == 0) {
          __half2 pair;
          pair.x = sch;
          pair.y = zph;
          reinterpret_cast<__half2 *>(sz)[row] = pair;
        }
      } else {
        if (vi < 0) continue;
        T *dst;
        if (vi < nq) {
          dst = static_cast<T *>(P.q_out) + (tok * P.Hq + vi) * D;
        } else if constexpr (MODE == kAlone) {
          dst = static_cast<T *>(P.k_out) + (tok * P.Hkv + (vi - nq)) * D;
        } else {
          const bool isv = vi >= nq + nk;
          const int h = vi - nq - (isv ? nk : 0);
          const int kvh = MODE == kFp8Mode ? a.h.str_heads[h] : h;
          const int idx = a.h.index[kvh];
          if (a.h.kind[kvh])
            dst = reinterpret_cast<T *>(isv ? a.p.ret_v : a.p.ret_k) +
                  ret_row(a.ret, b, idx, p - a.shard_lo) * D;
          else
            dst = reinterpret_cast<T *>(isv ? a.p.str_v : a.p.str_k) +
                  (((int64_t)b * a.n_str + idx) * a.Ws + ring_slot(p, a.S, a.R)) * D;
        }
        Lane<T, CPL>::store(dst + sl * CPL, x[i]);
      }
    }
  }
}

template <typename T, int D, int MODE>
cudaError_t run(const RopeRowsParams &P, int block_ctas, cudaStream_t s) {
  constexpr int CPL = MODE == kInt4 ? D / 32 : 8;
  constexpr int RPW = 32 * CPL / D;
  const int nq = P.q.p ? P.Hq : 0;
  const int nk = MODE == kFp8Mode ? P.a.n_str : P.Hkv;
  const int64_t vecs = nq + (MODE == kAlone ? nk : 2 * nk);
  // Vectors per warp: 4 steps share a token's angles, but a short call has
  // too few warps then, and one step each is faster.
  const int64_t warps4 = P.tokens * ((vecs + RPW * 4 - 1) / (RPW * 4));
  const bool four = warps4 >= 148 * 16;
  const int64_t warps = four ? warps4 : P.tokens * ((vecs + RPW - 1) / RPW);
  int64_t ctas = (warps + kThreads / 32 - 1) / (kThreads / 32);
  ctas = ctas < 148 * 64 ? ctas : 148 * 64;
  const unsigned grid = (unsigned)(block_ctas + ctas);
  if (grid == 0) return cudaSuccess;
  if (four) rope_rows_kernel<T, D, MODE, 4><<<grid, kThreads, 0, s>>>(P, block_ctas);
  else rope_rows_kernel<T, D, MODE, 1><<<grid, kThreads, 0, s>>>(P, block_ctas);
  return cudaGetLastError();
}

}  // namespace ra

cudaError_t launch_qk_norm_rope(const RopeRowsParams &P, int io_type, int D, cudaStream_t s) {
  using bf = __nv_bfloat16;
  if (P.tokens <= 0) return cudaSuccess;
  if (io_type == kF32) return D == 128 ? ra::run<float, 128, ra::kAlone>(P, 0, s) : ra::run<float, 64, ra::kAlone>(P, 0, s);
  return D == 128 ? ra::run<bf, 128, ra::kAlone>(P, 0, s) : ra::run<bf, 64, ra::kAlone>(P, 0, s);
}

cudaError_t launch_append_rope(const RopeRowsParams &Pin, int kv_type, cudaStream_t s) {
  using bf = __nv_bfloat16;
  RopeRowsParams P = Pin;
  const AppendParams &a = P.a;
  if (P.tokens <= 0) return cudaSuccess;
  const bool d128 = a.D == 128;
  if (kv_type == kF32) return d128 ? ra::run<float, 128, ra::kRaw>(P, 0, s) : ra::run<float, 64, ra::kRaw>(P, 0, s);
  if (kv_type == kBF16) return d128 ? ra::run<bf, 128, ra::kRaw>(P, 0, s) : ra::run<bf, 64, ra::kRaw>(P, 0, s);
  if (kv_type == kINT4) return d128 ? ra::run<bf, 128, ra::kInt4>(P, 0, s) : ra::run<bf, 64, ra::kInt4>(P, 0, s);
  if (kv_type != kFP8 || !d128) return cudaErrorInvalidValue;
  // 8-bit: per launch row one item per block that becomes full (at least
  // one), times groups of retrieval heads
  int64_t items = 0;
  for (int r = 0; r < a.rows.n; ++r) {
    const int64_t len = a.rows.len[r];
    const int64_t l0 = std::max<int64_t>(0, std::min<int64_t>(len, a.shard_hi) - a.shard_lo);
    const int64_t l1 = std::max<int64_t>(0, std::min<int64_t>(len + a.n_tok, a.shard_hi) - a.shard_lo);
    if (l1 > l0) items = std::max<int64_t>(items, std::max<int64_t>(1, (l1 >> kScaleShift) - (l0 >> kScaleShift)));
  }
  int64_t ctas = 0;
  P.block_items = (int)std::max<int64_t>(1, items);
  P.heads_per_cta = 1;
  if (items > 0 && a.n_ret > 0) {
    // several heads share a token's angles; one each while that leaves SMs idle
    while (P.heads_per_cta < a.n_ret &&
           (int64_t)a.rows.n * items * ((a.n_ret + 2 * P.heads_per_cta - 1) / (2 * P.heads_per_cta)) >= 148 * 4)
      P.heads_per_cta *= 2;
    ctas = (int64_t)a.rows.n * items * ((a.n_ret + P.heads_per_cta - 1) / P.heads_per_cta);
  }
  if (ctas > (1 << 30)) return cudaErrorInvalidValue;
  return ra::run<bf, 128, ra::kFp8Mode>(P, (int)ctas, s);
}

}  // namespace duo
