// Per-head RMS norm and position rotation of queries and keys, alone
// (duo_qk_norm_rope) or on the way into the cache (duo_append_rope), and the
// append of the 8-bit cache.
//
// For a head vector x of D channels with norm weight w:
//   y = x * rsqrt(mean(x^2) + eps) * w                        (w null: y = x)
//   (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s) for every rotated pair (a, b),
//   c + i s = mscale * e^(i * position * inv_freq[pair]).
// All of it in fp32, rounded once to the input's type.  The angle is formed in
// 64 bits, as a fixed-point fraction of a turn: at position 10^6 a 32-bit
// floating-point product is off by up to 0.06 radian.  Pages: "What is
// DuoAttention" (nav.superapi.store), section "Technical principles of
// DuoAttention" (what each kind of head keeps); the pages leave positions to
// the model.
//
// Layout.  A vector's channels are spread over D/8 lanes, 8 each: two quads of
// 4, chosen so that both channels of every rotated pair are in one lane
// (quads i and i + rot_dim/8, or neighbours when interleaved), so rotating
// needs no exchange.  Row CTAs take kTok tokens: the tokens' sines and cosines
// go to shared memory once and serve all their
// vectors, each lane holding the four (cos, sin) of its pairs.
//
// Bound: HBM, each vector read and written once.  Measured: 4096 tokens of 32
// + 8 bf16 heads 14.3 us (5.9 TB/s, 0.89 of the copy rate), 4 x 1777 tokens of
// 32 + 32 heads into a bf16 cache 43.7 us (0.72); short calls 2.7 us.  What is
// left is load latency, next to it instruction issue: 64 registers (four
// vectors waiting, packed) let 32 warps share an SM.  They fit the full
// rotation of halves; the other bf16 variants spill 48 to 112 bytes a thread:
// the same call with pairs of neighbours 17.6 us, with half the channels
// rotated 16.5, with both 19.6.  fp32, 80 registers: 32.7, 34.3, 33.0 and 34.8
// us for twice the bytes (0.78 to 0.73).  Slower: a ring of
// asynchronous copies in shared memory (23.5 us at 4096 tokens when the kernel
// took 19.4), two tokens a CTA (16.6 against 14.5), six vectors waiting (19.3).
//
// 8-bit cache: a CTA takes the K or V of one scale block (32 tokens) of one or
// more retrieval heads.  A block that the call completes is coded as a whole,
// its older tokens read from the bf16 tail; tokens of a block that stays open
// go to the tail.  scale = 2^e, the smallest e >= -120 with max|x| <= 448 *
// 2^e (finite values), code = x / scale rounded to nearest even e4m3,
// saturating (an infinity takes the largest code, a NaN stays one; at e = 120,
// where codes past 240 would stand for more than fp32 holds, 240 is the
// largest).  A power
// of two makes the division and the expansion to bf16 exact.  8192 tokens of 4
// retrieval heads with 32 query heads: 43.3 us (0.57); without queries 15.6, most
// of it the blocks: an angle is formed for four heads only, and each CTA's
// set-up, loads, largest values and stores follow one another.
#include <algorithm>

#include "common.cuh"
#include "kv8.h"

namespace duo {
namespace ra {

enum Mode : int { kAlone = 0, kRaw = 1, kInt4 = 2, kFp8Mode = 3 };

constexpr int kTok = 4;     // tokens of a row CTA
constexpr int kBatch = 4;   // vectors a lane group loads at once
// Heads a scale-block CTA has on their way, asynchronous copies into shared
// memory (8192 tokens of 32 heads: 38.9 us, three 39.4, loads into registers a
// head ahead 42.2).
constexpr int kRing = 2;

// Threads of a CTA.  Four warps: a chunk's CTAs are all on the SMs at once, and
// the set-up's latency is paid once (4096 tokens x 40 heads, 1024 CTAs: 15.6 us
// with 128 threads, 17.6 with 256).  A scale block takes 16 half-warps (3000
// tokens of 8 heads: 10 us, 13 in eight with four tokens each).
constexpr int kBlockThreads = 256, kRowThreads = 128;
constexpr int threads_of(int mode) { return mode == kFp8Mode ? kBlockThreads : kRowThreads; }
// CTAs an SM has to hold: 64 registers a thread, 80 for fp32; 72 for the
// appends (4 x 1777 tokens of 96 vectors: 43.5 us, 45.7 with 64, 47.0 with 80;
// the 4-bit append spills 28 bytes so and takes 95.7, its divisions);
// 80 for the 8-bit append, whose scale blocks spill with less (3000 tokens of 32
// heads: 22.4 us, 28.5 with 64).
constexpr int ctas_of(int mode, int elt) {
  return (elt == 4 || mode == kFp8Mode ? 768 : mode == kRaw || mode == kInt4 ? 896 : 1024) / threads_of(mode);
}

// A lane's two quads as loaded: what waits in registers for its turn.  Every
// input is read once, so it is not kept in the caches (4096 tokens x 40 heads:
// 19.6 us with plain loads, 17.7 with these).
template <typename T>
struct Raw;
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p, int qa, int qb) {
    a = __ldcs(reinterpret_cast<const float4 *>(p + qa));
    b = __ldcs(reinterpret_cast<const float4 *>(p + qb));
  }
  __device__ __forceinline__ void unpack(float (&x)[8]) const {
    x[0] = a.x, x[1] = a.y, x[2] = a.z, x[3] = a.w, x[4] = b.x, x[5] = b.y, x[6] = b.z, x[7] = b.w;
  }
};
template <>
struct Raw<__nv_bfloat16> {
  uint2 a, b;
  __device__ __forceinline__ void load(const __nv_bfloat16 *p, int qa, int qb) {
    a = __ldcs(reinterpret_cast<const uint2 *>(p + qa));
    b = __ldcs(reinterpret_cast<const uint2 *>(p + qb));
  }
  __device__ __forceinline__ void unpack(float (&x)[8]) const {
    const uint32_t w[4] = {a.x, a.y, b.x, b.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 f = bf16x2_to_f2(w[i]);
      x[2 * i] = f.x, x[2 * i + 1] = f.y;
    }
  }
  __device__ __forceinline__ void pack(const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t *>(&v);
    }
    a = make_uint2(w[0], w[1]), b = make_uint2(w[2], w[3]);
  }
  __device__ __forceinline__ void store(__nv_bfloat16 *p, int qa, int qb) const {
    *reinterpret_cast<uint2 *>(p + qa) = a;
    *reinterpret_cast<uint2 *>(p + qb) = b;
  }
};

// Four channels of one lane.
__device__ __forceinline__ void load_quad(const float *p, float *x) {
  const float4 v = *reinterpret_cast<const float4 *>(p);
  x[0] = v.x, x[1] = v.y, x[2] = v.z, x[3] = v.w;
}
__device__ __forceinline__ void load_quad(const __nv_bfloat16 *p, float *x) {
  const uint2 v = *reinterpret_cast<const uint2 *>(p);
  const float2 a = bf16x2_to_f2(v.x), b = bf16x2_to_f2(v.y);
  x[0] = a.x, x[1] = a.y, x[2] = b.x, x[3] = b.y;
}
__device__ __forceinline__ void store_quad(float *p, const float *x) {
  *reinterpret_cast<float4 *>(p) = make_float4(x[0], x[1], x[2], x[3]);
}
__device__ __forceinline__ void store_quad(__nv_bfloat16 *p, const float *x) {
  const __nv_bfloat162 a = __floats2bfloat162_rn(x[0], x[1]), b = __floats2bfloat162_rn(x[2], x[3]);
  *reinterpret_cast<uint2 *>(p) =
      make_uint2(*reinterpret_cast<const uint32_t *>(&a), *reinterpret_cast<const uint32_t *>(&b));
}

// First channels of a lane's two quads.
struct Quads {
  int a, b;
};
__device__ __forceinline__ Quads quads_of(const RopeParams &r, int sl) {
  const int n = r.interleaved ? 0 : r.rot_dim >> 3;  // lanes whose quads are partners
  if (sl < n) return {4 * sl, 4 * (sl + n)};
  return {8 * sl, 8 * sl + 4};
}

// inv_freq / (2 pi) as a 64-bit fraction of a turn, modulo whole turns: the
// 24-bit significand times the leading 64 bits of 1 / (2 pi) (scaled by 2^66),
// shifted by the exponent.  Off by less than |inv_freq| / 4 + 1 units of 2^-64
// (the constant's truncation and the shift's); of finite frequencies only.
__device__ __forceinline__ uint64_t turn_rate(float inv_freq) {
  constexpr uint64_t kInvTwoPi = 0xA2F9836E4E441529ull;
  const uint32_t u = __float_as_uint(inv_freq);
  const int e = (u >> 23) & 0xff;
  const uint64_t m = (u & 0x7fffffu) | (e ? 0x800000u : 0u);
  const int sh = 152 - max(e, 1);
  const uint64_t hi = __umul64hi(m, kInvTwoPi), lo = m * kInvTwoPi;
  uint64_t f;
  if (sh >= 64) f = sh < 128 ? hi >> (sh - 64) : 0;
  else if (sh > 0) f = lo >> sh | hi << (64 - sh);
  else f = sh > -64 ? lo << -sh : 0;
  return u >> 31 ? 0 - f : f;
}

// (cos, sin) of pos * rate turns.  The product modulo 2^64 is the turn's
// fraction with nothing lost (a far position keeps its phase); its upper half
// is split into the nearest quarter turn and a rest of at most pi/4, whose
// sine and cosine are their Taylor sums (the first terms left out are below
// 2e-9 and 3e-8).  Integer and fp32 pipes only: a scale-block CTA forms 2048
// angles, and 64-bit floating-point work for them took it a microsecond more.
__device__ __forceinline__ float2 cos_sin(int64_t pos, uint64_t rate) {
  const uint32_t t = (uint32_t)(((uint64_t)pos * rate) >> 32);
  const uint32_t q = (t + 0x20000000u) >> 30;  // nearest quarter turn
  const int32_t r = (int32_t)(t - (q << 30));
  // x + dx = r * 2 pi / 2^32 to twice the precision, so that a key's rounding
  // does not depend on the angle's
  constexpr float kUnit = 1.46291807e-9f, kUnitLow = (float)(6.283185307179586 / 4294967296.0 - (double)kUnit);
  const float rh = (float)(r & ~255), rl = (float)(r & 255);  // both exact
  const float x = rh * kUnit;
  const float dx = fmaf(rl, kUnit, fmaf(rh, kUnitLow, fmaf(rh, kUnit, -x)));
  const float z = x * x;
  float c = fmaf(z, 2.4801587e-5f, -1.3888889e-3f);  // 1/8!, -1/6!
  c = fmaf(z, c, 4.1666667e-2f);                     // 1/4!
  c = z * fmaf(z, c, -0.5f);                         // cos x - 1
  float s = fmaf(z, 2.7557319e-6f, -1.9841270e-4f);  // 1/9!, -1/7!
  s = fmaf(z, s, 8.3333333e-3f);                     // 1/5!
  s = x * z * fmaf(z, s, -0.16666667f);              // sin x - x, -1/3!
  const float sx = x + s;
  s = x + fmaf(dx, 1.f + c, s);
  c = 1.f + fmaf(-dx, sx, c);
  const float a = q & 1 ? s : c, b = q & 1 ? c : s;
  // quarter turns: (c, s), (-s, c), (-c, -s), (s, -c)
  return make_float2(__uint_as_float(__float_as_uint(a) ^ (((q + 1) & 2) << 30)),
                     __uint_as_float(__float_as_uint(b) ^ ((q & 2) << 30)));
}

// mscale * cosines and sines of NT tokens into shared memory, [token][D/2]
// each; pairs past rot_dim/2 turn by nothing.  pos(i, p) puts token i's
// position into p, or returns false: its angles are not needed.  The
// positions are all read before any is used.
template <int D, int NT, int THREADS, typename PosFn>
__device__ __forceinline__ void fill_angles(const RopeParams &r, float *s_cos, float *s_sin, PosFn pos) {
  constexpr int kPer = THREADS / (D / 2), kIt = (NT + kPer - 1) / kPer;  // tokens at once, rounds
  static_assert(THREADS % (D / 2) == 0, "a thread keeps to one pair");
  const int pair = threadIdx.x % (D / 2), first = threadIdx.x / (D / 2);
  int64_t p[kIt];
  bool need[kIt];
#pragma unroll
  for (int k = 0; k < kIt; ++k) {
    p[k] = 0;
    need[k] = first + k * kPer < NT && pos(first + k * kPer, p[k]);
  }
  const bool turns = pair < (r.rot_dim >> 1);
  const float freq = turns ? r.inv_freq[pair] : 0.f;
  const uint64_t rate = turn_rate(freq);
  const float ms = turns ? r.mscale + (freq - freq) : 1.f;  // NaN where the frequency is not finite
#pragma unroll
  for (int k = 0; k < kIt; ++k) {
    if (!need[k]) continue;
    const float2 cs = cos_sin(p[k], rate);
    s_cos[threadIdx.x + k * THREADS] = cs.x * ms;  // pair's column of token first + k * kPer
    s_sin[threadIdx.x + k * THREADS] = cs.y * ms;
  }
}

// Whether the lane's channels turn: all eight or none (rot_dim is a multiple
// of 16), and those that do not keep their bits.  PART: not every lane does
// (asked of every call, the check costs 4096 tokens x 40 heads 1.4 of 14.5 us).
template <bool PART>
__device__ __forceinline__ bool lane_turns(const RopeParams &r, int sl) {
  return !PART || sl < r.rot_dim >> 3;
}

// Sum over the LPR lanes of a vector.
template <int LPR>
__device__ __forceinline__ float vec_sum(float v) {
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// The lane's part of a vector's sum of squares.
__device__ __forceinline__ float squares8(const float (&x)[8]) {
  float2 s = fmul2(make_float2(x[0], x[1]), make_float2(x[0], x[1]));
#pragma unroll
  for (int i = 1; i < 4; ++i)
    s = ffma2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(x[2 * i], x[2 * i + 1]), s);
  return s.x + s.y;
}

// 1 / root of the mean of D squares of sum ss, plus eps.
template <int D>
__device__ __forceinline__ float inv_rms(float ss, float eps) {
  // one Newton step behind the approximate root, so that a result's rounding
  // does not depend on it (the correctly rounded root costs 5% of the append)
  const float var = ss * (1.f / D) + eps;
  float inv = rsqrtf(var);
  const float err = fmaf(-var * inv, inv, 1.f);
  return fabsf(err) < 0.5f ? fmaf(0.5f * inv, err, inv) : inv;  // not for 0 and infinity
}

// (The weight first: a bf16 value's product with a bf16 weight is exact.)
__device__ __forceinline__ void scale8(float inv, const float (&w)[8], float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 y = fmul2(fmul2(make_float2(x[2 * i], x[2 * i + 1]), make_float2(w[2 * i], w[2 * i + 1])),
                           make_float2(inv, inv));
    x[2 * i] = y.x, x[2 * i + 1] = y.y;
  }
}

// Norm of one vector with the lane's weights w.
template <int D>
__device__ __forceinline__ void norm8(float eps, const float (&w)[8], float (&x)[8]) {
  scale8(inv_rms<D>(vec_sum<D / 8>(squares8(x)), eps), w, x);
}

// Norms of two vectors: even lanes sum the first's squares and odd lanes the
// second's, so that the pair takes one sum's steps and one root.  (Each sum is
// the tree that norm8 adds up: the results have the same bits.)
template <int D>
__device__ __forceinline__ void norm8(float eps, const float (&w)[8], float (&x)[8], float (&y)[8]) {
  const bool odd = threadIdx.x & 1;
  const float sx = squares8(x), sy = squares8(y);
  float ss = (odd ? sy : sx) + __shfl_xor_sync(0xffffffffu, odd ? sx : sy, 1);
#pragma unroll
  for (int o = 2; o < D / 8; o <<= 1) ss += __shfl_xor_sync(0xffffffffu, ss, o);
  const float inv = inv_rms<D>(ss, eps);
  const int even = threadIdx.x & 30;
  scale8(__shfl_sync(0xffffffffu, inv, even), w, x);
  scale8(__shfl_sync(0xffffffffu, inv, even + 1), w, y);
}

// Rotation of the lane's four pairs, two at a time.
template <bool IL>
__device__ __forceinline__ void rotate8(const float4 &c, const float4 &s, float (&x)[8]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float2 cc = i ? make_float2(c.z, c.w) : make_float2(c.x, c.y);
    const float2 sn = i ? make_float2(s.z, s.w) : make_float2(s.x, s.y);
    float &a0 = x[IL ? 4 * i : 2 * i], &a1 = x[IL ? 4 * i + 2 : 2 * i + 1];
    float &b0 = x[IL ? 4 * i + 1 : 4 + 2 * i], &b1 = x[IL ? 4 * i + 3 : 5 + 2 * i];
    const float2 a = make_float2(a0, a1), b = make_float2(b0, b1);
    const float2 na = ffma2(a, cc, fmul2(b, make_float2(-sn.x, -sn.y)));
    const float2 nb = ffma2(b, cc, fmul2(a, sn));
    a0 = na.x, a1 = na.y, b0 = nb.x, b1 = nb.y;
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

// Codes 256 .. 448 at the largest exponent would stand for 2^128 and more,
// which neither fp32 nor bf16 holds: there values past code 240's take that
// code (bf16's largest is off by 6%, not infinite when it is read).  A NaN
// compares false and stays.
constexpr int kTopExp = 120;
__device__ __forceinline__ void cap_top(float (&x)[8]) {
  constexpr float kTop = 240.f * 1.329227995784916e36f;  // 240 * 2^120
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (fabsf(x[j]) > kTop) x[j] = copysignf(kTop, x[j]);
}

__device__ __forceinline__ float pow2i(int e) { return __int_as_float((127 + e) << 23); }

// Four codes of x * inv, first in the low byte.
__device__ __forceinline__ uint32_t e4m3x4(const float *x, float inv) {
  uint16_t lo, hi;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x[1] * inv), "f"(x[0] * inv));
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x[3] * inv), "f"(x[2] * inv));
  return lo | (uint32_t)hi << 16;
}

__device__ __forceinline__ float finite_abs(float x) {
  const float a = fabsf(x);
  return a < INFINITY ? a : 0.f;  // infinities and NaN do not set the scale
}

// Eight bytes into shared memory, or zeros (bytes 0: nothing is read).
__device__ __forceinline__ void cp_async8(void *to, const void *from, int bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"((uint32_t)__cvta_generic_to_shared(to)),
               "l"(from), "r"(bytes)
               : "memory");
}

// One scale-block CTA: launch row r, K or V (isv), heads [h0, h1), item `item`
// (see the launch).  A half-warp takes NB neighbouring tokens.
template <bool IL, bool PART>
__device__ __forceinline__ void block_cta(const RopeRowsParams &P, int r, bool isv, int h0, int h1,
                                          int item, float *s_cos, float *s_sin) {
  using bf = __nv_bfloat16;
  constexpr int D = 128;
  constexpr int NB = kScaleBlock / (kBlockThreads / 16);  // tokens of a half-warp
  __shared__ float s_max[2][kBlockThreads / 32];
  // heads on their way, each thread's own quads
  __shared__ __align__(16) uint2 s_ring[kRing][NB][2][kBlockThreads];
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
  if (item >= (int)max((int64_t)1, done - fb)) return;
  const bool turn = !isv && P.rope.rot_dim > 0, turn_mine = turn && lane_turns<PART>(P.rope, sl);
  const bool norm = !isv && P.rope.k_norm != nullptr;
  const Quads qd = quads_of(P.rope, sl);
  float w[8];
  if (norm) {
    load_quad(static_cast<const bf *>(P.rope.k_norm) + qd.a, w);
    load_quad(static_cast<const bf *>(P.rope.k_norm) + qd.b, w + 4);
  }
  const HeadView &in = isv ? P.v : P.k;
  bf *tails = reinterpret_cast<bf *>(isv ? P.tail.v : P.tail.k);
  uint8_t *codes = isv ? a.p.ret_v : a.p.ret_k;
  float *scales = reinterpret_cast<float *>(isv ? a.p.ret_v_sz : a.p.ret_k_sz);
  int buf = 0;
  // Item 0 also writes the block that stays open, after the first block's
  // older tokens have been read from the same tail rows.
  for (int part = 0; part < 2; ++part) {
    const int64_t blk = part == 0 ? fb + item : done;
    const bool full = part == 0;
    if (part == 0 && blk >= done) continue;
    if (part == 1 && (item != 0 || !open)) break;
    const int64_t first = blk << kScaleShift;  // local row of the block's first token
    const int64_t t0 = first + a.shard_lo - len;  // its token of the call (negative: older)
    const int64_t tok0 = (int64_t)r * a.n_tok + t0;
    const bf *src = static_cast<const bf *>(in.p) + (tok0 + hw * NB) * in.tok;
    bool fresh[NB];
#pragma unroll
    for (int i = 0; i < NB; ++i) {
      const int64_t l = first + hw * NB + i;
      fresh[i] = l >= l0 && l < l1;
    }
    // head h into its slot: the input's tokens, older ones from the tail,
    // zeros where the open block has neither
    auto fetch = [&](int h) {
      if (h < h1) {
        const bf *in_h = src + (int64_t)a.h.ret_heads[h] * in.head;
        const bf *tail = tails + (((int64_t)b * a.n_ret + h) * kScaleBlock + hw * NB) * D;
        const int slot = (h - h0) % kRing;
#pragma unroll
        for (int i = 0; i < NB; ++i) {
          const bf *from = fresh[i] ? in_h + i * in.tok : tail + i * D;
          const int bytes = fresh[i] || full ? 8 : 0;
          cp_async8(&s_ring[slot][i][0][tid], from + qd.a, bytes);
          cp_async8(&s_ring[slot][i][1][tid], from + qd.b, bytes);
        }
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
#pragma unroll
    for (int i = 0; i < kRing; ++i) fetch(h0 + i);
    // (a table entry is read once for all heads; an open block's is not needed)
    const int64_t row0 = full ? ret_row(a.ret, b, 0, first) : 0;
    const int64_t head_step = a.ret.table ? kPageTokens : a.ret.cap;
    if (part == 1) __syncthreads();  // angles and tail of part 0 are no longer read
    if (turn)
      fill_angles<D, kScaleBlock, kBlockThreads>(P.rope, s_cos, s_sin, [&](int i, int64_t &p) {
        const int64_t t = t0 + i;
        if (t < 0 || t >= a.n_tok) return false;  // not the call's
        p = P.positions ? P.positions[tok0 + i] : len + t;
        return true;
      });
    __syncthreads();
    for (int h = h0; h < h1; ++h) {
      float mx = 0.f;
      Raw<bf> z[NB];  // finished: rounded to bf16, what rotated keys are everywhere else
      asm volatile("cp.async.wait_group %0;" ::"n"(kRing - 1) : "memory");
      const int slot = (h - h0) % kRing;
#pragma unroll
      for (int i = 0; i < NB; ++i) z[i].a = s_ring[slot][i][0][tid], z[i].b = s_ring[slot][i][1][tid];
#pragma unroll
      for (int i = 0; i < NB; i += 2) {
        float x[2][8];
        z[i].unpack(x[0]);
        z[i + 1].unpack(x[1]);
        if (norm) norm8<D>(P.rope.eps, w, x[0], x[1]);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (turn_mine) {
            const int at = (hw * NB + i + k) * (D / 2) + 4 * sl;
            const float4 c = *reinterpret_cast<const float4 *>(s_cos + at);
            const float4 s = *reinterpret_cast<const float4 *>(s_sin + at);
            rotate8<IL>(c, s, x[k]);
          }
          if (fresh[i + k]) z[i + k].pack(x[k]);
          z[i + k].unpack(x[k]);
#pragma unroll
          for (int j = 0; j < 8; ++j) mx = fmaxf(mx, finite_abs(x[k][j]));
        }
      }
      if (!full) {
        bf *tail = tails + (((int64_t)b * a.n_ret + h) * kScaleBlock + hw * NB) * D;
#pragma unroll
        for (int i = 0; i < NB; ++i)
          if (fresh[i]) z[i].store(tail + i * D, qd.a, qd.b);
        fetch(h + kRing);
        continue;
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
      // two sets of slots in turn: one barrier a head
      if ((tid & 31) == 0) s_max[buf][warp] = mx;
      __syncthreads();
      fetch(h + kRing);  // (the slot's values have been used)
#pragma unroll
      for (int i = 0; i < kBlockThreads / 32; ++i) mx = fmaxf(mx, s_max[buf][i]);
      buf ^= 1;
      const int e = scale_exp(mx);
      const float inv = pow2i(-e);
      const int64_t row = row0 + h * head_step;
#pragma unroll
      for (int i = 0; i < NB; ++i) {
        float x[8];
        z[i].unpack(x);
        if (e == kTopExp) cap_top(x);
        uint8_t *at = codes + (row + hw * NB + i) * D;
        *reinterpret_cast<uint32_t *>(at + qd.a) = e4m3x4(x, inv);
        *reinterpret_cast<uint32_t *>(at + qd.b) = e4m3x4(x + 4, inv);
      }
      if (tid == 0) scales[row >> kScaleShift] = pow2i(e);
    }
  }
}

// ------------------------------------------------------------ vectors

// 4-bit codes of a vector, this lane's quads (a, b): the arithmetic of the
// 4-bit append (quant_int4.cuh), the extremes over D/8 lanes.
template <int D>
__device__ __forceinline__ void quantise8(const float (&x)[8], uint32_t *qa, uint32_t *qb, __half2 *sz) {
  float mn = x[0], mx = x[0];
#pragma unroll
  for (int j = 1; j < 8; ++j) {
    mn = fminf(mn, x[j]);
    mx = fmaxf(mx, x[j]);
  }
#pragma unroll
  for (int o = 1; o < D / 8; o <<= 1) {
    mn = fminf(mn, __shfl_xor_sync(0xffffffffu, mn, o));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
  }
  const __half sch = __float2half_rn(__fdiv_rn(__fsub_rn(mx, mn), 15.0f));
  const __half zph = __float2half_rn(mn);
  const float scf = __half2float(sch), zpf = __half2float(zph);
  uint32_t u[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    float q = 0.0f;
    if (scf != 0.0f) q = fminf(15.0f, fmaxf(0.0f, rintf(__fdiv_rn(__fsub_rn(x[j], zpf), scf))));
    u[j >> 2] |= (uint32_t)q << (4 * (j & 3));
  }
  *qa = u[0];
  *qb = u[1];
  sz->x = sch;
  sz->y = zph;
}

// Row CTAs: kTok tokens x vecs_per_cta of their head vectors: the Hq queries
// (when given), then the K heads and, for an append, the V heads; 8-bit
// caches may list their streaming heads only, and no list holds streaming heads
// when none of the CTA's tokens survives in their windows.  A group of D/8
// lanes keeps to one token; every group of a warp is at the same vector of its
// own token.
template <typename T, int D, int MODE, bool IL, bool PART>
__global__ void __launch_bounds__(threads_of(MODE), ctas_of(MODE, sizeof(T)))
    rope_rows_kernel(const __grid_constant__ RopeRowsParams P, int block_ctas, int vecs_per_cta) {
  constexpr int THREADS = threads_of(MODE);
  constexpr int LPR = D / 8, GROUPS = THREADS / LPR, SUB = GROUPS / kTok;
  // the 8-bit mode's scale-block CTAs hold 32 tokens' angles
  constexpr int NT = MODE == kFp8Mode ? kScaleBlock : kTok;
  __shared__ __align__(16) float s_cos[NT * (D / 2)], s_sin[NT * (D / 2)];
  const AppendParams &a = P.a;
  if constexpr (MODE == kFp8Mode) {
    if ((int)blockIdx.x < block_ctas) {
      const int groups = (a.n_ret + P.heads_per_cta - 1) / P.heads_per_cta;
      int y = blockIdx.x;
      const bool isv = y & 1;
      y >>= 1;
      const int item = y % P.block_items;
      y /= P.block_items;
      const int h0 = (y % groups) * P.heads_per_cta;
      block_cta<IL, PART>(P, y / groups, isv, h0, min(a.n_ret, h0 + P.heads_per_cta), item, s_cos, s_sin);
      return;
    }
  }
  // 8-bit: retrieval heads are listed when no row completes a block; their
  // tokens then go to the tails (else the scale-block CTAs take them)
  const bool tails = MODE == kFp8Mode && P.tails_in_rows;
  const int nq = P.q.p ? P.Hq : 0;
  const int nk_all = MODE == kFp8Mode && !tails ? a.n_str : P.Hkv;
  const int vgroups = (nq + (MODE == kAlone ? 1 : 2) * nk_all + vecs_per_cta - 1) / vecs_per_cta;
  const int cta = (int)blockIdx.x - block_ctas;
  const int64_t tok0 = (int64_t)(vgroups == 1 ? cta : cta / vgroups) * kTok;
  const int group = threadIdx.x / LPR, sl = threadIdx.x % LPR;
  const int sub = group / kTok;
  const bool alive = tok0 + group % kTok < P.tokens;
  const int64_t tok = alive ? tok0 + group % kTok : P.tokens - 1;
  const Quads qd = quads_of(P.rope, sl);
  // launch row of a token (a 64-bit division only where it is needed)
  auto row_of = [&](int64_t tk) {
    if (a.rows.n == 1) return 0;
    return P.tokens >> 32 ? (int)(tk / a.n_tok) : (int)((uint32_t)tk / (uint32_t)a.n_tok);
  };
  // which heads keep the token
  bool kept_ret = true, kept_str = true, all_kv = true;
  int nk = nk_all;
  if constexpr (MODE != kAlone) {
    const int lr = row_of(tok);
    const int b = a.rows.row[lr];
    const int64_t len = a.rows.len[lr];
    const int64_t p = len + (tok - (int64_t)lr * a.n_tok);
    kept_ret = (MODE != kFp8Mode || tails) && a.n_ret > 0 && p >= a.shard_lo && p < a.shard_hi;
    kept_str = a.n_str > 0 && (p < a.S || p >= len + a.n_tok - a.R);
    // (a long chunk's middle: retrieval heads only)
    all_kv = __syncthreads_or(alive && kept_str);
    if (!all_kv) nk = MODE == kFp8Mode && !tails ? 0 : a.n_ret;
  }
  const int vecs = nq + (MODE == kAlone ? nk : 2 * nk);
  const int v0 = (vgroups == 1 ? 0 : cta % vgroups) * vecs_per_cta, v1 = min(vecs, v0 + vecs_per_cta);
  if (v0 >= v1) return;  // the same in the whole CTA
  auto head_of = [&](int h) {
    if (MODE == kAlone) return h;
    if (MODE == kFp8Mode && !tails) return (int)a.h.str_heads[h];
    return all_kv ? h : (int)a.h.ret_heads[h];
  };
  const bool turn = P.rope.rot_dim > 0 && v0 < nq + nk, turn_mine = turn && lane_turns<PART>(P.rope, sl);
  float4 c = make_float4(1.f, 1.f, 1.f, 1.f), s = make_float4(0.f, 0.f, 0.f, 0.f);
  if (turn) {
    fill_angles<D, kTok, THREADS>(P.rope, s_cos, s_sin, [&](int i, int64_t &p) {
      const int64_t tk = tok0 + i;
      if (tk >= P.tokens) return false;
      if (MODE == kAlone || P.positions) {
        p = P.positions[tk];
      } else {
        const int lr = row_of(tk);
        p = (int64_t)a.rows.len[lr] + (tk - (int64_t)lr * a.n_tok);
      }
      return true;
    });
    __syncthreads();
    c = *reinterpret_cast<const float4 *>(s_cos + (group % kTok) * (D / 2) + 4 * sl);
    s = *reinterpret_cast<const float4 *>(s_sin + (group % kTok) * (D / 2) + 4 * sl);
  }
  // The vectors of one kind, [first, first + count) of the token's list, that
  // this CTA takes: norm weights wp or null; each finished vector goes to
  // put(vector of the kind, values, wanted).  Whole batches are loaded before
  // any of them is used; what is left goes one by one.
  auto walk = [&](int first, int count, const HeadView &view, bool kv, const void *wp, bool rotated, auto put) {
    const int lo = max(v0, first) - first, hi = min(v1, first + count) - first;
    if (lo >= hi) return;
    float w[8];
    if (wp) {
      load_quad(static_cast<const T *>(wp) + qd.a, w);
      load_quad(static_cast<const T *>(wp) + qd.b, w + 4);
    }
    const T *in = static_cast<const T *>(view.p) + tok * view.tok;
    auto fetch = [&](Raw<T> &raw, int v) {
      if (MODE != kAlone && kv) {
        const int h = head_of(v);
        const bool live = alive && (a.h.kind[h] ? kept_ret : kept_str);
        raw = Raw<T>{};
        if (live) raw.load(in + (int64_t)h * view.head, qd.a, qd.b);
        return live;
      }
      raw.load(in + (int64_t)v * view.head, qd.a, qd.b);
      return alive;
    };
    auto finish = [&](float (&x)[8], int v, bool ok) {
      if (rotated) rotate8<IL>(c, s, x);
      put(v, x, ok);
    };
    int v = lo + sub;  // the same in the whole warp
    for (; v + (kBatch - 1) * SUB < hi; v += kBatch * SUB) {
      Raw<T> raw[kBatch];
      bool ok[kBatch];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) ok[i] = fetch(raw[i], v + i * SUB);
#pragma unroll
      for (int i = 0; i < kBatch; i += 2) {
        // two norms at once where the registers allow (4096 tokens x 40 heads:
        // 14.4 us, 15.6 one by one; the other appends: 48.4 against 43.5)
        float x[8], y[8];
        raw[i].unpack(x);
        if constexpr (MODE == kAlone || MODE == kFp8Mode) {
          raw[i + 1].unpack(y);
          if (wp) norm8<D>(P.rope.eps, w, x, y);
          finish(x, v + i * SUB, ok[i]);
        } else {
          if (wp) norm8<D>(P.rope.eps, w, x);
          finish(x, v + i * SUB, ok[i]);
          raw[i + 1].unpack(y);
          if (wp) norm8<D>(P.rope.eps, w, y);
        }
        finish(y, v + (i + 1) * SUB, ok[i + 1]);
      }
    }
    for (; v < hi; v += SUB) {
      Raw<T> raw;
      const bool ok = fetch(raw, v);
      float x[8];
      raw.unpack(x);
      if (wp) norm8<D>(P.rope.eps, w, x);
      finish(x, v, ok);
    }
  };
  auto write = [&](T *dst, const float (&x)[8]) {
    store_quad(dst + qd.a, x);
    store_quad(dst + qd.b, x + 4);
  };
  walk(0, nq, P.q, false, P.rope.q_norm, turn_mine, [&](int v, float (&x)[8], bool ok) {
    if (ok) write(static_cast<T *>(P.q_out) + (tok * P.Hq + v) * D, x);
  });
  // where the token goes in the cache: rows of its heads, one stride apart
  // (behind the queries: registers)
  int64_t ret0 = 0, ret_step = 0, str0 = 0;
  if constexpr (MODE != kAlone) {
    const int lr = row_of(tok);
    const int b = a.rows.row[lr];
    const int64_t p = (int64_t)a.rows.len[lr] + (tok - (int64_t)lr * a.n_tok);
    if (kept_ret && MODE == kFp8Mode) {
      ret0 = (int64_t)b * a.n_ret * kScaleBlock + ((p - a.shard_lo) & (kScaleBlock - 1));
      ret_step = kScaleBlock;
    } else if (kept_ret) {
      ret0 = ret_row(a.ret, b, 0, p - a.shard_lo);
      ret_step = a.ret.table ? kPageTokens : a.ret.cap;
    }
    if (kept_str) {  // (positions and windows fit 31 bits)
      const uint32_t past = (uint32_t)p - (uint32_t)a.S;
      str0 = (int64_t)b * a.n_str * a.Ws + (p < a.S ? (uint32_t)p : (uint32_t)a.S + past % (uint32_t)a.R);
    }
  }
  // cache rows of K or V heads
  auto put_kv = [&](bool isv, int h, float (&x)[8], bool ok) {
    const int kvh = head_of(h);
    const bool ret = a.h.kind[kvh];
    const int64_t row = ret ? ret0 + a.h.index[kvh] * ret_step : str0 + (int64_t)a.h.index[kvh] * a.Ws;
    uint8_t *base = !ret               ? (isv ? a.p.str_v : a.p.str_k)
                    : MODE == kFp8Mode ? (isv ? P.tail.v : P.tail.k)
                                       : (isv ? a.p.ret_v : a.p.ret_k);
    if constexpr (MODE == kInt4) {
      uint8_t *szs = ret ? (isv ? a.p.ret_v_sz : a.p.ret_k_sz) : (isv ? a.p.str_v_sz : a.p.str_k_sz);
      // rounded to bf16 first, so that the codes are those of appending the
      // rotated keys
      uint32_t ua, ub;
      __half2 sz;
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = __bfloat162float(__float2bfloat16_rn(x[j]));
      quantise8<D>(x, &ua, &ub, &sz);
      if (!ok) return;
      uint8_t *at = base + row * (D / 2);
      *reinterpret_cast<uint16_t *>(at + qd.a / 2) = (uint16_t)ua;
      *reinterpret_cast<uint16_t *>(at + qd.b / 2) = (uint16_t)ub;
      if (sl == 0) reinterpret_cast<__half2 *>(szs)[row] = sz;
    } else {
      if (ok) write(reinterpret_cast<T *>(base) + row * D, x);
    }
  };
  walk(nq, nk, P.k, true, P.rope.k_norm, turn_mine, [&](int v, float (&x)[8], bool ok) {
    if constexpr (MODE == kAlone) {
      if (ok) write(static_cast<T *>(P.k_out) + (tok * P.Hkv + v) * D, x);
    } else {
      put_kv(false, v, x, ok);
    }
  });
  if constexpr (MODE != kAlone)
    walk(nq + nk, nk, P.v, true, nullptr, false,
         [&](int v, float (&x)[8], bool ok) { put_kv(true, v, x, ok); });
}

template <typename T, int D, int MODE>
cudaError_t run(const RopeRowsParams &P, int64_t block_ctas, cudaStream_t s) {
  constexpr int THREADS = threads_of(MODE), SUB = THREADS / (D / 8) / kTok;
  const int nq = P.q.p ? P.Hq : 0;
  const int nk = MODE == kFp8Mode && !P.tails_in_rows ? P.a.n_str : P.Hkv;
  const int64_t vecs = nq + (MODE == kAlone ? nk : 2 * nk);
  // A CTA takes all its tokens' vectors when there are tokens enough for
  // every SM, so that the set-up is paid once (8192 tokens of 40 heads in two
  // halves: 35.6 against 31.3 us); else fewer, down to what its lane groups
  // hold at once.  Equal shares: 1500 tokens 8.8 us as 20 + 20, 10.4 as 32 + 8.
  const int64_t tiles = (P.tokens + kTok - 1) / kTok;
  int64_t per = SUB;
  while (per < vecs && tiles * ((vecs + 2 * per - 1) / (2 * per)) >= 148 * 4) per *= 2;
  const int64_t shares = (vecs + per - 1) / per;
  if (shares > 0) per = ((vecs + shares - 1) / shares + SUB - 1) / SUB * SUB;
  const int64_t ctas = tiles * shares;
  if (block_ctas + ctas == 0) return cudaSuccess;
  if (block_ctas + ctas > 0x7fffffff) return cudaErrorInvalidValue;
  const unsigned grid = (unsigned)(block_ctas + ctas);
  const bool part = P.rope.rot_dim < D;
  const auto kernel = P.rope.interleaved ? (part ? rope_rows_kernel<T, D, MODE, true, true> : rope_rows_kernel<T, D, MODE, true, false>)
                                         : (part ? rope_rows_kernel<T, D, MODE, false, true> : rope_rows_kernel<T, D, MODE, false, false>);
  kernel<<<grid, THREADS, 0, s>>>(P, (int)block_ctas, (int)per);
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
  // 8-bit: per launch row one item per block that becomes full (at least one,
  // for the tail), times groups of retrieval heads, K and V apart.  A call
  // that completes no block, such as most decode steps, leaves the tails to
  // the row CTAs (64 rows x 1 token: 7.7 us with scale-block CTAs, 5.5 so).
  int64_t items = 0, full = 0;
  for (int r = 0; r < a.rows.n; ++r) {
    const int64_t len = a.rows.len[r];
    const int64_t l0 = std::max<int64_t>(0, std::min<int64_t>(len, a.shard_hi) - a.shard_lo);
    const int64_t l1 = std::max<int64_t>(0, std::min<int64_t>(len + a.n_tok, a.shard_hi) - a.shard_lo);
    const int64_t blocks = (l1 >> kScaleShift) - (l0 >> kScaleShift);
    full = std::max(full, blocks);
    if (l1 > l0) items = std::max(items, std::max<int64_t>(1, blocks));
  }
  P.tails_in_rows = full == 0;
  int64_t ctas = 0;
  P.block_items = (int)std::max<int64_t>(1, items);
  P.heads_per_cta = 1;
  if (full > 0 && a.n_ret > 0) {
    // A CTA's heads share its tokens' angles: as many as leave two CTAs an SM
    // (8192 tokens, 4 heads, with the queries: 48.5, 44.4 and 42.4 us for 1, 2
    // and 4 heads a CTA).
    while (P.heads_per_cta < a.n_ret &&
           2 * a.rows.n * items * ((a.n_ret + 2 * P.heads_per_cta - 1) / (2 * P.heads_per_cta)) >= 148 * 2)
      P.heads_per_cta *= 2;
    ctas = 2 * a.rows.n * items * ((a.n_ret + P.heads_per_cta - 1) / P.heads_per_cta);
  }
  return ra::run<bf, 128, ra::kFp8Mode>(P, ctas, s);
}

}  // namespace duo
