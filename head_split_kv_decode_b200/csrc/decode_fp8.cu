// Single-token decode attention over an 8-bit cache (head_dim 128): e4m3
// codes with one float32 scale per 32 tokens and KV head for retrieval heads,
// their newest, unfinished block and the streaming heads in bf16.
//
// Work split as in the bf16 tensor-core decode: split-K over retrieval pages
// (a share of the tail of each head's tiles claimed at run time, the last
// split of a head merges the partials), streaming slot buffers one per CTA or
// several per CTA on groups of warps.  Per warp and 32 keys (one scale block;
// 4 KB of K and 4 KB of V):
//   S^T[16 x 8] = K[16 x 128] . Q^T    per 16 keys, 8 k-steps
//   U[16 x 8]   = V^T[16 x 32] . P^T   per 16 channels, then O^T += scale_v * U
// with mma.sync m16n8k16 on f16 operands, fp32 accumulators.  An e4m3 code is
// an f16 value exactly, so the products see the codes as they are: K's scale
// multiplies the scores and V's multiplies U, each one number per tile, both
// in fp32.  Scores are computed transposed so that the codes fill the whole A
// operand; the same dot product in any channel order is the same sum, so each
// thread's K operand is 16 consecutive bytes of its key row (four k-steps)
// and its V operand 16 consecutive channels of its keys.  Queries enter as
// f16 too, scaled by a power of two per query so that the largest |q| lies in
// [2^14, 2^15): what f16's range cuts off is below 2^-38 of it.
// Probabilities are formed and summed in fp32 and meet V as two f16 numbers,
// the rounded value and what it lost (22 bits together; one f16 would be off by
// 2^-11 of each and the outputs by up to 1e-3), relative to m - 7: with the lazy
// rescale (m follows the running maximum when it grows by more than 2^8)
// p <= 2^15 stays in range, and f16's smallest step is 2^-31 of the largest.
// Of the product's eight columns G <= 4 queries leave the upper four idle:
// they repeat the queries and carry the remainders, at no further product; for
// more queries a second product takes them.  (One f16 against two, us: 128K
// GQA 26.8 and 27.1, 1M 83.2 and 83.4, 300 tokens 6.4 and 6.7, 64K with eight
// queries a head 20.0 to 21.4 and 20.7 to 21.0.)
// O takes U relative to m itself, so that values keep fp32's range (up to
// 2^119 over the number of keys of a split, as in the bf16 decode).
// bf16 rows (tail, streaming) use the same layout with bf16 operands, 16 keys
// at a time; there p is two bf16 numbers (16 bits).
//
// Bound: HBM, 256 bytes and 8/32 of a scale pair per key.  Measured on one
// layer of 32/8 heads: 1M tokens, 2 retrieval heads: 83.4 us, 0.98 of the copy
// rate; 128K, 4 retrieval heads: 27.1 us, 0.76 (about 18.4 us of main loop at 7.4
// TB/s, the rest is the way to the first tile, the reduction and the merge).
// 128 registers a thread: each variant spills a few (36 to 60 bytes; G = 1, which
// computes one of a thread's two columns, 48).
// 32 keys a tile and single-buffered registers: 16 keys loaded a tile ahead
// spill more and double the per-tile work (33.0 us at 128K), and the 16 warps'
// loads, 128 KB an SM, leave no room for a prefetch to help (1M 86 us with).
//
// Pages: "DuoAttention: Efficient Long-Context LLM Inference with Retrieval and
// Streaming Heads" (hotpaper.ai), abstract and section "기술적 접근법".
#include "common.cuh"
#include "decode_finish.cuh"
#include "kv8.h"

namespace duo {
namespace d8 {

constexpr int D = 128;
constexpr int NWARPS = 16;
constexpr int T = kScaleBlock;      // keys per warp tile
constexpr float kHeadroom = 7.f;    // p is taken relative to m - kHeadroom,
constexpr float kUnscale = 1.f / 128.f;  // 2^-kHeadroom: O and l leave relative to m

__device__ __forceinline__ uint4 ldg128(const void *p) {
  uint4 v;
  asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "l"(p));
  return v;
}

__device__ __forceinline__ void prefetch_l2(const void *ptr, uint32_t bytes) {
  asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(ptr), "r"(bytes) : "memory");
}

// Two e4m3 codes (low byte first) as an f16 pair, exactly.
__device__ __forceinline__ uint32_t f16x2_lo(uint32_t w) {
  uint32_t d;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(d) : "r"(w));
  return d;
}
__device__ __forceinline__ uint32_t f16x2_hi(uint32_t w) {
  uint32_t d;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, h;}" : "=r"(d) : "r"(w));
  return d;
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
      "{%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8x8 matrix of 16-bit elements held as the warp's fragments.
__device__ __forceinline__ uint32_t movm_trans(uint32_t a) {
  uint32_t d;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
  return d;
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ uint32_t pack_f16(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&h);
}

__device__ __forceinline__ float exp2i(int e) { return __int_as_float((127 + e) << 23); }

template <int G>
__global__ void __launch_bounds__(NWARPS * 32, 1)
    decode_fp8_kernel(const __grid_constant__ DecodeFp8Params PP) {
  const DecodeParams &P = PP.d;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ int s_last;
  // Query fragments of each warp group's head, as [group][4][32 lanes][4
  // words]: f16 for the codes, bf16 for the bf16 rows; reloaded per tile
  // rather than held in registers.
  __shared__ __align__(16) uint32_t s_qh[4 * 32 * 4];
  __shared__ __align__(16) uint32_t s_qb[kMaxStrPack * 4 * 32 * 4];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 2, t = lane & 3;  // mma fragment coordinates
  // G <= 4: columns 4..7 repeat the queries 0..3 and carry what their
  // probabilities lose in rounding; else a second product does
  constexpr bool kFold = G <= 4;
  const bool rest = kFold && t >= 2;  // this thread's two columns are remainders
  constexpr int E = G == 1 ? 1 : 2;   // columns of a thread that can hold a query

  // ---- work item: retrieval CTAs first (launch row, head, split), then per
  // launch row the streaming CTAs of str_pack heads each
  const int n_ret_ctas = P.cta0[P.rows.n];
  auto str_group = [&](int &r_, int &pidx0_, int &wph_) {
    const int x = (int)blockIdx.x - n_ret_ctas;
    const int hp = max(P.str_pack, 1);
    const int per_row = (P.n_str + hp - 1) / hp;
    r_ = x / per_row;
    pidx0_ = (x % per_row) * hp;
    wph_ = NWARPS / hp;
  };
  int r, kvh, pidx, split, nsplit;
  int wph = NWARPS, wsub = warp;
  bool retrieval, idle = false;
  if ((int)blockIdx.x < n_ret_ctas) {
    int lo = 0, hi = P.rows.n;  // the last r with cta0[r] <= blockIdx.x
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (P.cta0[mid] <= (int)blockIdx.x) lo = mid; else hi = mid;
    }
    r = lo;
    nsplit = P.nsplit_r[r];
    const int local = (int)blockIdx.x - P.cta0[r];
    pidx = local / nsplit;
    split = local % nsplit;
    kvh = P.h.ret_heads[pidx];
    retrieval = true;
  } else {
    int pidx0;
    str_group(r, pidx0, wph);
    wsub = warp % wph;
    pidx = pidx0 + warp / wph;
    idle = pidx >= P.n_str;  // a group past the row's last head: no keys, no output
    if (idle) pidx = P.n_str - 1;
    kvh = P.h.str_heads[pidx];
    retrieval = false;
    split = 0;
    nsplit = 1;
  }
  const int b = P.rows.row[r];
  const int n = P.rows.len[r];
  // retrieval rows of this shard, or filled slots
  const int keys = retrieval ? (int)max((int64_t)0, min((int64_t)n, P.shard_hi) - P.shard_lo)
                             : (idle ? 0 : min(n, P.W));
  // Tiles of T keys, one scale block each (a block never crosses a page);
  // the keys past the last full block are in the tail.
  const int tiles = retrieval ? keys >> kScaleShift : 0;
  const bool split_head = retrieval && nsplit > 1;
  const bool pooled = split_head && P.pool;
  // fixed share of each split; with the pool the shares cover 13/16 of the
  // tiles and the rest is claimed one tile at a time
  const int ts = !retrieval    ? 0
                 : !split_head ? tiles
                 : pooled      ? (tiles - 3 * tiles / 16) / nsplit
                               : (tiles + nsplit - 1) / nsplit;
  const int t1 = min(tiles, (split + 1) * ts);
  const int tt0 = split * ts + warp;

  // storage row of a tile's first key
  auto tile_row = [&](int tt) { return ret_row(P.ret, b, pidx, (int64_t)tt * T); };
  // A tile's K and V into L2 (one lane).  A block-table entry may be read
  // here before the wait below; it only aims a prefetch, and is clamped to
  // the pool so the address stays valid.
  auto prefetch_tile = [&](int tt) {
    int64_t row;
    if (P.ret.table) {
      const int kb = tt * T;
      int64_t blk = P.ret.table[(int64_t)b * P.ret.stride + (kb >> kPageShift)];
      blk = blk < 0 ? 0 : (blk >= P.ret.blocks ? P.ret.blocks - 1 : blk);
      row = ((blk * P.n_ret + pidx) << kPageShift) + (kb & (kPageTokens - 1));
    } else {
      row = tile_row(tt);
    }
    prefetch_l2(P.p.ret_k + row * D, T * D);
    prefetch_l2(P.p.ret_v + row * D, T * D);
  };
  // Launched with programmatic dependent launch: this may run while the
  // previous kernel finishes.  Writes land in L2, so a line fetched now
  // cannot be stale when the loads after the wait use it.
  if (lane == 0) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      if (tt0 + i * NWARPS < t1) prefetch_tile(tt0 + i * NWARPS);
  }
  asm volatile("griddepcontrol.wait;" ::: "memory");

  // In partial mode a rank that does not own the streaming heads leaves
  // their rows empty (another shard contributes them).
  if (P.part_o && !retrieval && !P.own_str) {
    int r_, pidx0, wph_;
    str_group(r_, pidx0, wph_);
    for (int hs = 0; hs < NWARPS / wph_ && pidx0 + hs < P.n_str; ++hs) {
      const int64_t row0 = (int64_t)r * P.Hq + (int64_t)P.h.str_heads[pidx0 + hs] * G;
      for (int i = tid; i < G * D; i += NWARPS * 32) P.part_o[row0 * D + i] = 0.f;
      if (tid < G) P.part_lse[row0 + tid] = -INFINITY;
    }
    return;
  }

  // ---- query fragments: column g of Q^T is query g (zero past G)
  const uint32_t sqh = smem_u32(s_qh) + (uint32_t)lane * 16;
  const uint32_t sqb = smem_u32(s_qb) + (uint32_t)((warp / wph) * 128 + lane) * 16;
  float c1[2];  // score factor (log2 units) of queries 2t, 2t+1 on raw f16 sums
  const float sl2 = P.scale_log2;
  {
    const int gq = kFold ? g & 3 : g;
    const __nv_bfloat16 *qrow =
        reinterpret_cast<const __nv_bfloat16 *>(P.q) + ((int64_t)r * P.Hq + (int64_t)kvh * G + gq) * D;
    const bool live = gq < G;
    if (wsub == 0 || retrieval) {
      // bf16: 16-byte chunk 32c + 8t (c = 0..3), words = k-steps 2c (2), 2c+1 (2)
      if (wsub == 0) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const uint4 v = live ? ldg128(qrow + 32 * c + 8 * t) : make_uint4(0, 0, 0, 0);
          *reinterpret_cast<uint4 *>(&s_qb[((warp / wph) * 128 + c * 32 + lane) * 4]) = v;
        }
      }
      if (retrieval) {
        // f16: this thread's channels 64c + 16t .. +15 (c = 0, 1); every warp
        // needs the scale, warp 0 stores
        uint4 v[2][2];
        float amax = 0.f;
#pragma unroll
        for (int c = 0; c < 2; ++c)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            v[c][h] = live ? ldg128(qrow + 64 * c + 16 * t + 8 * h) : make_uint4(0, 0, 0, 0);
            const uint32_t w[4] = {v[c][h].x, v[c][h].y, v[c][h].z, v[c][h].w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              const float2 f = bf16x2_to_f2(w[j]);
              amax = fmaxf(amax, fmaxf(fabsf(f.x), fabsf(f.y)));
            }
          }
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
        amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
        const int ex = ((__float_as_int(amax) >> 23) & 0xff) - 127;
        const int sh = min(14 - ex, 126);
        const float qs = exp2i(sh), cq = sl2 * exp2i(-sh);
        c1[0] = __shfl_sync(0xffffffffu, cq, (2 * t) << 2);
        c1[1] = __shfl_sync(0xffffffffu, cq, (2 * t + 1) << 2);
        if (warp == 0) {
#pragma unroll
          for (int c = 0; c < 2; ++c)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t w[4] = {v[c][h].x, v[c][h].y, v[c][h].z, v[c][h].w};
              uint32_t o[4];
#pragma unroll
              for (int j = 0; j < 4; ++j) {
                const float2 f = bf16x2_to_f2(w[j]);
                o[j] = pack_f16(f.x * qs, f.y * qs);
              }
              *reinterpret_cast<uint4 *>(&s_qh[((2 * c + h) * 32 + lane) * 4]) =
                  make_uint4(o[0], o[1], o[2], o[3]);
            }
        }
      }
    }
    __syncthreads();
  }

  // O^T: tile mt holds channels 16g + 2mt (rows g) and + 1 (rows g+8) of
  // queries 2t and 2t+1; softmax state of those queries (m the same in the
  // eight threads of a column, l partial over this thread's keys)
  float o[8][4];
#pragma unroll
  for (int i = 0; i < 8; ++i) o[i][0] = o[i][1] = o[i][2] = o[i][3] = 0.f;
  float mq[2] = {-INFINITY, -INFINITY}, lq[2] = {0.f, 0.f};

  // Raise the running maxima to cover a tile whose own largest scores (this
  // thread's keys) are mx; needed only when some lane passes m + 8.
  auto raise = [&](float (&mx)[2]) {
    if (!__any_sync(0xffffffffu, mx[0] > mq[0] + 8.f || (E > 1 && mx[1] > mq[1] + 8.f))) return;
    float alpha[2];
#pragma unroll
    for (int e = 0; e < E; ++e) {
#pragma unroll
      for (int off = kFold ? 2 : 4; off < 32; off <<= 1)  // (2: a query and its remainder keep one m)
        mx[e] = fmaxf(mx[e], __shfl_xor_sync(0xffffffffu, mx[e], off));
      alpha[e] = 1.f;
      if (mx[e] > mq[e] + 8.f) {
        alpha[e] = mq[e] == -INFINITY ? 0.f : fast_exp2(mq[e] - mx[e]);
        mq[e] = mx[e];
      }
      lq[e] *= alpha[e];
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      o[i][0] *= alpha[0];
      o[i][2] *= alpha[0];
      if constexpr (E > 1) {
        o[i][1] *= alpha[1];
        o[i][3] *= alpha[1];
      }
    }
  };

  // ---- 16 bf16 keys [kb, kb + 16) below hi of rows K/V (256 bytes a row)
  auto tile_bf16 = [&](const uint8_t *Kx, const uint8_t *Vx, int kb, int hi) {
    constexpr int RB = D * 2;
    uint4 kr[2][4], vr[4][2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int key = kb + 8 * h + g;
#pragma unroll
      for (int c = 0; c < 4; ++c)
        kr[h][c] = key < hi ? ldg128(Kx + (int64_t)key * RB + (32 * c + 8 * t) * 2) : make_uint4(0, 0, 0, 0);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int key = kb + 2 * t + (i & 1) + 8 * (i >> 1);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        vr[i][h] = key < hi ? ldg128(Vx + (int64_t)key * RB + (16 * g + 8 * h) * 2) : make_uint4(0, 0, 0, 0);
    }
    float acc[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      const uint4 qf = lds128(sqb + 512u * c);
      mma_bf16(acc, kr[0][c].x, kr[1][c].x, kr[0][c].y, kr[1][c].y, qf.x, qf.y);
      mma_bf16(acc, kr[0][c].z, kr[1][c].z, kr[0][c].w, kr[1][c].w, qf.z, qf.w);
    }
    float sc[2][2], mx[2];
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int e = 0; e < 2; ++e)
        sc[h][e] = kb + 8 * h + g < hi ? acc[2 * h + e] * sl2 : -INFINITY;
    mx[0] = fmaxf(sc[0][0], sc[1][0]);
    mx[1] = fmaxf(sc[0][1], sc[1][1]);
    raise(mx);
    uint32_t pb[2], pr[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float p[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < E; ++e) {
        p[e] = sc[h][e] == -INFINITY ? 0.f : fast_exp2(sc[h][e] - mq[e]);
        lq[e] = fmaf(p[e], 1.f / kUnscale, lq[e]);
      }
      const uint32_t hi = pack_bf16(p[0], p[1]);
      const float2 f = bf16x2_to_f2(hi);
      const uint32_t lo = pack_bf16(p[0] - f.x, p[1] - f.y);
      pb[h] = movm_trans(rest ? lo : hi);
      if (!kFold) pr[h] = movm_trans(lo);
    }
#pragma unroll
    for (int mt = 0; mt < 8; ++mt) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = (&vr[i][mt >> 2].x)[mt & 3];
      const uint32_t a[4] = {__byte_perm(w[0], w[1], 0x5410u), __byte_perm(w[0], w[1], 0x7632u),
                             __byte_perm(w[2], w[3], 0x5410u), __byte_perm(w[2], w[3], 0x7632u)};
      mma_bf16(o[mt], a[0], a[1], a[2], a[3], pb[0], pb[1]);
      if (!kFold) mma_bf16(o[mt], a[0], a[1], a[2], a[3], pr[0], pr[1]);
    }
  };

  // ---- 32 coded keys, one scale block
  auto tile_fp8 = [&](int tt) {
    const int64_t row = tile_row(tt);
    const uint8_t *Kt = P.p.ret_k + row * D + g * D + 16 * t;
    const uint8_t *Vt = P.p.ret_v + row * D + 2 * t * D + 16 * g;
    const float ks = __ldg(reinterpret_cast<const float *>(P.p.ret_k_sz) + (row >> kScaleShift));
    const float vs = __ldg(reinterpret_cast<const float *>(P.p.ret_v_sz) + (row >> kScaleShift));
    uint4 kr[4][2], vr[2][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)  // key 8i + g, channels 64c + 16t ..
#pragma unroll
      for (int c = 0; c < 2; ++c) kr[i][c] = ldg128(Kt + 8 * i * D + 64 * c);
#pragma unroll
    for (int kg = 0; kg < 2; ++kg)
#pragma unroll
      for (int i = 0; i < 4; ++i)  // key 16kg + 2t + (i & 1) + 8 (i >> 1), channels 16g ..
        vr[kg][i] = ldg128(Vt + (16 * kg + (i & 1) + 8 * (i >> 1)) * D);
    // ---------------------------------------------------------- S^T = K Q^T
    float acc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
#pragma unroll
    for (int c = 0; c < 2; ++c)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const uint4 qf = lds128(sqh + 512u * (2 * c + h));  // k-steps of words 2h, 2h+1
#pragma unroll
        for (int kg = 0; kg < 2; ++kg) {
          const uint4 &ka = kr[2 * kg][c], &kb = kr[2 * kg + 1][c];
          const uint32_t a0 = h ? ka.z : ka.x, b0 = h ? kb.z : kb.x;
          const uint32_t a1 = h ? ka.w : ka.y, b1 = h ? kb.w : kb.y;
          mma_f16(acc[kg], f16x2_lo(a0), f16x2_lo(b0), f16x2_hi(a0), f16x2_hi(b0), qf.x, qf.y);
          mma_f16(acc[kg], f16x2_lo(a1), f16x2_lo(b1), f16x2_hi(a1), f16x2_hi(b1), qf.z, qf.w);
        }
      }
    // ------------------------------------------------------- online softmax
    const float f[2] = {ks * c1[0], ks * c1[1]};
    float mx[2] = {-INFINITY, -INFINITY};
#pragma unroll
    for (int kg = 0; kg < 2; ++kg)
#pragma unroll
      for (int i = 0; i < 4; i += 3 - E) {
        acc[kg][i] *= f[i & 1];
        mx[i & 1] = fmaxf(mx[i & 1], acc[kg][i]);
      }
    raise(mx);
    uint32_t pb[2][2], pr[2][2];
    const float ref[2] = {mq[0] - kHeadroom, mq[1] - kHeadroom};
#pragma unroll
    for (int kg = 0; kg < 2; ++kg)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float p0 = fast_exp2(acc[kg][2 * h] - ref[0]);
        const float p1 = E > 1 ? fast_exp2(acc[kg][2 * h + 1] - ref[1]) : 0.f;
        lq[0] += p0;
        if constexpr (E > 1) lq[1] += p1;
        const uint32_t hi = pack_f16(p0, p1);
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&hi));
        const uint32_t lo = pack_f16(p0 - f.x, p1 - f.y);
        pb[kg][h] = movm_trans(rest ? lo : hi);
        if (!kFold) pr[kg][h] = movm_trans(lo);
      }
    // ------------------------------------------- O^T += scale * (V^T P^T)
    const float vu = vs * kUnscale;
#pragma unroll
    for (int w = 0; w < 4; ++w)
#pragma unroll
      for (int hh = 0; hh < 2; ++hh) {
        float u[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int kg = 0; kg < 2; ++kg) {
          const uint32_t sel = hh ? 0x7362u : 0x5140u;
          // (channel 2mt: keys 2t, 2t+1) low, (channel 2mt + 1) high
          const uint32_t ab = __byte_perm((&vr[kg][0].x)[w], (&vr[kg][1].x)[w], sel);
          const uint32_t cd = __byte_perm((&vr[kg][2].x)[w], (&vr[kg][3].x)[w], sel);
          const uint32_t a[4] = {f16x2_lo(ab), f16x2_hi(ab), f16x2_lo(cd), f16x2_hi(cd)};
          mma_f16(u, a[0], a[1], a[2], a[3], pb[kg][0], pb[kg][1]);
          if (!kFold) mma_f16(u, a[0], a[1], a[2], a[3], pr[kg][0], pr[kg][1]);
        }
        float(&od)[4] = o[2 * w + hh];
#pragma unroll
        for (int i = 0; i < 4; i += 3 - E) od[i] = fmaf(vu, u[i], od[i]);
      }
  };

  // ---- the bf16 rows of this warp: a streaming window, or (last split of a
  // retrieval head, its last two warps) the head's unfinished block
  {
    const uint8_t *bk, *bv;
    int start, end, step;
    if (retrieval) {
      const int64_t off = ((int64_t)b * P.n_ret + pidx) * (kScaleBlock * D * 2);
      bk = PP.tail.k + off;
      bv = PP.tail.v + off;
      start = (NWARPS - 1 - warp) * 16;
      end = split == nsplit - 1 ? keys & (kScaleBlock - 1) : 0;
      step = NWARPS * 16;
    } else {
      const int64_t off = ((int64_t)b * P.n_str + pidx) * P.Ws * (int64_t)(D * 2);
      bk = P.p.str_k + off;
      bv = P.p.str_v + off;
      start = wsub * 16;
      end = keys;
      step = wph * 16;
    }
    for (int kb = start; kb < end; kb += step) tile_bf16(bk, bv, kb, end);
  }
  // ---- the coded tiles: this split's share, then the pool's
  if (retrieval) {
    unsigned *next = P.ws_next + ((int64_t)r * P.n_ret + pidx) * kChunkCounterStride;
    const int pool0 = pooled ? nsplit * ts : tiles;
    unsigned c = 0;
    int tt = tt0;
    if (pooled && tt >= t1 && lane == 0) c = atomicAdd(next, 1u);
    bool pool = false;
    for (;;) {
      if (!pool) {
        if (tt >= t1) {
          if (!pooled) break;
          pool = true;
          c = __shfl_sync(0xffffffffu, c, 0);
          tt = pool0 + (int)c;
          if (tt >= tiles) break;
          continue;
        }
        // the first claim is issued during the share's last tile
        if (pooled && tt + NWARPS >= t1 && lane == 0) c = atomicAdd(next, 1u);
        tile_fp8(tt);
        tt += NWARPS;
      } else {
        unsigned nx = 0;  // claim the following tile now; needed only after this one
        if (lane == 0) nx = atomicAdd(next, 1u);
        tile_fp8(tt);
        tt = pool0 + (int)__shfl_sync(0xffffffffu, nx, 0);
        if (tt >= tiles) break;
      }
    }
  }

  // the epilogue's parameter fields back into the uniform cache
  if (tid == 0) {
    const char *pp = reinterpret_cast<const char *>(&P);
    asm volatile("prefetchu.L1 [%0];" ::"l"(pp + offsetof(DecodeParams, out)));
    asm volatile("prefetchu.L1 [%0];" ::"l"(pp + offsetof(DecodeParams, part_o)));
    asm volatile("prefetchu.L1 [%0];" ::"l"(pp + offsetof(DecodeParams, ws_o)));
    asm volatile("prefetchu.L1 [%0];" ::"l"(pp + offsetof(DecodeParams, out_f32)));
  }
  asm volatile("griddepcontrol.launch_dependents;");

  // ---- per-warp state -> shared memory (queries < G only)
  float *red_m = reinterpret_cast<float *>(smem);
  float *red_l = red_m + NWARPS * G;
  float *red_o = red_l + NWARPS * G;
#pragma unroll
  for (int e = 0; e < E; ++e)
#pragma unroll
    for (int off = 4; off < 32; off <<= 1) lq[e] += __shfl_xor_sync(0xffffffffu, lq[e], off);
  if (g == 0) {
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (2 * t + e < G) {
        red_m[warp * G + 2 * t + e] = mq[e];
        red_l[warp * G + 2 * t + e] = lq[e] * kUnscale;
      }
  }
#pragma unroll
  for (int mt = 0; mt < 8; ++mt) {
    const int ch = 16 * g + 2 * mt;
#pragma unroll
    for (int e = 0; e < E; ++e)
      if constexpr (kFold) {
        // query and remainder meet: threads t < 2 finish the tile's even
        // channels, their partners t + 2 the odd ones
        const float got = __shfl_xor_sync(0xffffffffu, rest ? o[mt][e] : o[mt][2 + e], 2);
        const int q = (2 * t + e) & 3;
        if (q < G) red_o[(warp * G + q) * D + ch + rest] = (rest ? o[mt][2 + e] : o[mt][e]) + got;
      } else if (2 * t + e < G) {
        red_o[(warp * G + 2 * t + e) * D + ch] = o[mt][e];
        red_o[(warp * G + 2 * t + e) * D + ch + 1] = o[mt][2 + e];
      }
  }
  __syncthreads();
  if (!retrieval && P.str_pack > 1) {
    int r_, pidx0, wph_;
    str_group(r_, pidx0, wph_);
    decode_store_groups<__nv_bfloat16, D, G, NWARPS>(P, smem, wph_, r_, pidx0);
    return;
  }
  decode_reduce_store<__nv_bfloat16, D, G, NWARPS>(
      P, smem, &s_last, nsplit == 1, (int64_t)r * P.Hq + (int64_t)kvh * G, (int64_t)r * P.n_ret + pidx,
      (int64_t)(retrieval ? P.cta0[r] : 0) + (int64_t)pidx * nsplit, nsplit, split);
}

template <int G>
cudaError_t run(const DecodeFp8Params &p, cudaStream_t s, DecodeConfig *cfg) {
  auto kern = decode_fp8_kernel<G>;
  const DecodeParams &d = p.d;
  const int smem = (int)sizeof(float) * (NWARPS * G * D + 2 * NWARPS * G);
  static bool smem_done[kMaxDevices] = {};
  cudaError_t e = allow_dynamic_smem(kern, smem, smem_done);
  if (e != cudaSuccess) return e;
  if (cfg) {
    int occ = 0, dev = 0, sms = 0;
    if ((e = cudaOccupancyMaxActiveBlocksPerMultiprocessor(&occ, kern, NWARPS * 32, smem)) != cudaSuccess)
      return e;
    if ((e = cudaGetDevice(&dev)) != cudaSuccess) return e;
    if ((e = cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev)) != cudaSuccess) return e;
    cfg->tile_rows = decode_fp8_tile_rows();
    cfg->ctas_per_sm = occ;
    cfg->num_sms = sms;
    return cudaSuccess;
  }
  const int hp = d.str_pack > 1 ? d.str_pack : 1;
  const int grid = d.cta0[d.rows.n] + d.rows.n * ((d.n_str + hp - 1) / hp);
  if (grid == 0) return cudaSuccess;
  cudaLaunchConfig_t lc = {};
  lc.gridDim = dim3(grid);
  lc.blockDim = dim3(NWARPS * 32);
  lc.dynamicSmemBytes = smem;
  lc.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  lc.attrs = attr;
  lc.numAttrs = d.pdl ? 1 : 0;
  return cudaLaunchKernelEx(&lc, kern, p);
}

cudaError_t dispatch(const DecodeFp8Params &p, int G, cudaStream_t s, DecodeConfig *cfg) {
  switch (G) {
    case 1: return run<1>(p, s, cfg);
    case 2: return run<2>(p, s, cfg);
    case 3: return run<3>(p, s, cfg);
    case 4: return run<4>(p, s, cfg);
    case 5: return run<5>(p, s, cfg);
    case 6: return run<6>(p, s, cfg);
    case 7: return run<7>(p, s, cfg);
    case 8: return run<8>(p, s, cfg);
    default: return cudaErrorInvalidValue;
  }
}

}  // namespace d8

bool decode_fp8_supported(int D, int G) { return D == 128 && G >= 1 && G <= 8; }

int decode_fp8_tile_rows() { return d8::NWARPS * d8::T; }

cudaError_t decode_fp8_config(int G, DecodeConfig *cfg) {
  DecodeFp8Params dummy{};
  return d8::dispatch(dummy, G, nullptr, cfg);
}

cudaError_t launch_decode_fp8(const DecodeFp8Params &p, cudaStream_t s) {
  return d8::dispatch(p, p.d.G, s, nullptr);
}

}  // namespace duo
