// Internal interface of the rotary and 8-bit cache kernels (beside kernels.h).
#pragma once

#include "kernels.h"

namespace duo {

// KvType of the 8-bit cache: retrieval heads hold e4m3 codes with one
// power-of-two float32 scale per block of kScaleBlock tokens and KV head (K
// and V apart); the newest, unfinished block of each (row, head) stays in bf16
// in a tail buffer [B][n_ret][kScaleBlock][D] until it is full.  Streaming
// heads keep bf16 rows.
constexpr int kFP8 = 3;
constexpr int kScaleShift = 5;
constexpr int kScaleBlock = 1 << kScaleShift;

struct TailPtrs {
  uint8_t *k, *v;  // bf16 [B][n_ret][kScaleBlock][D]; null for other types
};

// Per-head norm and position rotation of queries and keys (duo_rope_desc).
struct RopeParams {
  const float *inv_freq;         // device [rot_dim / 2]
  const void *q_norm, *k_norm;   // device [D] in the inputs' type, or null
  float eps, mscale;
  int rot_dim, interleaved;
};

// A [tokens][heads][D] input with strides in elements.
struct HeadView {
  const void *p;
  int64_t tok, head;
};

// Rows of the standalone pass and of the append with rotation.  Token i of
// the inputs belongs to launch row i / n_tok.
struct RopeRowsParams {
  HeadView q, k, v;           // v unused by the standalone pass; q.p may be null
  void *q_out, *k_out;        // dense [tokens][heads][D]; k_out only standalone
  const int64_t *positions;   // [tokens], or null: the cache position (append only)
  RopeParams rope;
  int Hq, Hkv;
  int64_t tokens;             // all rows together
  // append: where the K and V rows go (AppendParams' k and v are unused)
  AppendParams a;
  TailPtrs tail;
  // 8-bit cache: CTAs of scale blocks in front of the row CTAs
  int block_items;            // scale-block items per (row, head group), at most over rows
  int heads_per_cta;          // retrieval heads one scale-block CTA walks
  int tails_in_rows;          // no row completes a block: the row CTAs write the tails
};

struct DecodeFp8Params {
  DecodeParams d;             // p.ret_k_sz / p.ret_v_sz: float32 scales
  TailPtrs tail;
};

// History of an 8-bit cache expanded to bf16 for the pre-fill.
struct DequantFp8Params {
  DequantParams d;            // p.str_*: bf16 rows
  TailPtrs tail;
};

// Pre-fill with a retrieval item's tiles cut into ns runs: each run's
// normalised output [256][128] and log-sum-exp (base 2) [256], by CTA.
struct PrefillSplit {
  float *o, *lse;
  int ns;
};
// Most retrieval CTAs of a split pre-fill (twice the SMs): bounds its workspace.
constexpr int kPrefillSplitCtas = 296;

cudaError_t launch_qk_norm_rope(const RopeRowsParams &p, int io_type, int D, cudaStream_t s);
cudaError_t launch_append_rope(const RopeRowsParams &p, int kv_type, cudaStream_t s);
cudaError_t launch_dequant_fp8(const DequantFp8Params &p, cudaStream_t s);
bool decode_fp8_supported(int D, int G);
cudaError_t decode_fp8_config(int G, DecodeConfig *cfg);
cudaError_t launch_decode_fp8(const DecodeFp8Params &p, cudaStream_t s);
// Keys a CTA of the 8-bit decode walks per iteration; host only.
int decode_fp8_tile_rows();

int prefill_splits(const PrefillParams &p, int num_sms, int forced);  // 1: do not split; forced 0: choose
size_t prefill_split_bytes();
cudaError_t launch_prefill_split(const PrefillParams &p, int ns, void *ws, cudaStream_t s);

}  // namespace duo
