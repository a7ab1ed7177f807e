// History of an 8-bit cache as bf16 rows, for the chunked pre-fill.
//
// The pre-fill's tensor-core products take bf16 operands, so the part of an
// 8-bit cache that a chunk reads is expanded into a bf16 scratch laid out like
// a bf16 cache: retrieval rows at the storage rows of their codes (packed or
// paged), streaming rows [batch][n_streaming][S + R][d].  A code times its
// power-of-two scale is a bf16 value (4 significant bits), so nothing is
// rounded; rows of the unfinished block come from the bf16 tail as they are.
// The pre-fill's key tiles are 128 rows: rows past a row's length up to the
// end of that tile, and unfilled streaming slots, are written as zeros, so
// that probability 0 times their value stays 0 whatever the scratch or a
// released sequence left there.  Bound: HBM, 128 bytes read and 256 written
// per (key, head) of K and of V; it is about 4% of a 1000-query chunk on
// 15000 tokens.  Pages: "DuoAttention: Efficient
// Long-Context LLM Inference with Retrieval and Streaming Heads"
// (hotpaper.ai), abstract (the split applies to pre-filling too).
#include "common.cuh"
#include "kv8.h"

namespace duo {
namespace {

constexpr int D = 128;

__device__ __forceinline__ uint32_t scaled_pair(uint32_t codes, float s) {  // low 16 bits: two codes
  uint32_t h;
  asm("{.reg .b16 l, h; mov.b32 {l, h}, %1; cvt.rn.f16x2.e4m3x2 %0, l;}" : "=r"(h) : "r"(codes));
  const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
  const __nv_bfloat162 b = __floats2bfloat162_rn(f.x * s, f.y * s);
  return *reinterpret_cast<const uint32_t *>(&b);
}

// One thread per 16 channels of one (key, head) row; blockIdx.y = (launch
// row, head, K or V).
__global__ void dequant_fp8_kernel(const __grid_constant__ DequantFp8Params p) {
  const DequantParams &d = p.d;
  const int heads = d.n_ret + d.n_str;
  const int which = blockIdx.y & 1;  // 0 = K, 1 = V
  const int hh = (blockIdx.y >> 1) % heads;
  const int r = (blockIdx.y >> 1) / heads;
  const int b = d.rows.row[r];
  const int n = d.rows.len[r];
  const bool ret = hh < d.n_ret;
  const int pidx = ret ? hh : hh - d.n_ret;
  const int keys = ret ? n : min(n, d.W);
  const int coded = ret ? n & ~(kScaleBlock - 1) : 0;
  const int64_t rows = ret ? ((int64_t)n + 127) / 128 * 128 : (keys > 0 ? d.W : 0);
  constexpr int CH = 16;
  constexpr int kPerRow = D / CH;
  const uint8_t *codes = which ? d.p.ret_v : d.p.ret_k;
  const float *scales = reinterpret_cast<const float *>(which ? d.p.ret_v_sz : d.p.ret_k_sz);
  const uint8_t *raw = ret ? (which ? p.tail.v : p.tail.k) + ((int64_t)b * d.n_ret + pidx) * (kScaleBlock * D * 2)
                           : (which ? d.p.str_v : d.p.str_k) + ((int64_t)b * d.n_str + pidx) * d.Ws * (int64_t)(D * 2);
  __nv_bfloat16 *dst = ret ? (which ? d.ret_v : d.ret_k) : (which ? d.str_v : d.str_k);
  for (int64_t i = blockIdx.x * (int64_t)blockDim.x + threadIdx.x; i < rows * kPerRow;
       i += (int64_t)gridDim.x * blockDim.x) {
    const int key = (int)(i / kPerRow);
    const int c = (int)(i % kPerRow) * CH;
    const int64_t row = ret ? ret_row(d.ret, b, pidx, key) : ((int64_t)b * d.n_str + pidx) * d.W + key;
    uint4 out[2];
    if (key < coded) {
      const uint4 w = *reinterpret_cast<const uint4 *>(codes + row * D + c);
      const float s = __ldg(scales + (row >> kScaleShift));
      const uint32_t in[4] = {w.x, w.y, w.z, w.w};
      uint32_t o[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[2 * j] = scaled_pair(in[j], s);
        o[2 * j + 1] = scaled_pair(in[j] >> 16, s);
      }
      out[0] = make_uint4(o[0], o[1], o[2], o[3]);
      out[1] = make_uint4(o[4], o[5], o[6], o[7]);
    } else if (key < keys) {
      const uint4 *src = reinterpret_cast<const uint4 *>(raw + ((int64_t)(key - coded) * D + c) * 2);
      out[0] = src[0];
      out[1] = src[1];
    } else {
      out[0] = out[1] = make_uint4(0, 0, 0, 0);
    }
    uint4 *q = reinterpret_cast<uint4 *>(dst + row * D + c);
    q[0] = out[0];
    q[1] = out[1];
  }
}

}  // namespace

cudaError_t launch_dequant_fp8(const DequantFp8Params &p, cudaStream_t s) {
  const DequantParams &d = p.d;
  if (d.rows.n <= 0) return cudaSuccess;
  if (d.D != D) return cudaErrorInvalidValue;
  int64_t max_rows = 0;
  for (int r = 0; r < d.rows.n; ++r) {
    const int64_t n = d.rows.len[r];
    max_rows = max(max_rows, max((n + 127) / 128 * 128, n > 0 ? (int64_t)d.W : (int64_t)0));
  }
  if (max_rows == 0) return cudaSuccess;
  const int threads = 256;
  const int64_t need = (max_rows * (D / 16) + threads - 1) / threads;
  dim3 grid((unsigned)(need < 1024 ? need : 1024), (unsigned)(d.rows.n * (d.n_ret + d.n_str) * 2));
  dequant_fp8_kernel<<<grid, threads, 0, s>>>(p);
  return cudaGetLastError();
}

}  // namespace duo
