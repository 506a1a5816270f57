// Internal launchers of what follows a model's last layer: the norm that
// leaves 8-bit rows (norm_quant.hip), fp8 products with block scales
// (gemm_block.hip), and sampling (sample.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace rq {

constexpr int kBlock = 128;  // columns (and weight rows) that share a power of two

// Bytes of one row of block scales: one per 128 columns, in words of four.
constexpr int64_t scale_row_bytes(int64_t k) { return 4 * ((k + 4 * kBlock - 1) / (4 * kBlock)); }

// ---- norm and 8-bit rows ------------------------------------------------------
enum NormKind { NORM_NONE = 0, NORM_RMS = 1, NORM_LAYER = 2 };
enum RowFormat { ROW_FP8 = 0, ROW_INT8 = 1, ROW_BLOCK = 2 };

struct NormQuant {
  const void* x;      // [rows][ld]
  const void* delta;  // [rows][ld] or null
  float alpha;
  int rows, width, ld;
  const float* gamma;  // [width] or null
  const float* beta;   // [width] or null
  float eps;
  void* x_out;    // [rows][ld] or null
  void* codes;    // [rows][width]
  void* scales;   // fp32 [rows], or bytes [rows][scale_row_bytes(width)]
};
constexpr int kNormMostWidth = 16384;  // a row is held in the registers of one workgroup
hipError_t launch_norm_quant(const NormQuant& p, int norm, int format, bool bf16, hipStream_t st);

// ---- fp8 products with block scales ---------------------------------------------
enum OutType { OUT_F16 = 0, OUT_BF16 = 1, OUT_F32 = 2 };

struct BlockGemm {
  const uint8_t* xq;  // e4m3 [m][k]
  const uint8_t* sx;  // [m][scale_row_bytes(k)]
  const uint8_t* wq;  // e4m3 [n][k]
  const uint8_t* sw;  // [ceil(n / 128)][scale_row_bytes(k)]
  void* y;            // [m][ldy]
  int m, n, k, ldy;
};
hipError_t launch_gemm_block(const BlockGemm& p, int out, hipStream_t st);

// ---- sampling -------------------------------------------------------------------
struct Sample {
  const void* logits;  // [rows][ld]
  int rows, vocab, ld;
  const float* temperature;  // [rows], as the next three; each may be null
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* u;
  int32_t* token;
  float* logprob;  // or null
};
constexpr int kMostVocab = 1 << 20;
hipError_t launch_sample(const Sample& p, int type, hipStream_t st);  // type: OutType

}  // namespace rq
