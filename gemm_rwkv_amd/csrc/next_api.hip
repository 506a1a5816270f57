// C ABI of what follows a model's last layer (include/rq.h): argument checks,
// then the launches on the caller's stream.
#include <hip/hip_runtime.h>
#include <string.h>

#include "buffers.h"
#include "next_token.h"
#include "rq.h"
#include "validate.h"

using rqv::Buffers;

namespace {

int hip_status(hipError_t e) { return e == hipSuccess ? RQ_OK : RQ_ERR_HIP; }

// a type of rows as the launchers count them, or -1
int out_type(int dtype) {
  switch (dtype) {
    case RQ_F16: return rq::OUT_F16;
    case RQ_BF16: return rq::OUT_BF16;
    case RQ_F32: return rq::OUT_F32;
  }
  return -1;
}

// grids of one launch: a workgroup has a row or a tile
constexpr int64_t kMostRows = (int64_t)1 << 21;
constexpr int64_t kMostOutputs = (int64_t)1 << 27;

}  // namespace

extern "C" {

int rq_norm_quantize(int dtype, int norm, const void* x, const void* delta, float alpha, int64_t rows, int64_t width,
                     int64_t ld, const float* gamma, const float* beta, float eps, int format, void* x_out, void* codes,
                     void* scales, void* stream) {
  if (dtype != RQ_F16 && dtype != RQ_BF16) return RQ_ERR_FORMAT;
  if (norm != RQ_NORM_NONE && norm != RQ_NORM_RMS && norm != RQ_NORM_LAYER) return RQ_ERR_VALUE;
  int kind;
  switch (format) {
    case RQ_FP8_E4M3_CH: kind = rq::ROW_FP8; break;
    case RQ_I8_CH: kind = rq::ROW_INT8; break;
    case RQ_FP8_E4M3_B128: kind = rq::ROW_BLOCK; break;
    default: return RQ_ERR_FORMAT;
  }
  if (rows < 0 || rows >= rqv::kMaxDim || width < 1 || width > rq::kNormMostWidth ||
      width % (kind == rq::ROW_BLOCK ? rq::kBlock : 16) != 0)
    return RQ_ERR_SHAPE;
  if (ld < width || ld >= rqv::kMaxDim || rows * ld >= ((int64_t)1 << 40)) return RQ_ERR_SHAPE;
  if (ld % 8) return RQ_ERR_ALIGN;
  if (!(eps >= 0.f && eps <= 1e30f)) return RQ_ERR_VALUE;
  Buffers io;
  const size_t srow = kind == rq::ROW_BLOCK ? (size_t)rq::scale_row_bytes(width) : 4;
  io.read_rows(x, rows, width, ld);
  io.read_rows(delta, rows, width, ld, false);
  io.read(gamma, (size_t)width * 4, false);
  io.read(beta, (size_t)width * 4, false);
  io.write_rows(x_out, rows, width, ld, false, x);
  io.write(codes, (size_t)rows * width, rows > 0);
  io.write(scales, (size_t)rows * srow, rows > 0);
  int st;
  if ((st = io.check(nullptr, 0)) != RQ_OK) return st;
  if (rows == 0) return RQ_OK;
  rq::NormQuant p;
  memset(&p, 0, sizeof(p));
  p.x = x;
  p.delta = delta;
  p.alpha = alpha;
  p.rows = (int)rows;
  p.width = (int)width;
  p.ld = (int)ld;
  p.gamma = gamma;
  p.beta = beta;
  p.eps = eps;
  p.x_out = x_out;
  p.codes = codes;
  p.scales = scales;
  return hip_status(rq::launch_norm_quant(p, norm, kind, dtype == RQ_BF16, (hipStream_t)stream));
}

int rq_gemm_fp8_block(const uint8_t* xq, const uint8_t* sx, int64_t m, const rq_qweight* w, int dtype, void* y,
                      int64_t ldy, void* stream) {
  int st = rqv::check_weight(w);
  if (st != RQ_OK) return st;
  if (w->format != RQ_FP8_E4M3_B128) return RQ_ERR_FORMAT;
  const int out = out_type(dtype);
  if (out < 0) return RQ_ERR_FORMAT;
  if (m < 0 || m >= kMostRows || w->n > kMostOutputs || ldy < w->n || ldy < 1 || ldy >= rqv::kMaxDim || m * ldy >= ((int64_t)1 << 40) ||
      m * w->k >= ((int64_t)1 << 40))
    return RQ_ERR_SHAPE;
  Buffers io;
  rqv::Span spans[4];
  rqv::weight_spans(w, spans);
  for (int i = 0; i < 2; ++i) io.in[io.nin++] = spans[i];
  const int64_t elem = out == rq::OUT_F32 ? 4 : 2;
  io.read(xq, (size_t)m * w->k, m > 0);
  io.read(sx, (size_t)m * rq::scale_row_bytes(w->k), m > 0);
  io.write(y, m > 0 ? (size_t)((m - 1) * ldy + w->n) * elem : 0, m > 0 && w->n > 0);
  if ((st = io.check(nullptr, 0)) != RQ_OK) return st;
  if (m == 0 || w->n == 0) return RQ_OK;
  rq::BlockGemm p;
  memset(&p, 0, sizeof(p));
  p.xq = xq;
  p.sx = sx;
  p.wq = (const uint8_t*)w->codes;
  p.sw = (const uint8_t*)w->scales;
  p.y = y;
  p.m = (int)m;
  p.n = (int)w->n;
  p.k = (int)w->k;
  p.ldy = (int)ldy;
  return hip_status(rq::launch_gemm_block(p, out, (hipStream_t)stream));
}

int rq_sample(int dtype, const void* logits, int64_t rows, int64_t vocab, int64_t ld, const float* temperature,
              const int32_t* top_k, const float* top_p, const float* min_p, const float* u, int32_t* token,
              float* logprob, void* stream) {
  const int type = out_type(dtype);
  if (type < 0) return RQ_ERR_FORMAT;
  if (rows < 0 || rows >= kMostRows || vocab < 1 || vocab > rq::kMostVocab || ld < vocab || ld >= rqv::kMaxDim ||
      rows * ld >= ((int64_t)1 << 40))
    return RQ_ERR_SHAPE;
  if (ld % 8) return RQ_ERR_ALIGN;
  const bool any = rows > 0;
  Buffers io;
  io.read(logits, any ? (size_t)((rows - 1) * ld + vocab) * (type == rq::OUT_F32 ? 4 : 2) : 0, any);
  io.read_index(temperature, rows);
  io.read_index(top_k, rows);
  io.read_index(top_p, rows);
  io.read_index(min_p, rows);
  io.read_index(u, rows, any);
  io.write_index(token, rows, any);
  io.write_index(logprob, rows, false);
  int st;
  if ((st = io.check(nullptr, 0)) != RQ_OK) return st;
  if (!any) return RQ_OK;
  rq::Sample p;
  memset(&p, 0, sizeof(p));
  p.logits = logits;
  p.rows = (int)rows;
  p.vocab = (int)vocab;
  p.ld = (int)ld;
  p.temperature = temperature;
  p.top_k = top_k;
  p.top_p = top_p;
  p.min_p = min_p;
  p.u = u;
  p.token = token;
  p.logprob = logprob;
  return hip_status(rq::launch_sample(p, type, (hipStream_t)stream));
}

}  // extern "C"
