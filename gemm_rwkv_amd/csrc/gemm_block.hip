// fp8 products with a power of two per block of 128:
//
//   y[m][n] = sum_b 2^(ex[m][b] + ew[n / 128][b]) sum_{k in block b} x[m][k] w[n][k]
//
// of e4m3 codes, b over blocks of 128 k.  v_mfma_scale_f32_16x16x128_f8f6f4
// takes a whole block and both of its scales: lane (r, q) = (lane % 16,
// lane / 16) holds 32 of the 128 k of row r of either operand, and the scale of
// row r as an E8M0 byte, so the scales cost no arithmetic and sums stay in the
// accumulators for all of K.  Which 32 k a lane holds is free as long as x and w
// agree: it takes the 16-byte segments q and q + 4 of the block's row.  w is the
// first operand, so that a lane's four results are consecutive outputs of one
// row of y.
//
// That instruction adds products that it has cut 13 binary places below the
// largest exponent among them (measured: 448 + 2^-5 * 0.9 is 448): some 2^-14 of
// y, under the half step of a 16-bit y (2^-11, 2^-8).  A y in fp32 is due more,
// so there the codes are widened to fp16, which holds each of them, their
// products go through the fp16 instruction, which keeps fp32, and each block's
// sum is scaled as it joins the row's.
#include "mix.h"
#include "next_token.h"

namespace rq {

namespace {

typedef _Float16 halves2 __attribute__((ext_vector_type(2)));

// Eight e4m3 codes as fp16, exactly.
__device__ __forceinline__ half8 widen8(const uint32_t* c) {
  const halves2 a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[0], 1.f, false);
  const halves2 b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[0], 1.f, true);
  const halves2 d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[1], 1.f, false);
  const halves2 e = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c[1], 1.f, true);
  return half8{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

template <int OUT>
__device__ __forceinline__ void put(void* y, size_t at, float v) {
  if constexpr (OUT == OUT_F32)
    ((float*)y)[at] = v;
  else if constexpr (OUT == OUT_F16)
    ((uint16_t*)y)[at] = f32_to_f16_bits(v);
  else
    ((uint16_t*)y)[at] = __builtin_bit_cast(uint16_t, (__bf16)v);
}

// The E8M0 bytes of a block of w and one of x.
struct Scales {
  int w, x;
};

// c += a block's products: 32 codes per lane of 16 rows of w and of x.
template <bool EXACT>
__device__ __forceinline__ float4v mfma_block(const uint4* w, const uint4* x, Scales e, float4v c) {
  if constexpr (EXACT) {
    float4v sum = {0, 0, 0, 0};
    const uint32_t ww[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
    const uint32_t xx[8] = {x[0].x, x[0].y, x[0].z, x[0].w, x[1].x, x[1].y, x[1].z, x[1].w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      sum = __builtin_amdgcn_mfma_f32_16x16x32_f16(widen8(ww + 2 * i), widen8(xx + 2 * i), sum, 0, 0, 0);
    const float one = e.w == 255 || e.x == 255 ? __builtin_nanf("") : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) c[i] = __builtin_fmaf(__builtin_amdgcn_ldexpf(sum[i], e.w + e.x - 254), one, c[i]);
    return c;
  } else {
    const int8v wv = {(int)w[0].x, (int)w[0].y, (int)w[0].z, (int)w[0].w, (int)w[1].x, (int)w[1].y, (int)w[1].z, (int)w[1].w};
    const int8v xv = {(int)x[0].x, (int)x[0].y, (int)x[0].z, (int)x[0].w, (int)x[1].x, (int)x[1].y, (int)x[1].z, (int)x[1].w};
    return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wv, xv, c, 0, 0, 0, e.w, 0, e.x);
  }
}

// Few rows: the weights stream from memory straight into registers.
//
// A workgroup has 16 NT rows of w and all of x; its KW waves take the k blocks
// wave, wave + KW, ... in groups of U whose loads are issued together, and
// their sums meet in LDS in wave order.  Rows past m or n read the last one:
// they only reach outputs that are never stored.
template <int MT, int NT, int KW, int U, int OUT>
__global__ void __launch_bounds__(64 * KW) gemm_block_stream_kernel(BlockGemm p) {
  __shared__ float4v red[KW][MT * NT][64];
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, q = lane >> 4;
  const int m0 = blockIdx.y * 16 * MT, n0 = blockIdx.x * 16 * NT;
  const int blocks = p.k >> 7;
  const int srow = (int)scale_row_bytes(p.k);
  const uint8_t *xs[MT], *ws[NT], *xe[MT], *we[NT];
#pragma unroll
  for (int a = 0; a < MT; ++a) {
    const size_t row = (size_t)min(m0 + 16 * a + r, p.m - 1);
    xs[a] = p.xq + row * p.k + 16 * q;
    xe[a] = p.sx + row * srow;
  }
#pragma unroll
  for (int b = 0; b < NT; ++b) {
    const size_t row = (size_t)min(n0 + 16 * b + r, p.n - 1);
    ws[b] = p.wq + row * p.k + 16 * q;
    we[b] = p.sw + (row >> 7) * srow;
  }
  float4v acc[MT][NT];
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b) acc[a][b] = float4v{0, 0, 0, 0};

  for (int first = wave; first < blocks; first += KW * U) {
    uint4 x[U][MT][2], w[U][NT][2];
    int ex[U][MT], ew[U][NT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      // past the end: the last block again, with its product left out
      const int kb = min(first + u * KW, blocks - 1);
#pragma unroll
      for (int b = 0; b < NT; ++b) {
        w[u][b][0] = *(const uint4*)(ws[b] + (size_t)kb * 128);
        w[u][b][1] = *(const uint4*)(ws[b] + (size_t)kb * 128 + 64);
        ew[u][b] = we[b][kb];
      }
#pragma unroll
      for (int a = 0; a < MT; ++a) {
        x[u][a][0] = *(const uint4*)(xs[a] + (size_t)kb * 128);
        x[u][a][1] = *(const uint4*)(xs[a] + (size_t)kb * 128 + 64);
        ex[u][a] = xe[a][kb];
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (first + u * KW < blocks)
#pragma unroll
        for (int a = 0; a < MT; ++a)
#pragma unroll
          for (int b = 0; b < NT; ++b) acc[a][b] = mfma_block<OUT == OUT_F32>(w[u][b], x[u][a], Scales{ew[u][b], ex[u][a]}, acc[a][b]);
  }
#pragma unroll
  for (int a = 0; a < MT; ++a)
#pragma unroll
    for (int b = 0; b < NT; ++b) red[wave][a * NT + b][lane] = acc[a][b];
  __syncthreads();
  for (int t = wave; t < MT * NT; t += KW) {
    float4v v = red[0][t][lane];
#pragma unroll
    for (int w = 1; w < KW; ++w) v += red[w][t][lane];
    const int m = m0 + (t / NT) * 16 + r;
    if (m >= p.m) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + (t % NT) * 16 + 4 * q + i;
      if (n < p.n) put<OUT>(p.y, (size_t)m * p.ldy + n, v[i]);
    }
  }
}

template <int MT, int OUT>
hipError_t launch_stream(const BlockGemm& p, hipStream_t st) {
  const dim3 grid((p.n + 15) / 16, (p.m + 16 * MT - 1) / (16 * MT));
  hipLaunchKernelGGL((gemm_block_stream_kernel<MT, 1, 4, 2, OUT>), grid, dim3(256), 0, st, p);
  return hipGetLastError();
}

template <int OUT>
hipError_t launch_out(const BlockGemm& p, hipStream_t st) {
  if (p.m <= 16) return launch_stream<1, OUT>(p, st);
  return launch_stream<4, OUT>(p, st);
}

}  // namespace

hipError_t launch_gemm_block(const BlockGemm& p, int out, hipStream_t st) {
  switch (out) {
    case OUT_F16: return launch_out<OUT_F16>(p, st);
    case OUT_BF16: return launch_out<OUT_BF16>(p, st);
    default: return launch_out<OUT_F32>(p, st);
  }
}

}  // namespace rq
