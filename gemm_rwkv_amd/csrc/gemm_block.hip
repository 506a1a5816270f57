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
// That instruction adds the products of each eight consecutive k after it has cut
// them 13 binary places below the largest exponent among the eight, subnormal
// codes counting as 2^-6 (measured: 448 + 2^-5 * 0.9 is 448, and nothing is lost
// across groups of eight or beside the accumulator).  A y is off by up to 7 * 2^-13
// of each group's largest product: some 2^-14 of y on ordinary rows, far more of a
// y in which large products cancel.  A y in fp32 is due more, and up to 16 rows,
// where the weight's way from HBM is the bound, more costs little.  There the codes
// are widened to fp16, which holds each of them, their products go through the fp16
// instruction, which keeps fp32, and each block's sum is scaled as it joins the
// row's.  In us, fp8 instruction and widened: 1 x 2048 x 2048 2.9 and 3.2, 1 x 16384 x
// 4096 13.3 and 13.8, 16 x 65536 x 4096 53.0 and 53.5.  With more rows the matrix
// instructions count, and a 16-bit y takes the fp8 one: 32 x 2048 x 2048 3.5 and
// 4.5, 32 x 16384 x 4096 13.1 and 14.1, 64 x 4096 x 4096 7.4 and 9.1, 1024 x 16384 x
// 4096 62 and 149.
//
// Up to some 64 rows the weight's way from HBM bounds it: 32 x 65536 x 4096 into
// fp32 takes 63 us, 4.4 TB/s.  Past that it is the copies from L2 to LDS, which a
// compute unit takes at some 41 GB/s whatever their depth, and the matrix
// instructions: 1024 x 16384 x 4096 takes 61 us (2.25 PFLOP/s), its instructions
// alone 44 and its copies alone 51.
#include <atomic>

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

// Four consecutive outputs of row m from column n on, those that y has.
template <int OUT>
__device__ __forceinline__ void put4(const BlockGemm& p, int m, int n, float4v v) {
  if (m >= p.m || n >= p.n) return;
  const size_t at = (size_t)m * p.ldy + n;
  if (n + 4 <= p.n && (p.ldy & 3) == 0) {
    if constexpr (OUT == OUT_F32) {
      *(float4v*)((float*)p.y + at) = v;
    } else {
      uint2 o;
      o.x = OUT == OUT_F16 ? F16::down2(v[0], v[1]) : BF16::down2(v[0], v[1]);
      o.y = OUT == OUT_F16 ? F16::down2(v[2], v[3]) : BF16::down2(v[2], v[3]);
      *(uint2*)((uint16_t*)p.y + at) = o;
    }
    return;
  }
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (n + i < p.n) put<OUT>(p.y, at + i, v[i]);
}

// The E8M0 bytes of a block of w and one of x, in the lowest byte.
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
    e.w &= 255;
    e.x &= 255;
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

// One LDS DMA: 16 (4) bytes per lane from g to base + 16 (4) * lane.  Inline
// assembly, since the compiler cannot tell which LDS bytes a DMA writes and
// would wait for all of them before any LDS read; it writes no register, and
// every read of its bytes comes after an explicit wait.
__device__ __forceinline__ void dma16(const void* g, uint32_t base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %0, off" ::"v"(g), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void dma4(const void* g, uint32_t base) {
  asm volatile("s_mov_b32 m0, %1\n\ts_nop 0\n\tglobal_load_lds_dword %0, off" ::"v"(g), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_address(const void* p) {
  return (uint32_t)(uintptr_t)(__attribute__((address_space(3))) const uint8_t*)p;
}

// Rows in whole lines: a workgroup has 16 TM rows of x and 16 TN of w; its KW
// waves take the k blocks wave, wave + KW, ... and each covers the whole tile,
// through two private stages of LDS that DMA fills: an instruction copies 8 rows
// x 128 bytes, whole lines, where a load in the operands' own layout touches
// half of each line and gets half of the bytes per clock.  The 16-byte segment s
// of row r lies at slot s ^ (r % 8), so that the sixteen lanes that LDS serves
// together read sixteen bank groups.  The scales of the tile's rows come to LDS
// first.
template <int TM, int TN, int KW, int OUT>
__global__ void __launch_bounds__(64 * KW) gemm_block_lines_kernel(BlockGemm p) {
  constexpr bool EXACT = OUT == OUT_F32 || TM == 1;
  constexpr int BM = 16 * TM, BN = 16 * TN, STAGE = (BM + BN) * 128;
  extern __shared__ uint4 lds4[];
  uint8_t* const lds = (uint8_t*)lds4;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int r = lane & 15, q = lane >> 4;
  const int m0 = blockIdx.y * BM, n0 = blockIdx.x * BN;
  const int blocks = p.k >> 7, srow = (int)scale_row_bytes(p.k);
  uint8_t* const sx = lds + KW * 2 * STAGE;  // [BM][srow], then w's [srow]

  const uint8_t* src[2 * (TM + TN)];
  const int drow = lane >> 3, dslot = lane & 7;
#pragma unroll
  for (int i = 0; i < 2 * (TM + TN); ++i) {
    const int row = 8 * i + drow;
    const int seg = (dslot ^ (row & 7)) << 4;
    src[i] = (i < 2 * TM ? p.xq + (size_t)min(m0 + row, p.m - 1) * p.k : p.wq + (size_t)min(n0 + row - BM, p.n - 1) * p.k) + seg;
  }
  const uint32_t ring = lds_address(lds) + wave * 2 * STAGE;
  auto dma = [&](int stage, int kb) {
#pragma unroll
    for (int i = 0; i < 2 * (TM + TN); ++i) dma16(src[i] + (size_t)kb * 128, ring + stage * STAGE + i * 1024);
  };
  if (wave < blocks) dma(0, wave);
  for (int i = tid; i < (BM + 1) * (srow >> 2); i += 64 * KW) {
    const int row = i / (srow >> 2), at = i - row * (srow >> 2);
    const uint8_t* from = row < BM ? p.sx + (size_t)min(m0 + row, p.m - 1) * srow : p.sw + (size_t)(n0 >> 7) * srow;
    ((uint32_t*)sx)[i] = ((const uint32_t*)from)[at];
  }
  __syncthreads();

  const int swz = r & 7;
  const int o0 = r * 128 + ((q ^ swz) << 4), o1 = r * 128 + (((q + 4) ^ swz) << 4);
  float4v acc[TM][TN];
#pragma unroll
  for (int a = 0; a < TM; ++a)
#pragma unroll
    for (int b = 0; b < TN; ++b) acc[a][b] = float4v{0, 0, 0, 0};
  int stage = 0;
  for (int kb = wave; kb < blocks; kb += KW, stage ^= 1) {
    if (kb + KW < blocks) {
      dma(stage ^ 1, kb + KW);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * (TM + TN)) : "memory");  // block kb has landed
    } else {
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    }
    const uint8_t* at = lds + (wave * 2 + stage) * STAGE;
    uint4 x[TM][2], w[TN][2];
    int ex[TM];
#pragma unroll
    for (int a = 0; a < TM; ++a) {
      x[a][0] = *(const uint4*)(at + a * 2048 + o0);
      x[a][1] = *(const uint4*)(at + a * 2048 + o1);
      ex[a] = sx[(16 * a + r) * srow + kb];
    }
#pragma unroll
    for (int b = 0; b < TN; ++b) {
      w[b][0] = *(const uint4*)(at + (TM + b) * 2048 + o0);
      w[b][1] = *(const uint4*)(at + (TM + b) * 2048 + o1);
    }
    const int ew = sx[BM * srow + kb];
#pragma unroll
    for (int a = 0; a < TM; ++a)
#pragma unroll
      for (int b = 0; b < TN; ++b) acc[a][b] = mfma_block<EXACT>(w[b], x[a], Scales{ew, ex[a]}, acc[a][b]);
  }
  // the waves' sums, one row of tiles at a time, in the stages that are free now
  float4v(*red)[TN][64] = (float4v(*)[TN][64])lds4;
#pragma unroll
  for (int a = 0; a < TM; ++a) {
    __syncthreads();
#pragma unroll
    for (int b = 0; b < TN; ++b) red[wave][b][lane] = acc[a][b];
    __syncthreads();
    for (int b = wave; b < TN; b += KW) {
      float4v v = red[0][b][lane];
#pragma unroll
      for (int w = 1; w < KW; ++w) v += red[w][b][lane];
      put4<OUT>(p, m0 + 16 * a + r, n0 + 16 * b + 4 * q, v);
    }
  }
}

// Many rows: a tile of BM = 16 XT WX rows of x and BN = 16 WT WW of w by WX x WW
// waves, each with XT x WT blocks of 16 x 16 over all of K.  The waves copy every
// k block together into a ring of NB stages, in whole lines and with the same
// swizzle, so that it crosses from L2 once per workgroup.
template <int XT, int WT, int WX, int WW, int NB, int OUT, bool EXACT>
__global__ void __launch_bounds__(64 * WX * WW) gemm_block_tile_kernel(BlockGemm p) {
  constexpr int WAVES = WX * WW, BM = 16 * XT * WX, BN = 16 * WT * WW;
  constexpr int STAGE = (BM + BN) * 128, PER = (BM + BN) / 8 / WAVES;
  static_assert((BM + BN) / 8 % WAVES == 0 && (BM + BN) % 64 == 0, "copies divide over the waves");
  extern __shared__ uint4 lds4[];
  uint8_t* const lds = (uint8_t*)lds4;
  uint32_t* const scales = (uint32_t*)(lds + NB * STAGE);  // [2][BM + BN]: four blocks' bytes each
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), lane = threadIdx.x & 63;
  const int r = lane & 15, q = lane >> 4;
  const int m0 = blockIdx.y * BM, n0 = blockIdx.x * BN;
  const int blocks = p.k >> 7, srow = (int)scale_row_bytes(p.k);
  const int wx = wave / WW, ww = wave % WW;

  const uint8_t* src[PER];
  const int drow = lane >> 3, dslot = lane & 7;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    const int row = 8 * (wave * PER + i) + drow;
    const int seg = (dslot ^ (row & 7)) << 4;
    src[i] = (row < BM ? p.xq + (size_t)min(m0 + row, p.m - 1) * p.k : p.wq + (size_t)min(n0 + row - BM, p.n - 1) * p.k) + seg;
  }
  // and the scales of 64 rows at a time
  constexpr int PARTS = (BM + BN) / 64, EACH = (PARTS + WAVES - 1) / WAVES;
  const uint8_t* ssrc[EACH];
#pragma unroll
  for (int i = 0; i < EACH; ++i) {
    const int row = 64 * (wave + i * WAVES) + lane;
    ssrc[i] = row < BM ? p.sx + (size_t)min(m0 + row, p.m - 1) * srow : p.sw + (size_t)(min(n0 + row - BM, p.n - 1) >> 7) * srow;
  }
  const uint32_t base = lds_address(lds), sbase = base + NB * STAGE;
  auto dma = [&](int kb) {
    if ((kb & 3) == 0)
#pragma unroll
      for (int i = 0; i < EACH; ++i)
        if (wave + i * WAVES < PARTS) dma4(ssrc[i] + kb, sbase + ((kb >> 2) & 1) * 4 * (BM + BN) + (wave + i * WAVES) * 256);
#pragma unroll
    for (int i = 0; i < PER; ++i) dma16(src[i] + (size_t)kb * 128, base + (kb % NB) * STAGE + (wave * PER + i) * 1024);
  };

  const int swz = r & 7;
  const int o0 = r * 128 + ((q ^ swz) << 4), o1 = r * 128 + (((q + 4) ^ swz) << 4);
  float4v acc[XT][WT];
#pragma unroll
  for (int a = 0; a < XT; ++a)
#pragma unroll
    for (int b = 0; b < WT; ++b) acc[a][b] = float4v{0, 0, 0, 0};
  int ex[XT], ew[WT];

#pragma unroll
  for (int j = 0; j < NB - 1; ++j)
    if (j < blocks) dma(j);
  for (int kb = 0; kb < blocks; ++kb) {
    // at most the blocks behind the next may still be on their way
    if (NB > 2 && kb + NB - 2 < blocks)
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"((NB - 2) * PER) : "memory");
    else
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();  // every wave's part of block kb is in; block kb - 1 is done
    if (kb + NB - 1 < blocks) dma(kb + NB - 1);
    const uint8_t* at = lds + (kb % NB) * STAGE;
    const uint8_t* xat = at + wx * XT * 2048;
    const uint8_t* wat = at + BM * 128 + ww * WT * 2048;
    if ((kb & 3) == 0) {
      const uint32_t* s = scales + ((kb >> 2) & 1) * (BM + BN);
#pragma unroll
      for (int a = 0; a < XT; ++a) ex[a] = (int)s[(wx * XT + a) * 16 + r];
#pragma unroll
      for (int b = 0; b < WT; ++b) ew[b] = (int)s[BM + (ww * WT + b) * 16 + r];
    }
    uint4 x[XT][2];
#pragma unroll
    for (int a = 0; a < XT; ++a) {
      x[a][0] = *(const uint4*)(xat + a * 2048 + o0);
      x[a][1] = *(const uint4*)(xat + a * 2048 + o1);
    }
#pragma unroll
    for (int b = 0; b < WT; ++b) {
      uint4 w[2];
      w[0] = *(const uint4*)(wat + b * 2048 + o0);
      w[1] = *(const uint4*)(wat + b * 2048 + o1);
#pragma unroll
      for (int a = 0; a < XT; ++a) acc[a][b] = mfma_block<EXACT>(w, x[a], Scales{ew[b], ex[a]}, acc[a][b]);
    }
#pragma unroll
    for (int a = 0; a < XT; ++a) ex[a] = (int)((uint32_t)ex[a] >> 8);
#pragma unroll
    for (int b = 0; b < WT; ++b) ew[b] = (int)((uint32_t)ew[b] >> 8);
  }
#pragma unroll
  for (int a = 0; a < XT; ++a)
#pragma unroll
    for (int b = 0; b < WT; ++b) put4<OUT>(p, m0 + (wx * XT + a) * 16 + r, n0 + (ww * WT + b) * 16 + 4 * q, acc[a][b]);
}

constexpr size_t kLds = 160 << 10;

// LDS past 64 KB is asked for once per kernel and device.
template <typename K>
bool allow_lds(K kernel, size_t bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess) return false;
  const uint64_t bit = 1ull << (dev & 63);
  if (done.load(std::memory_order_relaxed) & bit) return true;
  if (hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, (int)bytes) != hipSuccess) return false;
  done.fetch_or(bit, std::memory_order_relaxed);
  return true;
}

int64_t tiles(const BlockGemm& p, int rows, int cols) {
  return (int64_t)((p.m + rows - 1) / rows) * ((p.n + cols - 1) / cols);
}

template <int TM, int TN, int KW>
constexpr size_t lines_lds(int64_t k) {
  return (size_t)KW * 2 * 16 * (TM + TN) * 128 + (16 * TM + 1) * (size_t)scale_row_bytes(k);
}
template <int TM, int TN, int KW, int OUT>
hipError_t launch_lines(const BlockGemm& p, hipStream_t st) {
  static std::atomic<uint64_t> done{0};
  if (!allow_lds(gemm_block_lines_kernel<TM, TN, KW, OUT>, kLds, done)) return hipErrorInvalidConfiguration;
  const dim3 grid((p.n + 16 * TN - 1) / (16 * TN), (p.m + 16 * TM - 1) / (16 * TM));
  hipLaunchKernelGGL((gemm_block_lines_kernel<TM, TN, KW, OUT>), grid, dim3(64 * KW), (lines_lds<TM, TN, KW>(p.k)), st, p);
  return hipGetLastError();
}

template <int XT, int WT, int WX, int WW, int NB, int OUT, bool EXACT = OUT == OUT_F32>
hipError_t launch_tile(const BlockGemm& p, hipStream_t st) {
  constexpr int BM = 16 * XT * WX, BN = 16 * WT * WW;
  constexpr size_t lds = (size_t)NB * (BM + BN) * 128 + 8 * (BM + BN);
  static_assert(lds <= kLds, "the ring fits LDS");
  static std::atomic<uint64_t> done{0};
  if (!allow_lds(gemm_block_tile_kernel<XT, WT, WX, WW, NB, OUT, EXACT>, lds, done)) return hipErrorInvalidConfiguration;
  hipLaunchKernelGGL((gemm_block_tile_kernel<XT, WT, WX, WW, NB, OUT, EXACT>), dim3((p.n + BN - 1) / BN, (p.m + BM - 1) / BM),
                     dim3(64 * WX * WW), lds, st, p);
  return hipGetLastError();
}

// The largest tile that still gives most of the 256 compute units one.  Measured
// in us on both sides of each border (m x n x k, 16-bit y):
//   16 x 16, waves 8, or 16 x 32, waves 4, for up to 16 rows: 16 x 2048 x 2048 3.9
//     and 4.6, 16 x 16384 x 4096 17.5 and 17.1, 16 x 32768 x 4096 30.6 and 28.8, 16 x
//     65536 x 4096 56.9 and 53.9; 1 x 16384 x 4096 15.7 and 17.4, 1 x 65536 x 4096
//     49.5 and 51.7, 1 x 65536 x 2048 31 and 25;
//   32 x 16 or 32 x 32: 64 x 2048 x 2048 (256 or 128 tiles) 4.2 and 4.6, 64 x 4096
//     x 4096 (512 or 256) 9.8 and 8.6;
//   32 x 32 or 32 x 64: 64 x 4096 x 4096 (256 or 128) 8.6 and 10.6, 128 x 4096 x
//     4096 (512 or 256) 11.3 and 10.8, 32 x 10240 x 2560 (320 or 160) 10.4 and 9.6;
//   32 x 64 or 64 x 64: 128 x 4096 x 4096 (256 or 128) 10.8 and 13.2, 256 x 4096 x
//     4096 (512 or 256) 17.2 and 13.2, 64 x 10240 x 2560 (320 or 160) 12.7 and 11.8;
//   64 x 64 or 128 x 128: 128 x 8192 x 2048 (256 or 64) 9.2 and 13.6, 200 x 8192 x
//     2048 (512 or 128) 14.9 and 13.1, 512 x 4096 x 4096 (512 or 128) 22.4 and 21.9;
//     with up to 64 rows the larger one is half empty: 64 x 16384 x 4096 19.2 and 22;
//   128 x 128 with four stages or, two workgroups to a compute unit, with two: 256
//     x 16384 x 4096 (256) 26.2 and 34.9, 512 x 16384 x 4096 (512) 46 and 39;
//   128 x 128 or 256 x 256: 1000 x 10240 x 2560 (640 or 160) 41 and 40..48, 1024 x
//     16384 x 4096 (1024 or 256) 71..75 and 60..68.
// A y in fp32 does twice the matrix work, and past 64 x 64 it always takes 128 x
// 128 in two stages: 512 x 4096 x 4096 (128 tiles) 46, in tiles of 64 x 64 32, 200
// x 10240 x 2560 (160) 31.5 and 33, 1000 x 16384 x 4096 150 (four stages 183).
// Scales of a k so long that they do not fit LDS beside the stages (past 64512, or
// 739840 for up to 16 rows) go with the 128 x 128 tile too, which takes four blocks'
// at a time: 2 x 200 x 65664 280 us, in tiles of 16 x 16 23.5.
template <int OUT>
hipError_t launch_out(const BlockGemm& p, hipStream_t st) {
  constexpr bool F32OUT = OUT == OUT_F32;
  if (p.m <= 16) {
    if (lines_lds<1, 1, 8>(p.k) > kLds) return launch_tile<4, 4, 2, 2, 2, OUT, true>(p, st);
    return tiles(p, 16, 16) < 2048 ? launch_lines<1, 1, 8, OUT>(p, st) : launch_lines<1, 2, 4, OUT>(p, st);
  }
  const int64_t t128 = tiles(p, 128, 128);
  if (lines_lds<4, 4, 4>(p.k) > kLds || (p.m > 64 && t128 >= (F32OUT ? 160 : 128))) {
    if constexpr (F32OUT) {
      return launch_tile<4, 4, 2, 2, 2, OUT>(p, st);
    } else {
      if (tiles(p, 256, 256) >= 192) return launch_tile<4, 4, 4, 4, 2, OUT>(p, st);
      return t128 > 256 ? launch_tile<4, 2, 2, 4, 2, OUT>(p, st) : launch_tile<4, 2, 2, 4, 4, OUT>(p, st);
    }
  }
  if (p.m > 32 && tiles(p, 64, 64) >= 160) return launch_lines<4, 4, 4, OUT>(p, st);
  if (tiles(p, 32, 64) >= 160) return launch_lines<2, 4, 4, OUT>(p, st);
  if (tiles(p, 32, 32) >= 160) return launch_lines<2, 2, 4, OUT>(p, st);
  return launch_lines<2, 1, 4, OUT>(p, st);
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
