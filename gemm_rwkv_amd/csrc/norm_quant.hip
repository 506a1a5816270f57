// The norm before an 8-bit product, with the residual before it and the codes
// behind it:
//
//   x' = x + alpha delta,   h = n(x') gamma + beta,
//   n(x') = x',  x' / sqrt(mean x'^2 + eps)  or  (x' - mean) / sqrt(var + eps)
//
// and h in 8 bits, either with one fp32 scale per row (e4m3: absmax / 448,
// int8: absmax / 127, codes the nearest to h / scale) or, in e4m3, with one
// power of two per 128 columns, the smallest with absmax <= 448 of it.  h
// itself is never stored.  Bound by memory: 3 bytes a value, 7 with the
// residual.
//
// A workgroup owns a run of rows and holds a row in registers, 8 channels a
// vector, so that every statistic is of what was read once; gamma and beta
// stay in registers over the run, and the next row is on its way while this
// one is reduced.  A block of 128 columns is 16 consecutive lanes, so its
// scale takes four lane moves and no barrier.
#include "mix.h"
#include "next_token.h"

namespace rq {

namespace {

// Largest bit pattern over the 16 lanes of a row / the wave.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
__device__ __forceinline__ uint32_t row_max(uint32_t v) {
  v = max(v, dpp_u<0x128>(v));
  v = max(v, dpp_u<0x124>(v));
  v = max(v, dpp_u<0x122>(v));
  v = max(v, dpp_u<0x121>(v));
  return v;
}
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = row_max(v);
  v = max(v, (uint32_t)__shfl_xor((int)v, 16));
  return max(v, (uint32_t)__shfl_xor((int)v, 32));
}

// h / s as a float whose rounding to 8 bits is the rounding of the exact
// quotient: where the quotient is no float, the one of its two neighbours whose
// last bit is set, so that no tie arises that is none.  inv: 1 / s.
__device__ __forceinline__ float quotient(float h, float s, float inv) {
  const float q0 = h * inv;
  const float q = __builtin_fmaf(__builtin_fmaf(-q0, s, h), inv, q0);
  const float left = __builtin_fmaf(-q, s, h);
  uint32_t b = __builtin_bit_cast(uint32_t, q);
  if (left != 0.f && !(b & 1u)) b += ((left > 0.f) == (h > 0.f)) ? 1u : ~0u;
  return __builtin_copysignf(__builtin_bit_cast(float, b), h);  // -0 stays -0
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}
__device__ __forceinline__ uint32_t int8x4(float a, float b, float c, float d) {
  return ((uint32_t)(int)rintf(a) & 255u) | ((uint32_t)(int)rintf(b) & 255u) << 8 |
         ((uint32_t)(int)rintf(c) & 255u) << 16 | (uint32_t)(int)rintf(d) << 24;
}

constexpr uint32_t kInf = 0x7f800000u, kNaN = 0x7fc00000u;

template <typename T, int NORM, int FMT, int NV>
__global__ void __launch_bounds__(512) norm_quant_kernel(NormQuant p, int run) {
  // gamma and beta of up to two vectors stay in registers; rows of four
  // (width above 8192) read them again each time
  constexpr bool KEEP = NV <= 2;
  __shared__ float sums[2][2][8];
  __shared__ uint32_t most[2][8];
  const int tid = threadIdx.x, wave = tid >> 6, waves = blockDim.x >> 6;
  const int vecs = p.width >> 3;
  const int begin = blockIdx.x * run, end = run_end(p.rows, begin, run);
  bool on[NV];
  float gm[KEEP ? NV : 1][8], bt[KEEP ? NV : 1][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = j * blockDim.x + tid;
    on[j] = v < vecs;
    if constexpr (KEEP) {
#pragma unroll
      for (int i = 0; i < 8; ++i) gm[j][i] = 1.f, bt[j][i] = -0.f;  // -0 + x is x, also for -0
      if (on[j] && p.gamma) load8f(p.gamma + 8 * v, gm[j]);
      if (on[j] && p.beta) load8f(p.beta + 8 * v, bt[j]);
    }
  }
  uint4 xr[NV], dr[NV];
  auto fetch = [&](int row) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const size_t at = (size_t)row * p.ld + 8 * (j * blockDim.x + tid);
      xr[j] = on[j] ? *(const uint4*)((const uint16_t*)p.x + at) : make_uint4(0, 0, 0, 0);
      if (p.delta) dr[j] = on[j] ? *(const uint4*)((const uint16_t*)p.delta + at) : make_uint4(0, 0, 0, 0);
    }
  };
  fetch(begin);
  int buf = 0;
  for (int row = begin; row < end; ++row, buf ^= 1) {
    float x[NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      up2<T>(xr[j].x, x[j]);
      up2<T>(xr[j].y, x[j] + 2);
      up2<T>(xr[j].z, x[j] + 4);
      up2<T>(xr[j].w, x[j] + 6);
      if (p.delta) {
        float d[8];
        up2<T>(dr[j].x, d);
        up2<T>(dr[j].y, d + 2);
        up2<T>(dr[j].z, d + 4);
        up2<T>(dr[j].w, d + 6);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] = __builtin_fmaf(p.alpha, d[i], x[j][i]);
      }
      if (p.x_out && on[j]) store8<T>(p.x_out, (size_t)row * p.ld + 8 * (j * blockDim.x + tid), x[j]);
    }
    if (row + 1 < end) fetch(row + 1);

    // statistics: two passes over the registers, sums in a fixed order
    float mean = 0.f, rstd = 1.f;
    if constexpr (NORM == NORM_LAYER) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on[j])
#pragma unroll
          for (int i = 0; i < 8; ++i) s += x[j][i];
      s = wave_sum(s);
      if ((tid & 63) == 0) sums[buf][0][wave] = s;
      __syncthreads();
      for (int w = 0; w < waves; ++w) mean += sums[buf][0][w];
      mean /= (float)p.width;
    }
    if constexpr (NORM != NORM_NONE) {
      float s = 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on[j])
#pragma unroll
          for (int i = 0; i < 8; ++i) {
            x[j][i] -= mean;
            s = __builtin_fmaf(x[j][i], x[j][i], s);
          }
      s = wave_sum(s);
      if ((tid & 63) == 0) sums[buf][1][wave] = s;
      __syncthreads();
      float ss = 0.f;
      for (int w = 0; w < waves; ++w) ss += sums[buf][1][w];
      // squares past fp32 must not pass for a large norm
      rstd = finite_f32(ss) ? 1.f / sqrtf(ss / (float)p.width + p.eps) : __builtin_bit_cast(float, kNaN);
    }
    // h, and the largest |h| as a bit pattern (NaN and infinities come out on top)
    uint32_t top[NV], all = 0;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      top[j] = 0;
      if (!KEEP) {
#pragma unroll
        for (int i = 0; i < 8; ++i) gm[0][i] = 1.f, bt[0][i] = -0.f;
        if (on[j] && p.gamma) load8f(p.gamma + 8 * (j * blockDim.x + tid), gm[0]);
        if (on[j] && p.beta) load8f(p.beta + 8 * (j * blockDim.x + tid), bt[0]);
      }
      if (on[j])
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[j][i] = __builtin_fmaf(x[j][i] * rstd, gm[KEEP ? j : 0][i], bt[KEEP ? j : 0][i]);
          top[j] = max(top[j], __builtin_bit_cast(uint32_t, x[j][i]) & 0x7fffffffu);
        }
      all = max(all, top[j]);
    }
    uint8_t* codes = (uint8_t*)p.codes + (size_t)row * p.width;
    if constexpr (FMT == ROW_BLOCK) {
      const int groups = p.width / kBlock, srow = (int)scale_row_bytes(p.width);
      uint8_t* scales = (uint8_t*)p.scales + (size_t)row * srow;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        const uint32_t t = row_max(top[j]);
        const bool bad = t >= kInf;
        // 448 = 1.75 * 2^8: the exponent of the largest, less 8, and one more
        // where its mantissa exceeds 1.75
        const int byte = max((int)(t >> 23) - 8 + ((t & 0x7fffffu) > 0x600000u), 0);
        const float inv = __builtin_bit_cast(float, (uint32_t)(254 - byte) << 23);
        if (!on[j]) continue;
        const int v = j * blockDim.x + tid;
        uint2 c;
        c.x = e4m3x4(x[j][0] * inv, x[j][1] * inv, x[j][2] * inv, x[j][3] * inv);
        c.y = e4m3x4(x[j][4] * inv, x[j][5] * inv, x[j][6] * inv, x[j][7] * inv);
        if (bad) c = make_uint2(0, 0);
        *(uint2*)(codes + 8 * v) = c;
        if ((v & 15) == 0) scales[v >> 4] = bad ? 0xff : (uint8_t)byte;
      }
      if (groups + tid < srow) scales[groups + tid] = 0;
    } else {
      constexpr float kMost = FMT == ROW_FP8 ? 448.f : 127.f;
      all = wave_max(all);
      if ((tid & 63) == 0) most[buf][wave] = all;
      __syncthreads();
      all = 0;
      for (int w = 0; w < waves; ++w) all = max(all, most[buf][w]);
      const bool bad = all >= kInf;
      const float scale = __builtin_bit_cast(float, all) / kMost;
      // tiny rows: the quotient's remainder stays a normal number
      const float up = scale < 0x1p-60f ? 0x1p64f : 1.f;
      const float s = scale * up, inv = 1.f / s;
      const bool none = bad || scale == 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!on[j]) continue;
        uint2 c = make_uint2(0, 0);
        if (!none) {
          float q[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf(quotient(x[j][i] * up, s, inv), -kMost), kMost);
          if constexpr (FMT == ROW_FP8) {
            c.x = e4m3x4(q[0], q[1], q[2], q[3]);
            c.y = e4m3x4(q[4], q[5], q[6], q[7]);
          } else {
            c.x = int8x4(q[0], q[1], q[2], q[3]);
            c.y = int8x4(q[4], q[5], q[6], q[7]);
          }
        }
        *(uint2*)(codes + 8 * (j * blockDim.x + tid)) = c;
      }
      if (tid == 0) ((float*)p.scales)[row] = bad ? __builtin_bit_cast(float, kNaN) : scale;
    }
  }
}

template <typename T, int NORM, int FMT>
hipError_t launch_format(const NormQuant& p, hipStream_t st) {
  const int vecs = p.width / 8;
  const int nv = vecs <= 512 ? 1 : vecs <= 1024 ? 2 : 4;
  const int per = (vecs + nv - 1) / nv;
  const int threads = (per + 63) / 64 * 64;
  const int run = 1 + p.rows / 4096;
  const dim3 grid(run_count(p.rows, run)), block(threads);
  if (nv == 1)
    hipLaunchKernelGGL((norm_quant_kernel<T, NORM, FMT, 1>), grid, block, 0, st, p, run);
  else if (nv == 2)
    hipLaunchKernelGGL((norm_quant_kernel<T, NORM, FMT, 2>), grid, block, 0, st, p, run);
  else
    hipLaunchKernelGGL((norm_quant_kernel<T, NORM, FMT, 4>), grid, block, 0, st, p, run);
  return hipGetLastError();
}

template <typename T, int NORM>
hipError_t launch_norm(const NormQuant& p, int format, hipStream_t st) {
  switch (format) {
    case ROW_FP8: return launch_format<T, NORM, ROW_FP8>(p, st);
    case ROW_INT8: return launch_format<T, NORM, ROW_INT8>(p, st);
    default: return launch_format<T, NORM, ROW_BLOCK>(p, st);
  }
}

template <typename T>
hipError_t launch_type(const NormQuant& p, int norm, int format, hipStream_t st) {
  switch (norm) {
    case NORM_NONE: return launch_norm<T, NORM_NONE>(p, format, st);
    case NORM_RMS: return launch_norm<T, NORM_RMS>(p, format, st);
    default: return launch_norm<T, NORM_LAYER>(p, format, st);
  }
}

}  // namespace

hipError_t launch_norm_quant(const NormQuant& p, int norm, int format, bool bf16, hipStream_t st) {
  return bf16 ? launch_type<BF16>(p, norm, format, st) : launch_type<F16>(p, norm, format, st);
}

}  // namespace rq
