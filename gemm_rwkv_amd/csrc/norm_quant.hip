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
//
// All of it is fp64, from x' (exact unless x and alpha delta lie 2^18 apart) over
// the sums to h: with any of them in fp32 some h in a million came out on the
// other side of a border between two codes.
//
// 8192 rows of 4096 with residual, layer norm and block scales take 54 us, 4.3
// TB/s, where a large copy reaches 5.0 (x' and the sums in fp32 52, h too 47), and
// without residual 41, for 20 at the copy's rate: vector instructions then, some 36
// a value.  One scale a row, whose quotients are in fp64, takes 73, and 61 to 63.  A
// few rows take the latency of their reads and of two reductions: 2.8 us for one of
// 2048.
#include "mix.h"
#include "next_token.h"

namespace rq {

namespace {

// Largest over the 16 lanes of a row / the wave.
template <int CTRL>
__device__ __forceinline__ uint32_t moved(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xf, 0xf, true);
}
template <int CTRL>
__device__ __forceinline__ uint64_t moved(uint64_t v) {
  return (uint64_t)moved<CTRL>((uint32_t)(v >> 32)) << 32 | moved<CTRL>((uint32_t)v);
}
template <int CTRL>
__device__ __forceinline__ double moved(double v) {
  return __builtin_bit_cast(double, moved<CTRL>(__builtin_bit_cast(uint64_t, v)));
}
template <typename N>
__device__ __forceinline__ N row_max(N v) {
  v = max(v, moved<0x128>(v));  // row_ror 8, 4, 2, 1
  v = max(v, moved<0x124>(v));
  v = max(v, moved<0x122>(v));
  v = max(v, moved<0x121>(v));
  return v;
}
__device__ __forceinline__ uint64_t wave_max(uint64_t v) {
  v = row_max(v);
  v = max(v, (uint64_t)__shfl_xor((unsigned long long)v, 16));
  return max(v, (uint64_t)__shfl_xor((unsigned long long)v, 32));
}
__device__ __forceinline__ double sum64(double v) {
  v += moved<0x128>(v);
  v += moved<0x124>(v);
  v += moved<0x122>(v);
  v += moved<0x121>(v);
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}
// 1 / sqrt(v) to 2^-42, of a first value in fp32 (the library's root and quotient
// in fp64 would be some hundred instructions that a row waits for)
__device__ __forceinline__ double inverse_root(double v) {
  if (v < 0x1p-100) return 1.0 / sqrt(v);
  const double y = __builtin_amdgcn_rsqf((float)v);
  return __builtin_fma(y * 0.5, __builtin_fma(-v * y, y, 1.0), y);
}

// The upper half of a double, its last bit set where the lower half is not zero:
// 20 bits of the value that round to 8-bit codes as all of it does.
__device__ __forceinline__ uint32_t upper(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  return (uint32_t)(b >> 32) | min((uint32_t)b, 1u);
}
// 2^-e of it as a float, 0 below 2^-126.
__device__ __forceinline__ float from_upper(uint32_t u, int e) {
  const uint32_t a = __builtin_elementwise_sub_sat(u & 0x7fffffffu, (uint32_t)(1023 - 127 + e) << 20);
  return __builtin_bit_cast(float, a << 3 | (u & 0x80000000u));
}

// h / s, exact where it is a double.  inv: 1 / s.
__device__ __forceinline__ double quotient(double h, double s, double inv) {
  const double q = h * inv;
  return __builtin_copysign(__builtin_fma(__builtin_fma(-q, s, h), inv, q), h);  // -0 stays -0
}

__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int v = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, v, true);
}
__device__ __forceinline__ uint32_t int8x4(float a, float b, float c, float d) {
  return ((uint32_t)(int)rintf(a) & 255u) | ((uint32_t)(int)rintf(b) & 255u) << 8 |
         ((uint32_t)(int)rintf(c) & 255u) << 16 | (uint32_t)(int)rintf(d) << 24;
}

constexpr uint32_t kNaN = 0x7fc00000u;
constexpr uint32_t kPastFloat = 0x47f00000u;  // upper half of 2^128: what fp32 cannot say is not finite

// Sums past fp32 (and NaN) make a row not finite.
__device__ __forceinline__ bool past_float(double sum) { return !(__builtin_fabs(sum) <= 3.4028234663852886e38); }

template <typename T, int NORM, int FMT, int NV>
__global__ void __launch_bounds__(512) norm_quant_kernel(NormQuant p, int run) {
  // gamma and beta of up to two vectors stay in registers; rows of four
  // (width above 8192) read them again each time
  constexpr bool KEEP = NV <= 2;
  __shared__ double sums[2][2][8];
  __shared__ uint64_t most[2][8];
  const int tid = threadIdx.x, wave = tid >> 6, waves = blockDim.x >> 6;
  const int vecs = p.width >> 3;
  const int begin = blockIdx.x * run, end = run_end(p.rows, begin, run);
  const double part = 1.0 / p.width;
  bool on[NV];
  double gm[KEEP ? NV : 1][8], bt[KEEP ? NV : 1][8];
  auto params = [&](int j, int at) {
    float g[8], b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = 1.f, b[i] = -0.f;  // -0 + x is x, also for -0
    if (on[at] && p.gamma) load8f(p.gamma + 8 * (at * blockDim.x + tid), g);
    if (on[at] && p.beta) load8f(p.beta + 8 * (at * blockDim.x + tid), b);
#pragma unroll
    for (int i = 0; i < 8; ++i) gm[j][i] = g[i], bt[j][i] = b[i];
  };
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    const int v = j * blockDim.x + tid;
    on[j] = v < vecs;
    if constexpr (KEEP) params(j, j);
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
    double x[NV][8];
    double h[FMT == ROW_BLOCK ? 1 : NV][8];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      float f[8];
      up2<T>(xr[j].x, f);
      up2<T>(xr[j].y, f + 2);
      up2<T>(xr[j].z, f + 4);
      up2<T>(xr[j].w, f + 6);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = f[i];
      if (p.delta) {
        float d[8];
        up2<T>(dr[j].x, d);
        up2<T>(dr[j].y, d + 2);
        up2<T>(dr[j].z, d + 4);
        up2<T>(dr[j].w, d + 6);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          x[j][i] = __builtin_fma((double)p.alpha, (double)d[i], x[j][i]);
          f[i] = (float)x[j][i];
        }
      }
      if (p.x_out && on[j]) store8<T>(p.x_out, (size_t)row * p.ld + 8 * (j * blockDim.x + tid), f);
    }
    if (row + 1 < end) fetch(row + 1);

    // statistics: two passes over the registers, sums in a fixed order
    double rstd = 1;
    if constexpr (NORM == NORM_LAYER) {
      double s = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on[j])
#pragma unroll
          for (int i = 0; i < 8; ++i) s += x[j][i];
      const double w = sum64(s);
      if ((tid & 63) == 0) sums[buf][0][wave] = w;
      __syncthreads();
      double sum = 0;
      for (int w = 0; w < waves; ++w) sum += sums[buf][0][w];
      // the quotient, rounded right: a row of one value has no other mean
      double mean = sum * part;
      mean = __builtin_fma(__builtin_fma(-mean, (double)p.width, sum), part, mean);
      if (past_float(sum)) mean = __builtin_nan("");
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] -= mean;
    }
    if constexpr (NORM != NORM_NONE) {
      double s = 0;
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on[j])
#pragma unroll
          for (int i = 0; i < 8; ++i) s = __builtin_fma(x[j][i], x[j][i], s);
      const double w = sum64(s);
      if ((tid & 63) == 0) sums[buf][1][wave] = w;
      __syncthreads();
      double ss = 0;
      for (int w = 0; w < waves; ++w) ss += sums[buf][1][w];
      rstd = past_float(ss) ? __builtin_nan("") : inverse_root(__builtin_fma(ss, part, (double)p.eps));
    }
    // h, and the largest |h| as a bit pattern (NaN and infinities come out on top)
    uint64_t all = 0;
    uint8_t* codes = (uint8_t*)p.codes + (size_t)row * p.width;
    const int groups = p.width / kBlock, srow = (int)scale_row_bytes(p.width);
    uint8_t* scales = (uint8_t*)p.scales + (size_t)row * srow;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      constexpr bool kBlocks = FMT == ROW_BLOCK;
      if (!KEEP) params(0, j);
      double* hj = h[kBlocks ? 0 : j];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        double n = x[j][i];
        if constexpr (NORM != NORM_NONE) n *= rstd;
        hj[i] = __builtin_fma(n, gm[KEEP ? j : 0][i], bt[KEEP ? j : 0][i]);
        // (both of one type: of two, max() would be that of doubles)
        if (!kBlocks && on[j]) all = max(all, __builtin_bit_cast(uint64_t, __builtin_fabs(hj[i])));
      }
      if constexpr (FMT == ROW_BLOCK) {
        uint32_t u[8], t = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          u[i] = upper(hj[i]);
          t = max(t, u[i] & 0x7fffffffu);
        }
        t = row_max(on[j] ? t : 0u);
        const bool bad = t >= kPastFloat;
        // 448 = 1.75 * 2^8: the exponent of the largest, less 8, and one more
        // where its mantissa exceeds 1.75
        const int byte = max((int)(t >> 20) - 1023 + 127 - 8 + ((t & 0xfffffu) > 0xc0000u), 0);
        if (!on[j]) continue;
        const int v = j * blockDim.x + tid;
        float q[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) q[i] = from_upper(u[i], byte - 127);
        uint2 c;
        c.x = e4m3x4(q[0], q[1], q[2], q[3]);
        c.y = e4m3x4(q[4], q[5], q[6], q[7]);
        if (bad) c = make_uint2(0, 0);
        *(uint2*)(codes + 8 * v) = c;
        if ((v & 15) == 0) scales[v >> 4] = bad ? 0xff : (uint8_t)byte;
      }
    }
    if constexpr (FMT == ROW_BLOCK) {
      if (groups + tid < srow) scales[groups + tid] = 0;
    } else {
      constexpr float kMost = FMT == ROW_FP8 ? 448.f : 127.f;
      all = wave_max(all);
      if ((tid & 63) == 0) most[buf][wave] = all;
      __syncthreads();
      all = 0;
      for (int w = 0; w < waves; ++w) all = max(all, most[buf][w]);
      const bool bad = (uint32_t)(all >> 32) >= kPastFloat;
      const float scale = (float)(__builtin_bit_cast(double, all) / (double)kMost);
      const double s = scale, inv = 1.0 / s;
      const bool none = bad || scale == 0.f;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!on[j]) continue;
        uint2 c = make_uint2(0, 0);
        if (!none) {
          float q[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) q[i] = fminf(fmaxf(from_upper(upper(quotient(h[j][i], s, inv)), 0), -kMost), kMost);
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

// As few vectors a thread as 512 threads allow, and a row a workgroup until 4096
// rows, then one more for each 4096.  In us, fp16 with residual:
//   one vector or two, block scales: 1 x 4096 3.5 and 4.0, 1021 x 2048 6.0 and 6.2,
//     1021 x 4096 10.2 and 10.6, 8192 x 2048 28.7 and 29.5; many rows of some 4096
//     would rather have two, 8192 x 4096 55.5 and 51.7 (61 and 52 with one scale a
//     row);
//   two or four: 1 x 8192 4.5 and 5.4, 1021 x 8192 19.0 and 17.7, 4096 x 8192 60
//     and 61 (75 and 68);
//   one, two, three, four and eight rows, block scales: 4000 x 4096 30 29 30 28 28,
//     8192 x 4096 54 55 54 53 52, 16384 x 4096 108 102 100 98 97, 8192 x 8192 131 110
//     111 108 107, 40000 x 1024 (ten by the rule) 71 61 59 60 61.
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
