// The norm before a block and its mixtures with the token before, and their
// gradient:
//
//   x' = x + alpha delta,   h_t = (x'_t - mean) rstd gamma + beta,
//   out_i,t = h_t + (h_{t-1} - h_t) mu_i,   i < nmix
//
// where h_{-1} of a sequence is the row that the call before left behind
// (shift_in; zeros without one) and the last h of each sequence is left for
// the next (shift_out).  One pass: two rows in, 1 + nmix out.  Bound by memory.
//
// A workgroup owns a run of consecutive rows and holds a row in registers,
// eight channels per thread and vector; h of the row before stays in registers
// from one row to the next and is computed again where a run begins inside a
// sequence.
#include "mix.h"

namespace rq {

namespace {

// Sums of two values over the workgroup, in a fixed order.  buf alternates
// between calls, so one barrier per call is enough.
__device__ __forceinline__ void block_sum2(float& a, float& b, float2 (*red)[16], int& buf, int waves) {
  a = wave_sum(a);
  b = wave_sum(b);
  if ((threadIdx.x & 63) == 0) red[buf][threadIdx.x >> 6] = make_float2(a, b);
  __syncthreads();
  float sa = 0.f, sb = 0.f;
  for (int i = 0; i < waves; ++i) {
    const float2 v = red[buf][i];
    sa += v.x;
    sb += v.y;
  }
  a = sa;
  b = sb;
  buf ^= 1;
}

// mean and 1 / sqrt(var + eps) of a row held in registers, in two passes
template <int NV>
__device__ __forceinline__ void row_stats(const float (*x)[8], const bool* on, int width, float eps, float2 (*red)[16],
                                          int& buf, int waves, float& mean, float& rstd) {
  float s = 0.f, z = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (on[j])
#pragma unroll
      for (int i = 0; i < 8; ++i) s += x[j][i];
  block_sum2(s, z, red, buf, waves);
  mean = s / (float)width;
  float q = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (on[j])
#pragma unroll
      for (int i = 0; i < 8; ++i) q = fmaf(x[j][i] - mean, x[j][i] - mean, q);
  block_sum2(q, z, red, buf, waves);
  rstd = rsqrtf(q / (float)width + eps);
}

}  // namespace

template <typename T, int NV>
__global__ void __launch_bounds__(512) shift_norm_kernel(ShiftNorm p, int rows, int tiles) {
  __shared__ float2 red[2][16];
  int buf = 0;
  const int waves = blockDim.x >> 6;
  const int width = p.width;

  // the workgroups past the last tile carry the rows of empty sequences over
  if ((int)blockIdx.x >= tiles) {
    const int i = blockIdx.x - tiles;
    int b, e;
    seq_span(p.seq, i, b, e);
    const int slot = slot_of(p.slots, i);
    if (b == e && slot >= 0)
      for (int c = threadIdx.x * 8; c < width; c += blockDim.x * 8) {
        const size_t at = (size_t)slot * width + c;
        *(uint4*)((uint16_t*)p.shift_out + at) =
            p.shift_in ? *(const uint4*)((const uint16_t*)p.shift_in + at) : make_uint4(0, 0, 0, 0);
      }
    return;
  }

  int col[NV];
  bool on[NV];
  float gamma[NV][8], beta[NV][8];
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    col[j] = (j * blockDim.x + threadIdx.x) * 8;
    on[j] = col[j] < width;
    if (!on[j]) col[j] = 0;
    load8f(p.gamma + col[j], gamma[j]);
    load8f(p.beta + col[j], beta[j]);
  }

  // x' of row t in registers
  auto fetch = [&](int t, float (*x)[8]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const size_t at = (size_t)t * p.ld + col[j];
      load8<T>(p.x, at, x[j]);
      if (p.delta) {
        float d[8];
        load8<T>(p.delta, at, d);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] = fmaf(p.alpha, d[i], x[j][i]);
      }
    }
  };
  auto norm = [&](float (*x)[8]) {
    float mean, rstd;
    row_stats<NV>(x, on, width, p.eps, red, buf, waves, mean, rstd);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = fmaf((x[j][i] - mean) * rstd, gamma[j][i], beta[j][i]);
  };

  const int t0 = blockIdx.x * rows, t1 = min(p.seq.tokens, t0 + rows);
  int s = seq_of(p.seq, t0), begin, end;
  seq_span(p.seq, s, begin, end);
  float h[NV][8], prev[NV][8];
  if (t0 > begin) {
    fetch(t0 - 1, prev);
    norm(prev);
  }
  for (int t = t0; t < t1; ++t) {
    while (t >= end && s + 1 < p.seq.nseq) seq_span(p.seq, ++s, begin, end);
    if (t == begin) {
      const int slot = slot_of(p.slots, s);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (p.shift_in && slot >= 0)
          load8<T>(p.shift_in, (size_t)slot * width + col[j], prev[j]);
        else
#pragma unroll
          for (int i = 0; i < 8; ++i) prev[j][i] = 0.f;
      }
      // the sequence's last row, by the workgroup that has read its shift_in,
      // so that shift_out may be the same array
      if (p.shift_out && slot >= 0 && end > begin) {
        fetch(end - 1, h);
        norm(h);
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (on[j]) store8<T>(p.shift_out, (size_t)slot * width + col[j], h[j]);
      }
    }
    fetch(t, h);
    if (p.x_out)
#pragma unroll
      for (int j = 0; j < NV; ++j)
        if (on[j]) store8<T>(p.x_out, (size_t)t * p.ld + col[j], h[j]);
    norm(h);
    for (int i = 0; i < p.nmix; ++i) {
      const float* mu = p.mu + (size_t)i * width;
      void* out = (uint16_t*)p.out + ((size_t)i * p.seq.tokens + t) * p.ldo;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!on[j]) continue;
        float m[8];
        load8f(mu + col[j], m);
#pragma unroll
        for (int q = 0; q < 8; ++q) m[q] = fmaf(prev[j][q] - h[j][q], m[q], h[j][q]);
        store8<T>(out, col[j], m);
      }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) prev[j][i] = h[j][i];
  }
}

namespace {
// threads of a workgroup that holds a row of `width` in nv vectors per thread
int threads_of(int width, int nv) { return (width / 8 + nv * 64 - 1) / (nv * 64) * 64; }
}  // namespace

hipError_t launch_shift_norm(const ShiftNorm& p, bool bf16, hipStream_t st) {
  const int nv = p.width > 4096 ? 2 : 1;
  // one row per workgroup while the rows do not fill the card, then four (a
  // run's first row costs the norm of the row before it)
  const int rows = p.seq.tokens <= 1024 ? 1 : 4 + p.seq.tokens / (1 << 22);
  const int tiles = (p.seq.tokens + rows - 1) / rows;
  const int empty = p.shift_out && (p.seq.cu || p.seq.tokens == 0) && p.shift_out != p.shift_in ? p.seq.nseq : 0;
  if (tiles + empty == 0) return hipSuccess;
  const dim3 grid(tiles + empty), block(threads_of(p.width, nv));
  if (bf16 && nv == 1)
    hipLaunchKernelGGL((shift_norm_kernel<BF16, 1>), grid, block, 0, st, p, rows, tiles);
  else if (bf16)
    hipLaunchKernelGGL((shift_norm_kernel<BF16, 2>), grid, block, 0, st, p, rows, tiles);
  else if (nv == 1)
    hipLaunchKernelGGL((shift_norm_kernel<F16, 1>), grid, block, 0, st, p, rows, tiles);
  else
    hipLaunchKernelGGL((shift_norm_kernel<F16, 2>), grid, block, 0, st, p, rows, tiles);
  return hipGetLastError();
}

// Backward.  With prev_t = h_{t-1} (or shift_in), p_t = sum_i dout_i,t mu_i and
// q_t = sum_i dout_i,t - p_t:
//   dh_t = q_t + p_{t+1} (next token of the same sequence) + dshift_out (last)
//   dmu_i = sum_t dout_i,t (prev_t - h_t),   dshift_in = p of the first token
//   dgamma = sum dh n, dbeta = sum dh, dn = dh gamma,
//   dx = dx_out + (dn - mean(dn) - n mean(dn n)) rstd,   ddelta = alpha dx
// A workgroup walks its run of rows once and finishes row t - 1 when it has
// p_t; it also reads the row after its run.  The parameter gradients stay in
// registers over the run and are written as one row of partial sums, which a
// second kernel adds in order.
template <typename T, int NV, int NM>
__global__ void __launch_bounds__(512) shift_norm_back_kernel(ShiftNormBack p, int rows) {
  __shared__ float2 red[2][16];
  int buf = 0;
  const int waves = blockDim.x >> 6;
  const int width = p.width;
  int col[NV];
  bool on[NV];
  float gamma[NV][8], beta[NV][8];
  float dgamma[NV][8] = {}, dbeta[NV][8] = {}, dmu[NM][NV][8] = {};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    col[j] = (j * blockDim.x + threadIdx.x) * 8;
    on[j] = col[j] < width;
    if (!on[j]) col[j] = 0;
    load8f(p.gamma + col[j], gamma[j]);
    load8f(p.beta + col[j], beta[j]);
  }
  // n of row t and its 1 / sqrt(var + eps)
  auto norm = [&](int t, float (*n)[8], float& rstd) {
    float mean;
#pragma unroll
    for (int j = 0; j < NV; ++j) load8<T>(p.x, (size_t)t * p.ld + col[j], n[j]);
    row_stats<NV>(n, on, width, p.eps, red, buf, waves, mean, rstd);
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) n[j][i] = (n[j][i] - mean) * rstd;
  };

  const int t0 = blockIdx.x * rows, t1 = min(p.seq.tokens, t0 + rows);
  // n and q of the row to finish, and its rstd
  float n[NV][8], q[NV][8], rstd = 0.f;
  if (t0 < t1) {
    int s = seq_of(p.seq, t0), begin, end;
    seq_span(p.seq, s, begin, end);
    if (t0 > begin) norm(t0 - 1, n, rstd);
    for (int t = t0; t <= t1; ++t) {
      // gradients that reach row t and the row before it
      float qt[NV][8] = {}, pt[NV][8] = {};
      bool first = t == p.seq.tokens;
      if (!first) {
        while (t >= end && s + 1 < p.seq.nseq) seq_span(p.seq, ++s, begin, end);
        first = t == begin;
      }
      float nt[NV][8], rstdt = 0.f;
      if (t < t1) norm(t, nt, rstdt);
      if (t < t1 || !first) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float h[8] = {};
          if (t < t1) {
            // prev - h
            if (first) {
              if (p.shift_in) load8<T>(p.shift_in, (size_t)s * width + col[j], h);
#pragma unroll
              for (int i = 0; i < 8; ++i) h[i] -= fmaf(nt[j][i], gamma[j][i], beta[j][i]);
            } else {
#pragma unroll
              for (int i = 0; i < 8; ++i) h[i] = (n[j][i] - nt[j][i]) * gamma[j][i];
            }
          }
#pragma unroll
          for (int m = 0; m < NM; ++m) {
            if (m < p.nmix) {
              float d[8], mu[8];
              load8<T>(p.dout, ((size_t)m * p.seq.tokens + t) * p.ldo + col[j], d);
              load8f(p.mu + (size_t)m * width + col[j], mu);
#pragma unroll
              for (int i = 0; i < 8; ++i) {
                pt[j][i] = fmaf(d[i], mu[i], pt[j][i]);
                qt[j][i] += d[i];
                if (t < t1) dmu[m][j][i] = fmaf(d[i], h[i], dmu[m][j][i]);
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 8; ++i) qt[j][i] -= pt[j][i];
          if (t < t1 && first && p.dshift_in && on[j]) store8<T>(p.dshift_in, (size_t)s * width + col[j], pt[j]);
          if (t < t1 && t + 1 == end && p.dshift_out) {
            float d[8];
            load8<T>(p.dshift_out, (size_t)s * width + col[j], d);
#pragma unroll
            for (int i = 0; i < 8; ++i) qt[j][i] += d[i];
          }
        }
      }
      if (t > t0) {
        // finish row t - 1
        float m1 = 0.f, m2 = 0.f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (on[j])
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              const float dh = first ? q[j][i] : q[j][i] + pt[j][i];
              dgamma[j][i] = fmaf(dh, n[j][i], dgamma[j][i]);
              dbeta[j][i] += dh;
              q[j][i] = dh * gamma[j][i];
              m1 += q[j][i];
              m2 = fmaf(q[j][i], n[j][i], m2);
            }
        block_sum2(m1, m2, red, buf, waves);
        m1 /= (float)width;
        m2 /= (float)width;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (!on[j]) continue;
          const size_t at = (size_t)(t - 1) * p.ld + col[j];
          float d[8] = {};
          if (p.dx_out) load8<T>(p.dx_out, at, d);
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] = fmaf(q[j][i] - m1 - n[j][i] * m2, rstd, d[i]);
          store8<T>(p.dx, at, d);
          if (p.ddelta) {
#pragma unroll
            for (int i = 0; i < 8; ++i) d[i] *= p.alpha;
            store8<T>(p.ddelta, at, d);
          }
        }
      }
      rstd = rstdt;
#pragma unroll
      for (int j = 0; j < NV; ++j)
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          n[j][i] = nt[j][i];
          q[j][i] = qt[j][i];
        }
    }
  }
  // the empty sequences' shift gradients pass through; workgroup 0 does them
  if (blockIdx.x == 0 && p.dshift_in && (p.seq.cu || p.seq.tokens == 0))
    for (int i = 0; i < p.seq.nseq; ++i) {
      int b, e;
      seq_span(p.seq, i, b, e);
      if (b != e) continue;
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        if (!on[j]) continue;
        const size_t at = (size_t)i * width + col[j];
        *(uint4*)((uint16_t*)p.dshift_in + at) =
            p.dshift_out ? *(const uint4*)((const uint16_t*)p.dshift_out + at) : make_uint4(0, 0, 0, 0);
      }
    }
  const bool alone = gridDim.x == 1;
  float* part = p.parts + (size_t)blockIdx.x * (2 + p.nmix) * width;
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    if (!on[j]) continue;
    auto put = [&](float* alone_to, int which, const float* f) {
      float* to = (alone ? alone_to : part + (size_t)which * width) + col[j];
      *(float4*)to = *(const float4*)f;
      *(float4*)(to + 4) = *(const float4*)(f + 4);
    };
    put(p.dgamma, 0, dgamma[j]);
    put(p.dbeta, 1, dbeta[j]);
#pragma unroll
    for (int m = 0; m < NM; ++m)
      if (m < p.nmix) put(p.dmu + (size_t)m * width, 2 + m, dmu[m][j]);
  }
}

namespace {
template <typename T, int NV>
void start_back(const ShiftNormBack& p, int rows, dim3 grid, dim3 block, hipStream_t st) {
  if (p.nmix == 1)
    hipLaunchKernelGGL((shift_norm_back_kernel<T, NV, 1>), grid, block, 0, st, p, rows);
  else if (p.nmix <= 6)
    hipLaunchKernelGGL((shift_norm_back_kernel<T, NV, 6>), grid, block, 0, st, p, rows);
  else
    hipLaunchKernelGGL((shift_norm_back_kernel<T, NV, 8>), grid, block, 0, st, p, rows);
}
}  // namespace

hipError_t launch_shift_norm_back(const ShiftNormBack& p, bool bf16, hipStream_t st) {
  const int nv = p.width > 4096 ? 2 : 1;
  const size_t row = (size_t)(2 + p.nmix) * p.width * 4;
  int64_t groups = 512;  // two workgroups per compute unit
  const int64_t fit = p.parts ? (int64_t)(p.parts_bytes / row) : 0;
  if (groups > fit) groups = fit;
  if (groups > p.seq.tokens) groups = p.seq.tokens;
  if (groups < 1) groups = 1;
  const int rows = (int)((p.seq.tokens + groups - 1) / groups);
  if (rows > 0) groups = (p.seq.tokens + rows - 1) / rows;
  const dim3 grid((unsigned)groups), block(threads_of(p.width, nv));
  if (bf16 && nv == 1)
    start_back<BF16, 1>(p, rows, grid, block, st);
  else if (bf16)
    start_back<BF16, 2>(p, rows, grid, block, st);
  else if (nv == 1)
    start_back<F16, 1>(p, rows, grid, block, st);
  else
    start_back<F16, 2>(p, rows, grid, block, st);
  hipError_t e = hipGetLastError();
  if (groups == 1 || e != hipSuccess) return e;
  const size_t stride = (size_t)(2 + p.nmix) * p.width;
  e = launch_sum_parts(p.parts, (int)groups, p.width, stride, p.dgamma, st);
  if (e == hipSuccess) e = launch_sum_parts(p.parts + p.width, (int)groups, p.width, stride, p.dbeta, st);
  if (e == hipSuccess) e = launch_sum_parts(p.parts + 2 * (size_t)p.width, (int)groups, p.nmix * p.width, stride, p.dmu, st);
  return e;
}

}  // namespace rq
