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
// several channels per thread; h of the row before stays in registers
// from one row to the next and is computed again where a run begins inside a
// sequence.  Measured with six mixtures: 4099 tokens of width 2560 in bf16 45
// us, 4.2 TB/s (a copy reaches 5.0); 32 tokens of width 4096 5.7 us, of which
// half is the launch and the rest one row's chain: offsets, slot, row, two sums.
#include "mix.h"

namespace rq {

namespace {

// Sums of N values over the workgroup, in a fixed order.  buf alternates
// between calls, so one barrier per call is enough.
template <int N>
__device__ __forceinline__ void block_sum(float (&v)[N], float (*red)[16][4], int& buf, int waves) {
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = wave_sum(v[k]);
  if ((threadIdx.x & 63) == 0)
#pragma unroll
    for (int k = 0; k < N; ++k) red[buf][threadIdx.x >> 6][k] = v[k];
  __syncthreads();
#pragma unroll
  for (int k = 0; k < N; ++k) v[k] = 0.f;
  for (int i = 0; i < waves; ++i) {
    const float4v x = *(const float4v*)red[buf][i];
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] += x[k];
  }
  buf ^= 1;
}

// A thread's share of a row's sum, and of its squares about the mean.
template <int NV, int CH>
__device__ __forceinline__ float part_sum(const float (*x)[CH], const bool* on) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (on[j])
#pragma unroll
      for (int i = 0; i < CH; ++i) s += x[j][i];
  return s;
}
template <int NV, int CH>
__device__ __forceinline__ float part_squares(const float (*x)[CH], const bool* on, float mean) {
  float s = 0.f;
#pragma unroll
  for (int j = 0; j < NV; ++j)
    if (on[j])
#pragma unroll
      for (int i = 0; i < CH; ++i) s = fmaf(x[j][i] - mean, x[j][i] - mean, s);
  return s;
}

template <typename T>
__device__ __forceinline__ void up8(uint4 v, float* f) {
  up2<T>(v.x, f);
  up2<T>(v.y, f + 2);
  up2<T>(v.z, f + 4);
  up2<T>(v.w, f + 6);
}
template <typename T>
__device__ __forceinline__ void up4(uint2 v, float* f) {
  up2<T>(v.x, f);
  up2<T>(v.y, f + 2);
}
// four channels of a row: the row's address is the same for all threads, so
// that it lies in scalar registers
__device__ __forceinline__ uint2 raw4(const void* base, size_t row, int col) {
  return *(const uint2*)((const uint16_t*)base + row + (unsigned)col);
}
template <typename T>
__device__ __forceinline__ void load4(const void* base, size_t row, int col, float* f) {
  up4<T>(raw4(base, row, col), f);
}
template <typename T>
__device__ __forceinline__ void store4(void* base, size_t row, int col, const float* f) {
  *(uint2*)((uint16_t*)base + row + (unsigned)col) = make_uint2(T::down2(f[0], f[1]), T::down2(f[2], f[3]));
}
__device__ __forceinline__ void load4f(const float* p, float* f) { *(float4*)f = *(const float4*)p; }
__device__ __forceinline__ uint4 raw8(const void* base, size_t elem) { return *(const uint4*)((const uint16_t*)base + elem); }

}  // namespace

template <typename T, int NV>
__global__ void __launch_bounds__(512) shift_norm_kernel(ShiftNorm p, int rows, int tiles) {
  __shared__ __align__(16) float red[2][16][4];
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

  uint4 rx[NV], rd[NV];
  auto fetch = [&](int t) {
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      const size_t at = (size_t)t * p.ld + col[j];
      rx[j] = raw8(p.x, at);
      if (p.delta) rd[j] = raw8(p.delta, at);
    }
  };
  auto sum = [&](float (*x)[8]) {  // x' of the row fetched
#pragma unroll
    for (int j = 0; j < NV; ++j) {
      up8<T>(rx[j], x[j]);
      if (p.delta) {
        float d[8];
        up8<T>(rd[j], d);
#pragma unroll
        for (int i = 0; i < 8; ++i) x[j][i] = fmaf(p.alpha, d[i], x[j][i]);
      }
    }
  };
  auto norm = [&](float (*x)[8], float mean, float rstd) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) x[j][i] = fmaf((x[j][i] - mean) * rstd, gamma[j][i], beta[j][i]);
  };
  const float inv = 1.f / (float)width;

  const int t0 = blockIdx.x * rows, t1 = run_end(p.seq.tokens, t0, rows);
  int s = seq_of(p.seq, t0), begin, end;
  seq_span(p.seq, s, begin, end);
  // Each turn has row t in h, its mean, and row t + 1 on its way; one barrier
  // sums row t's squares and row t + 1.
  float h[NV][8], next[NV][8], prev[NV][8];
  const int first = t0 > begin ? t0 - 1 : t0;
  fetch(first);
  sum(h);
  if (first + 1 < t1) fetch(first + 1);
  float v1[1] = {part_sum<NV>(h, on)};
  block_sum(v1, red, buf, waves);
  float mean = v1[0] * inv;
  bool opened = false;  // the sequence at hand begins in this run
  for (int t = first; t < t1; ++t) {
    const bool more = t + 1 < t1;
    if (more) {
      sum(next);
      if (t + 2 < t1) fetch(t + 2);
    }
    float v[2] = {part_squares<NV>(h, on, mean), more ? part_sum<NV>(next, on) : 0.f};
    block_sum(v, red, buf, waves);
    const float rstd = rsqrtf(v[0] * inv + p.eps);
    if (t >= t0) {
      while (t >= end && s + 1 < p.seq.nseq) {
        seq_span(p.seq, ++s, begin, end);
        opened = false;
      }
      if (p.x_out)
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (on[j]) store8<T>(p.x_out, (size_t)t * p.ld + col[j], h[j]);
    }
    norm(h, mean, rstd);
    if (t >= t0) {
      const int slot = slot_of(p.slots, s);
      if (t == begin) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (p.shift_in && slot >= 0)
            load8<T>(p.shift_in, (size_t)slot * width + col[j], prev[j]);
          else
#pragma unroll
            for (int i = 0; i < 8; ++i) prev[j][i] = 0.f;
        }
        opened = true;
        // The sequence's last row, by the workgroup that has read its
        // shift_in, so that shift_out may be the same array; here if it lies
        // past this run, below if within.
        if (p.shift_out && slot >= 0 && end > t1) {
          float x[NV][8];
          uint4 kx[NV], kd[NV];
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            kx[j] = rx[j];
            kd[j] = rd[j];
          }
          fetch(end - 1);
          sum(x);
#pragma unroll
          for (int j = 0; j < NV; ++j) {
            rx[j] = kx[j];
            rd[j] = kd[j];
          }
          float a[1] = {part_sum<NV>(x, on)};
          block_sum(a, red, buf, waves);
          const float m = a[0] * inv;
          a[0] = part_squares<NV>(x, on, m);
          block_sum(a, red, buf, waves);
          norm(x, m, rsqrtf(a[0] * inv + p.eps));
#pragma unroll
          for (int j = 0; j < NV; ++j)
            if (on[j]) store8<T>(p.shift_out, (size_t)slot * width + col[j], x[j]);
        }
      }
      if (t + 1 == end && opened && p.shift_out && slot >= 0)
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (on[j]) store8<T>(p.shift_out, (size_t)slot * width + col[j], h[j]);
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
    }
    mean = v[1] * inv;
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        prev[j][i] = h[j][i];
        h[j][i] = next[j][i];
      }
  }
}

namespace {
// threads of a workgroup that holds a row of `width` in nv vectors per thread
int threads_of(int width, int nv) { return (width / 8 + nv * 64 - 1) / (nv * 64) * 64; }
}  // namespace

hipError_t launch_shift_norm(const ShiftNorm& p, bool bf16, hipStream_t st) {
  const int nv = p.width > 4096 ? 2 : 1;
  const int rows = norm_rows(p.seq.tokens);
  const int tiles = run_count(p.seq.tokens, rows);
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
// p_t; it also reads the row after its run.  One barrier per row sums the four
// values that three rows in different stages need.  Four channels per thread:
// the sums of eight parameters' gradients and three rows take more than the 128
// registers that a workgroup of 1024 has: with six mixtures 18 spills to scratch
// memory, with eight 62 to 86, above width 4096 (two vectors per thread) some
// 310 and 450; with one mixture none and 2.  The parameter gradients are held
// over the run and written as one row of partial sums, which a second kernel
// adds in order.  Measured: 4096 tokens of width 2048, six
// mixtures, bf16, 64 us, 2.6 TB/s: two workgroups per compute unit do not hide
// each row's barrier, sums and spills, and their registers allow no third.
template <typename T, int NV, int NM>
__global__ void __launch_bounds__(1024) shift_norm_back_kernel(ShiftNormBack p, int rows, bool mu_lds) {
  extern __shared__ __align__(16) float mus[];  // mu, if it fits: each row needs all of it
  __shared__ __align__(16) float red[2][16][4];
  int buf = 0;
  const int waves = blockDim.x >> 6;
  const int width = p.width;
  int col[NV];
  bool on[NV];
  float gamma[NV][4];
  float dgamma[NV][4] = {}, dbeta[NV][4] = {}, dmu[NM][NV][4] = {};
#pragma unroll
  for (int j = 0; j < NV; ++j) {
    col[j] = (j * blockDim.x + threadIdx.x) * 4;
    on[j] = col[j] < width;
    if (!on[j]) col[j] = 0;
    load4f(p.gamma + col[j], gamma[j]);
  }
  if (mu_lds) {
    for (int i = threadIdx.x * 4; i < p.nmix * width; i += blockDim.x * 4) *(float4*)(mus + i) = *(const float4*)(p.mu + i);
    __syncthreads();
  }
  const float inv = 1.f / (float)width;
  auto row = [&](int t, float (*x)[4]) {
#pragma unroll
    for (int j = 0; j < NV; ++j) load4<T>(p.x, (size_t)t * p.ld, col[j], x[j]);
  };
  auto norm = [&](float (*x)[4], float mean, float rstd) {
#pragma unroll
    for (int j = 0; j < NV; ++j)
#pragma unroll
      for (int i = 0; i < 4; ++i) x[j][i] = (x[j][i] - mean) * rstd;
  };
  const int t0 = blockIdx.x * rows, t1 = run_end(p.seq.tokens, t0, rows);
  if (t0 < t1) {
    int s = seq_of(p.seq, t0), begin, end;
    seq_span(p.seq, s, begin, end);
    // n, q and 1 / sqrt of the row to finish (t - 1); n of row t; row t + 1 with
    // its mean; the planes of row t, and what finishes row t - 1, on their way
    float n[NV][4], q[NV][4], nt[NV][4];
    uint2 r1[NV] = {};
    float rstd = 0.f, rstdt, mean1;
    uint2 rd[NM][NV], rup[NV] = {}, rx[NV] = {};
    auto fetch = [&](int t) {
#pragma unroll
      for (int m = 0; m < NM; ++m)
        if (m < p.nmix)
#pragma unroll
          for (int j = 0; j < NV; ++j) rd[m][j] = raw4(p.dout, ((size_t)m * p.seq.tokens + t) * p.ldo, col[j]);
    };
    fetch(t0);
    {
      const bool before = t0 > begin;
      row(before ? t0 - 1 : t0, n);
      row(t0, nt);
      float x1[NV][4] = {};
      if (t0 + 1 < t1) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          r1[j] = raw4(p.x, (size_t)(t0 + 1) * p.ld, col[j]);
          up4<T>(r1[j], x1[j]);
        }
      }
      float a[3] = {part_sum<NV>(n, on), part_sum<NV>(nt, on), part_sum<NV>(x1, on)};
      block_sum(a, red, buf, waves);
      float c[2] = {part_squares<NV>(n, on, a[0] * inv), part_squares<NV>(nt, on, a[1] * inv)};
      block_sum(c, red, buf, waves);
      rstd = rsqrtf(c[0] * inv + p.eps);
      rstdt = rsqrtf(c[1] * inv + p.eps);
      norm(n, a[0] * inv, rstd);
      norm(nt, a[1] * inv, rstdt);
      mean1 = a[2] * inv;
    }
    if (t0 + 2 < t1)
#pragma unroll
      for (int j = 0; j < NV; ++j) rx[j] = raw4(p.x, (size_t)(t0 + 2) * p.ld, col[j]);
    for (int t = t0; t <= t1; ++t) {
      // gradients that reach row t and the row before it
      float qt[NV][4] = {}, pt[NV][4] = {};
      bool first = t == p.seq.tokens;
      if (!first) {
        while (t >= end && s + 1 < p.seq.nseq) seq_span(p.seq, ++s, begin, end);
        first = t == begin;
      }
      const bool inside = t < t1;
      if (inside || !first) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          float d0[4] = {};
          if (inside) {
            // prev - h
            if (first) {
              float beta[4];
              load4f(p.beta + col[j], beta);
              if (p.shift_in) load4<T>(p.shift_in, (size_t)s * width, col[j], d0);
#pragma unroll
              for (int i = 0; i < 4; ++i) d0[i] -= fmaf(nt[j][i], gamma[j][i], beta[i]);
            } else {
#pragma unroll
              for (int i = 0; i < 4; ++i) d0[i] = (n[j][i] - nt[j][i]) * gamma[j][i];
            }
          }
#pragma unroll
          for (int m = 0; m < NM; ++m) {
            if (m < p.nmix) {
              float d[4], mu[4];
              up4<T>(rd[m][j], d);
              load4f((mu_lds ? mus : p.mu) + (size_t)m * width + (unsigned)col[j], mu);
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                pt[j][i] = fmaf(d[i], mu[i], pt[j][i]);
                qt[j][i] += d[i];
                dmu[m][j][i] = fmaf(d[i], d0[i], dmu[m][j][i]);
              }
            }
          }
#pragma unroll
          for (int i = 0; i < 4; ++i) qt[j][i] -= pt[j][i];
          if (inside && first && p.dshift_in && on[j]) store4<T>(p.dshift_in, (size_t)s * width, col[j], pt[j]);
          if (inside && t + 1 == end && p.dshift_out) {
            float d[4];
            load4<T>(p.dshift_out, (size_t)s * width, col[j], d);
#pragma unroll
            for (int i = 0; i < 4; ++i) qt[j][i] += d[i];
          }
        }
      }
      // the next turn's planes (row t1's too, unless no token is there)
      if (t + 1 <= t1 && t + 1 < p.seq.tokens) fetch(t + 1);
      float v[4] = {};
      if (t > t0) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
          if (on[j])
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float dh = first ? q[j][i] : q[j][i] + pt[j][i];
              dgamma[j][i] = fmaf(dh, n[j][i], dgamma[j][i]);
              dbeta[j][i] += dh;
              q[j][i] = dh * gamma[j][i];
              v[0] += q[j][i];
              v[1] = fmaf(q[j][i], n[j][i], v[1]);
            }
      }
      float x[NV][4];
      if (t + 1 < t1) {
#pragma unroll
        for (int j = 0; j < NV; ++j) up4<T>(r1[j], x[j]);
        v[2] = part_squares<NV>(x, on, mean1);
      }
      if (t + 2 < t1) {
#pragma unroll
        for (int j = 0; j < NV; ++j) up4<T>(rx[j], x[j]);
        v[3] = part_sum<NV>(x, on);
      }
      block_sum(v, red, buf, waves);
      if (t > t0) {
        // finish row t - 1
        const float m1 = v[0] * inv, m2 = v[1] * inv;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
          if (!on[j]) continue;
          const size_t at = (size_t)(t - 1) * p.ld;
          float d[4] = {};
          if (p.dx_out) up4<T>(rup[j], d);
#pragma unroll
          for (int i = 0; i < 4; ++i) d[i] = fmaf(q[j][i] - m1 - n[j][i] * m2, rstd, d[i]);
          store4<T>(p.dx, at, col[j], d);
          if (p.ddelta) {
#pragma unroll
            for (int i = 0; i < 4; ++i) d[i] *= p.alpha;
            store4<T>(p.ddelta, at, col[j], d);
          }
        }
      }
      if (inside && p.dx_out)
#pragma unroll
        for (int j = 0; j < NV; ++j) rup[j] = raw4(p.dx_out, (size_t)t * p.ld, col[j]);
      rstd = rstdt;
      rstdt = rsqrtf(v[2] * inv + p.eps);
#pragma unroll
      for (int j = 0; j < NV; ++j) {
        up4<T>(r1[j], x[j]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          n[j][i] = nt[j][i];
          q[j][i] = qt[j][i];
          nt[j][i] = (x[j][i] - mean1) * rstdt;
        }
        r1[j] = rx[j];
        if (t + 3 < t1) rx[j] = raw4(p.x, (size_t)(t + 3) * p.ld, col[j]);
      }
      mean1 = v[3] * inv;
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
        *(uint2*)((uint16_t*)p.dshift_in + at) =
            p.dshift_out ? *(const uint2*)((const uint16_t*)p.dshift_out + at) : make_uint2(0, 0);
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
    };
    put(p.dgamma, 0, dgamma[j]);
    put(p.dbeta, 1, dbeta[j]);
#pragma unroll
    for (int m = 0; m < NM; ++m)
      if (m < p.nmix) put(p.dmu + (size_t)m * width, 2 + m, dmu[m][j]);
  }
}

namespace {
template <typename T, int NV, int NM>
hipError_t start_back(const ShiftNormBack& p, int rows, dim3 grid, dim3 block, hipStream_t st) {
  // mu in LDS up to six planes of 4096 channels; a larger one stays in L2
  constexpr int kMost = 96 * 1024;
  const size_t bytes = (size_t)p.nmix * p.width * 4;
  const bool mu_lds = bytes <= kMost;
  static const hipError_t attr =
      hipFuncSetAttribute((const void*)shift_norm_back_kernel<T, NV, NM>, hipFuncAttributeMaxDynamicSharedMemorySize, kMost);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL((shift_norm_back_kernel<T, NV, NM>), grid, block, mu_lds ? bytes : 0, st, p, rows, mu_lds);
  return hipGetLastError();
}
template <typename T, int NV>
hipError_t start_back(const ShiftNormBack& p, int rows, dim3 grid, dim3 block, hipStream_t st) {
  if (p.nmix == 1) return start_back<T, NV, 1>(p, rows, grid, block, st);
  if (p.nmix <= 6) return start_back<T, NV, 6>(p, rows, grid, block, st);
  return start_back<T, NV, 8>(p, rows, grid, block, st);
}
}  // namespace

hipError_t launch_shift_norm_back(const ShiftNormBack& p, bool bf16, hipStream_t st) {
  const int nv = p.width > 4096 ? 2 : 1;
  const size_t row = (size_t)(2 + p.nmix) * p.width * 4;
  // two workgroups per compute unit (with the sums after it 70 us for 4096
  // tokens of width 2048; 256 workgroups 71, 768 97, 1024 90)
  int64_t groups = 512;
  const int64_t fit = p.parts ? (int64_t)(p.parts_bytes / row) : 0;
  if (groups > fit) groups = fit;
  if (groups > p.seq.tokens) groups = p.seq.tokens;
  if (groups < 1) groups = 1;
  const int rows = run_rows(p.seq.tokens, (int)groups);
  if (p.seq.tokens > 0) groups = run_count(p.seq.tokens, rows);
  const dim3 grid((unsigned)groups), block((p.width / 4 + nv * 64 - 1) / (nv * 64) * 64);
  const hipError_t e = bf16 ? (nv == 1 ? start_back<BF16, 1>(p, rows, grid, block, st) : start_back<BF16, 2>(p, rows, grid, block, st))
                            : (nv == 1 ? start_back<F16, 1>(p, rows, grid, block, st) : start_back<F16, 2>(p, rows, grid, block, st));
  if (groups == 1 || e != hipSuccess) return e;
  return launch_sum_parts(p.parts, (int)groups, {{p.dgamma, p.dbeta, p.dmu}, {p.width, p.width, p.nmix * p.width}}, st);
}

}  // namespace rq
