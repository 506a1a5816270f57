// Gradient of the state recurrence.  Walking back from dS = dstate_out, with
// u = S_{t-1} a:
//
//   dS += dy r^T,  dr = S_t^T dy,  dk = dS^T v,  dv = dS k,  db = dS^T u,
//   du = dS b,  da = S_{t-1}^T du,  dw_j = sum_i dS_ij S_{t-1},ij,
//   dS_{t-1} = dS diag(w) + du a^T,  draw = dw w (-exp(-1/2)) s (1 - s)
//
// with s = sigmoid(raw).  One workgroup per (sequence, head).  A forward pass
// leaves the state before every run of 16 tokens in the workspace; the walk
// back computes the states within each run again into a second part of it.
#include "mix.h"

namespace rq {

namespace {
constexpr int kRun = 16;
constexpr int kState = kHead * kHead;

__device__ __forceinline__ float dot4(float4 a, float4 b) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, a.x * b.x)));
}
__device__ __forceinline__ float4 axpy4(float a, float4 x, float4 y) {
  return make_float4(fmaf(a, x.x, y.x), fmaf(a, x.y, y.y), fmaf(a, x.z, y.z), fmaf(a, x.w, y.w));
}
__device__ __forceinline__ float4 mul4(float4 a, float4 b) {
  return make_float4(a.x * b.x, a.y * b.y, a.z * b.z, a.w * b.w);
}
// over the four row groups of a wave
__device__ __forceinline__ float4 cols_sum(float4 v) {
  v.x += __shfl_xor(v.x, 16); v.y += __shfl_xor(v.y, 16); v.z += __shfl_xor(v.z, 16); v.w += __shfl_xor(v.w, 16);
  v.x += __shfl_xor(v.x, 32); v.y += __shfl_xor(v.y, 32); v.z += __shfl_xor(v.z, 32); v.w += __shfl_xor(v.w, 32);
  return v;
}
}  // namespace

template <typename T>
__global__ void __launch_bounds__(256) time_mix_back_kernel(TimeMixBack b) {
  const TimeMix& p = b.f;
  __shared__ __align__(16) float in[7][kRun][kHead];       // r, decay, k, v, a, b, dy
  __shared__ __align__(16) float part[5][4][kHead];        // dr, dw, dk, da, db of each wave
  __shared__ float res[6][kRun][kHead];                    // dr, dw, dk, dv, da, db
  const int head = blockIdx.x % p.heads, s = blockIdx.x / p.heads;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int begin, end;
  seq_span(p.seq, s, begin, end);
  const size_t state = ((size_t)s * p.heads + head) * kState;
  const int row = wave * 16 + lane / 16, col = lane % 16 * 4;
  const int runs = (end - begin + kRun - 1) / kRun;
  // states before each run: begin / 16 + s is at most the runs of all
  // sequences before this one
  float* before = p.parts + ((size_t)(begin / kRun + s) * p.heads + head) * kState;
  const size_t run_stride = (size_t)p.heads * kState;
  // states before each token of the run at hand
  float* within = p.parts + ((size_t)(p.seq.tokens / kRun + p.seq.nseq) * p.heads + (size_t)blockIdx.x * kRun) * kState;
  const int mine = row * kHead + col;

  const void* src[7] = {p.r, p.w, p.k, p.v, p.a, p.b, b.dy};
  auto stage = [&](int t0, int n) {
    __syncthreads();
    for (int i = threadIdx.x; i < 7 * n * 8; i += 256) {
      const int which = i / (n * 8), t = i / 8 % n, c = i % 8 * 8;
      float f[8];
      load8<T>(src[which], (size_t)(t0 + t) * p.ld + head * kHead + c, f);
      if (which == 1)
#pragma unroll
        for (int q = 0; q < 8; ++q) f[q] = __builtin_amdgcn_exp2f(log2_decay(f[q]));
      *(float4*)&in[which][t][c] = *(const float4*)f;
      *(float4*)&in[which][t][c + 4] = *(const float4*)(f + 4);
    }
    __syncthreads();
  };
  float4 S[4];
  auto step = [&](int t) {
    const float4 w = *(const float4*)&in[1][t][col], k = *(const float4*)&in[2][t][col];
    const float4 a = *(const float4*)&in[4][t][col], bb = *(const float4*)&in[5][t][col];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float u = row_sum(dot4(S[j], a));
      S[j] = axpy4(u, bb, axpy4(in[3][t][row + 4 * j], k, mul4(S[j], w)));
    }
  };
#pragma unroll
  for (int j = 0; j < 4; ++j)
    S[j] = p.state_in ? *(const float4*)(p.state_in + state + mine + 4 * j * kHead) : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = 0; c < runs; ++c) {
    const int t0 = begin + c * kRun, n = min(kRun, end - t0);
#pragma unroll
    for (int j = 0; j < 4; ++j) *(float4*)(before + c * run_stride + mine + 4 * j * kHead) = S[j];
    if (c + 1 == runs) break;
    stage(t0, n);
    for (int t = 0; t < n; ++t) step(t);
  }
  float4 D[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    D[j] = b.dstate_out ? *(const float4*)(b.dstate_out + state + mine + 4 * j * kHead) : make_float4(0.f, 0.f, 0.f, 0.f);
  for (int c = runs - 1; c >= 0; --c) {
    const int t0 = begin + c * kRun, n = min(kRun, end - t0);
    stage(t0, n);
    // each lane stores and loads its own elements only
#pragma unroll
    for (int j = 0; j < 4; ++j) S[j] = *(const float4*)(before + c * run_stride + mine + 4 * j * kHead);
    for (int t = 0; t < n; ++t) {
#pragma unroll
      for (int j = 0; j < 4; ++j) *(float4*)(within + t * kState + mine + 4 * j * kHead) = S[j];
      step(t);
    }
    for (int t = n - 1; t >= 0; --t) {
      const float4 r = *(const float4*)&in[0][t][col], w = *(const float4*)&in[1][t][col];
      const float4 k = *(const float4*)&in[2][t][col], a = *(const float4*)&in[4][t][col];
      const float4 bb = *(const float4*)&in[5][t][col];
      const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
      float4 dr = zero, dw = zero, dk = zero, da = zero, db = zero;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float dy = in[6][t][row + 4 * j], v = in[3][t][row + 4 * j];
        dr = axpy4(dy, S[j], dr);
        D[j] = axpy4(dy, r, D[j]);
        S[j] = *(const float4*)(within + t * kState + mine + 4 * j * kHead);  // the state before
        const float u = row_sum(dot4(S[j], a));
        const float du = row_sum(dot4(D[j], bb)), dv = row_sum(dot4(D[j], k));
        dk = axpy4(v, D[j], dk);
        db = axpy4(u, D[j], db);
        da = axpy4(du, S[j], da);
        const float4 ds = mul4(D[j], S[j]);
        dw = make_float4(dw.x + ds.x, dw.y + ds.y, dw.z + ds.z, dw.w + ds.w);
        D[j] = axpy4(du, a, mul4(D[j], w));
        if (lane % 16 == 0) res[3][t][row + 4 * j] = dv;
      }
      float4 all[5] = {dr, dw, dk, da, db};
#pragma unroll
      for (int q = 0; q < 5; ++q) {
        const float4 v = cols_sum(all[q]);
        if (lane < 16) *(float4*)&part[q][wave][col] = v;
      }
      __syncthreads();
      for (int i = threadIdx.x; i < 5 * kHead; i += 256) {
        const int q = i / kHead, c2 = i % kHead;
        const float v = ((part[q][0][c2] + part[q][1][c2]) + part[q][2][c2]) + part[q][3][c2];
        res[q < 3 ? q : q + 1][t][c2] = v;
      }
      __syncthreads();
    }
    void* dst[6] = {b.dr, b.dw, b.dk, b.dv, b.da, b.db};
    for (int i = threadIdx.x; i < 6 * n * 8; i += 256) {
      const int which = i / (n * 8), t = i / 8 % n, c2 = i % 8 * 8;
      float f[8];
      const size_t at = (size_t)(t0 + t) * p.ld + head * kHead + c2;
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = res[which][t][c2 + q];
      if (which == 1) {
        float raw[8];
        load8<T>(p.w, at, raw);
#pragma unroll
        for (int q = 0; q < 8; ++q) {
          const float sg = sigmoid_f32(raw[q]);
          f[q] *= in[1][t][c2 + q] * -kDecay * sg * (1.f - sg);
        }
      }
      store8<T>(dst[which], at, f);
    }
  }
  if (b.dstate_in)
#pragma unroll
    for (int j = 0; j < 4; ++j) *(float4*)(b.dstate_in + state + mine + 4 * j * kHead) = D[j];
}

size_t time_mix_back_bytes(int64_t tokens, int64_t heads, int64_t nseq) {
  return ((size_t)(tokens / kRun + nseq) + (size_t)nseq * kRun) * heads * kState * 4;
}

hipError_t launch_time_mix_back(const TimeMixBack& b, bool bf16, hipStream_t st) {
  const dim3 grid((unsigned)b.f.seq.nseq * b.f.heads), block(256);
  if (bf16)
    hipLaunchKernelGGL(time_mix_back_kernel<BF16>, grid, block, 0, st, b);
  else
    hipLaunchKernelGGL(time_mix_back_kernel<F16>, grid, block, 0, st, b);
  return hipGetLastError();
}

}  // namespace rq
