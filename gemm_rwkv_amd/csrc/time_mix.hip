// The state recurrence of RWKV-7's time mixing, per head of 64:
//
//   S_t = S_{t-1} diag(w_t) + (S_{t-1} a_t) b_t^T + v_t k_t^T,   y_t = S_t r_t
//
// with S[64 v][64 k] in fp32 and w_t = exp(-exp(-1/2) sigmoid(raw_t)).
//
// step kernel: one workgroup of four waves per (sequence, head), token by
// token in fp32.  The rows of S are independent of each other, so a wave owns
// sixteen of them; a row lies across sixteen lanes, four columns each, and the
// sums S a and S r are four lane rotations.  A run of up to sixteen tokens is
// staged in LDS as fp32.
#include "mix.h"

namespace rq {

namespace {
constexpr int kRun = 16;  // tokens staged at once
}

template <typename T>
__global__ void __launch_bounds__(256) time_mix_step_kernel(TimeMix p) {
  // r, w (as decay), k, v, a, b of the run, then y
  __shared__ __align__(16) float in[6][kRun][kHead];
  __shared__ float out[kRun][kHead];
  const int head = blockIdx.x % p.heads, s = blockIdx.x / p.heads;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int begin, end;
  seq_span(p.seq, s, begin, end);
  const int slot = slot_of(p.slots, s);
  const size_t state = ((size_t)(slot < 0 ? 0 : slot) * p.heads + head) * kHead * kHead;
  // rows row + 4 j, columns col .. col + 3
  const int row = wave * 16 + lane / 16, col = lane % 16 * 4;
  float4 S[4];
#pragma unroll
  for (int j = 0; j < 4; ++j)
    S[j] = p.state_in && slot >= 0 ? *(const float4*)(p.state_in + state + (row + 4 * j) * kHead + col)
                                   : make_float4(0.f, 0.f, 0.f, 0.f);
  const void* src[6] = {p.r, p.w, p.k, p.v, p.a, p.b};
  for (int t0 = begin; t0 < end; t0 += kRun) {
    const int n = min(kRun, end - t0);
    // 16-byte pieces: array, token, eighth of the head
    for (int i = threadIdx.x; i < 6 * n * 8; i += 256) {
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
    for (int t = 0; t < n; ++t) {
      const float4 r = *(const float4*)&in[0][t][col], w = *(const float4*)&in[1][t][col];
      const float4 k = *(const float4*)&in[2][t][col], a = *(const float4*)&in[4][t][col];
      const float4 b = *(const float4*)&in[5][t][col];
      float u[4], y[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        u[j] = fmaf(S[j].w, a.w, fmaf(S[j].z, a.z, fmaf(S[j].y, a.y, S[j].x * a.x)));
#pragma unroll
      for (int j = 0; j < 4; ++j) u[j] = row_sum(u[j]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const float v = in[3][t][row + 4 * j];
        S[j].x = fmaf(S[j].x, w.x, fmaf(u[j], b.x, v * k.x));
        S[j].y = fmaf(S[j].y, w.y, fmaf(u[j], b.y, v * k.y));
        S[j].z = fmaf(S[j].z, w.z, fmaf(u[j], b.z, v * k.z));
        S[j].w = fmaf(S[j].w, w.w, fmaf(u[j], b.w, v * k.w));
        y[j] = fmaf(S[j].w, r.w, fmaf(S[j].z, r.z, fmaf(S[j].y, r.y, S[j].x * r.x)));
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) y[j] = row_sum(y[j]);
      if (lane % 16 == 0)
#pragma unroll
        for (int j = 0; j < 4; ++j) out[t][row + 4 * j] = y[j];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < n * 8; i += 256) {
      const int t = i / 8, c = i % 8 * 8;
      float f[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) f[q] = out[t][c + q];
      store8<T>(p.y, (size_t)(t0 + t) * p.ldy + head * kHead + c, f);
    }
  }
  if (p.state_out && slot >= 0)
#pragma unroll
    for (int j = 0; j < 4; ++j) *(float4*)(p.state_out + state + (row + 4 * j) * kHead + col) = S[j];
}

hipError_t launch_time_mix(const TimeMix& p, bool bf16, hipStream_t st) {
  const dim3 grid((unsigned)p.seq.nseq * p.heads), block(256);
  if (bf16)
    hipLaunchKernelGGL(time_mix_step_kernel<BF16>, grid, block, 0, st, p);
  else
    hipLaunchKernelGGL(time_mix_step_kernel<F16>, grid, block, 0, st, p);
  return hipGetLastError();
}

}  // namespace rq
