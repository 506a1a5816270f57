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
#include "time_mix_chunk.h"

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

// chunk kernel: one workgroup of eight waves per (sequence, head).  Waves 0-3
// hold the state, sixteen channels of v each, and take it from chunk to chunk;
// waves 4-7 prepare the chunks' operands ahead of them, every fourth chunk
// each, in an LDS buffer of their own.  Two counters per buffer order them:
// `ready` chunks written, and `done` four per chunk read.  Every wait is for a
// count that the other side reaches by itself: a buffer's chunk c waits for
// the readers of chunk c - 4, who wait for nothing later than it.
namespace {
constexpr int kPreps = 4;

struct ChunkLds {
  ChunkOps ops[kPreps];
  int ready[kPreps], done[kPreps];
};

__device__ __forceinline__ void wait_for(int* count, int want) {
  while (__hip_atomic_load(count, __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_WORKGROUP) < want) __builtin_amdgcn_s_sleep(1);
}
__device__ __forceinline__ void signal(int* count, int lane) {
  if (lane == 0) __hip_atomic_fetch_add(count, 1, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_WORKGROUP);
}
}  // namespace

template <typename T>
__global__ void __launch_bounds__(512) time_mix_chunk_kernel(TimeMix p) {
  extern __shared__ __align__(16) uint8_t lds[];
  ChunkLds& sh = *(ChunkLds*)lds;
  const int head = blockIdx.x % p.heads, s = blockIdx.x / p.heads;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int begin, end;
  seq_span(p.seq, s, begin, end);
  const int chunks = (end - begin + kChunk - 1) / kChunk;
  if (threadIdx.x < kPreps) sh.ready[threadIdx.x] = sh.done[threadIdx.x] = 0;
  __syncthreads();
  if (wave >= 4) {
    const int mine = wave - 4;
    ChunkOps& o = sh.ops[mine];
    ChunkPrep<T> prep;
    auto load = [&](int c) { prep.load(p, head, begin + c * kChunk, min(kChunk, end - begin - c * kChunk), lane); };
    if (mine < chunks) load(mine);
    int read = 0;
    for (int c = mine; c < chunks; c += kPreps, read += 4) {
      prep.decays();
      prep.factors();
      prep.grams();
      wait_for(&sh.done[mine], read);
      prep.put_rows(o, lane);
      if (c + kPreps < chunks) load(c + kPreps);
      prep.solve(o, lane);
      signal(&sh.ready[mine], lane);
    }
    return;
  }
  const int slot = slot_of(p.slots, s);
  const size_t state = ((size_t)(slot < 0 ? 0 : slot) * p.heads + head) * kHead * kHead;
  ChunkState<T> st;
  st.load(p.state_in && slot >= 0 ? p.state_in + state : nullptr, wave, lane);
  const int q = lane & 15, g = lane >> 4;
  for (int c = 0; c < chunks; ++c) {
    wait_for(&sh.ready[c % kPreps], c / kPreps + 1);
    const float4v y = st.step(sh.ops[c % kPreps], wave, lane);
    signal(&sh.done[c % kPreps], lane);
    const int t = begin + c * kChunk + 4 * g;
    uint16_t* to = (uint16_t*)p.y + (size_t)t * p.ldy + head * kHead + 16 * wave + q;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t + i < end) to[(size_t)i * p.ldy] = (uint16_t)T::down2(y[i], 0.f);
  }
  if (p.state_out && slot >= 0) st.store(p.state_out + state, wave, lane);
}

namespace {
template <typename T>
hipError_t start_chunks(const TimeMix& p, hipStream_t st) {
  constexpr int kLds = sizeof(ChunkLds);
  static const hipError_t attr = hipFuncSetAttribute((const void*)time_mix_chunk_kernel<T>,
                                                     hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
  if (attr != hipSuccess) return attr;
  hipLaunchKernelGGL(time_mix_chunk_kernel<T>, dim3((unsigned)p.seq.nseq * p.heads), dim3(512), kLds, st, p);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_time_mix(const TimeMix& p, bool bf16, hipStream_t st) {
  const dim3 grid((unsigned)p.seq.nseq * p.heads), block(256);
  if (p.seq.tokens > p.seq.nseq) return bf16 ? start_chunks<BF16>(p, st) : start_chunks<F16>(p, st);
  if (bf16)
    hipLaunchKernelGGL(time_mix_step_kernel<BF16>, grid, block, 0, st, p);
  else
    hipLaunchKernelGGL(time_mix_step_kernel<F16>, grid, block, 0, st, p);
  return hipGetLastError();
}

}  // namespace rq
