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
// staged in LDS as fp32.  For single tokens the states' bytes bound it: 32
// sequences of 64 heads take 13.5 us, 5.1 TB/s (of a pool of 48, part of which
// the memory-side cache delivers; a large copy reaches 5.0).  For longer ones
// the chain from token to token does, 0.4 us each.
//
// chunk kernel: one workgroup of twelve waves per (sequence or segment, head),
// sixteen tokens at a time on matrix instructions (time_mix_chunk.h).
#include <climits>

#include "mix.h"
#include "time_mix_chunk.h"

namespace rq {

namespace {
constexpr int kRun = 16;  // tokens staged at once
}

template <typename T>
__global__ void __launch_bounds__(256) time_mix_step_kernel(TimeMix p, int most) {
  // r, w (as decay), k, v, a, b of the run, then y
  __shared__ __align__(16) float in[6][kRun][kHead];
  __shared__ float out[kRun][kHead];
  const int head = blockIdx.x % p.heads, s = blockIdx.x / p.heads;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int begin, end;
  seq_span(p.seq, s, begin, end);
  if (end - begin > most) return;
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

// Where a workgroup is: a sequence, or a segment of one.
//
// A sequence is a chain of chunks, and few sequences and heads leave most of
// the GPU idle.  Then each is cut into segments.  The state after a segment is
// S P + G, where G is what the segment leaves of a zero state and P its map of
// the 64 channels of k; both are the recurrence itself, started from zeros and
// from the identity (without v).  A first launch makes G and P of every middle
// segment, all at once, and walks the first one, which has its real state, to
// its end; in the second each later segment builds the state before it from
// those and then walks its chunks.  The walk with the map takes half as long
// again, so the first segment is longer, and both launches are level.
struct SegmentSplit {
  int len;        // tokens per segment, a multiple of 16; 0: whole sequences
  int first;      // tokens of a sequence's first segment, another one
  float* states;  // [segments][heads][G, P][64][64]
};

namespace {
struct Segment {
  int seq, begin, end;
  int nth, of;  // which of the sequence's segments
};

// Workgroup `idx`'s segment; false past the last one.
__device__ __forceinline__ bool find_segment(const Sequences& s, const SegmentSplit& split, int idx, Segment& g) {
  if (!split.len) {
    g.seq = idx;
    g.nth = 0;
    g.of = 1;
    seq_span(s, idx, g.begin, g.end);
    return true;
  }
  for (int i = 0; i < s.nseq; ++i) {
    int b, e;
    seq_span(s, i, b, e);
    const int n = 1 + max(0, e - b - split.first + split.len - 1) / split.len;
    if (idx < n) {
      g.seq = i;
      g.nth = idx;
      g.of = n;
      g.begin = idx ? b + split.first + (idx - 1) * split.len : b;
      g.end = min(e, b + split.first + idx * split.len);
      return true;
    }
    idx -= n;
  }
  return false;
}

// Walks a segment's chunks from the state before it, writing y.
template <typename T>
__device__ __forceinline__ void walk_out(const TimeMix& p, const Segment& sg, ChunkState& st, ChunkLds& sh, int head, int wave,
                                         int lane) {
  const int chunks = (sg.end - sg.begin + kChunk - 1) / kChunk;
  const int q = lane & 15, g = lane >> 4;
  uint16_t* to = (uint16_t*)p.y + (size_t)(sg.begin + 4 * g) * p.ldy + head * kHead + 16 * wave + q;
  walk_chunks<T, true, false>(st, chunks, sh, wave, lane, ~0u, [](int) {}, [](int, float4v) {}, [&](int c, float4v y) {
    const int left = sg.end - sg.begin - c * kChunk;
    const uint32_t y01 = T::down2(y[0], y[1]), y23 = T::down2(y[2], y[3]);
    if (left >= kChunk) {
      to[0] = (uint16_t)y01;
      to[p.ldy] = (uint16_t)(y01 >> 16);
      to[2 * (size_t)p.ldy] = (uint16_t)y23;
      to[3 * (size_t)p.ldy] = (uint16_t)(y23 >> 16);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (4 * g + i < left) to[(size_t)i * p.ldy] = (uint16_t)((i < 2 ? y01 : y23) >> (16 * (i & 1)));
    }
    to += (size_t)kChunk * p.ldy;
  }, [&](int c) {
    const int t = sg.begin + c * kChunk;
    return step_tokens<T>(p, head, t, min(kChunk, sg.end - t), st, wave, lane);
  });
}

__device__ __forceinline__ size_t state_at(const TimeMix& p, int slot, int head) {
  return ((size_t)(slot < 0 ? 0 : slot) * p.heads + head) * kHead * kHead;
}
}  // namespace

template <typename T>
__global__ void __launch_bounds__(64 * kWalkWaves) time_mix_chunk_kernel(TimeMix p, SegmentSplit split, int over) {
  extern __shared__ __align__(16) uint8_t lds[];
  ChunkLds& sh = *(ChunkLds*)lds;
  const int head = blockIdx.x % p.heads, idx = blockIdx.x / p.heads;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Segment sg;
  if (!find_segment(p.seq, split, idx, sg) || sg.end - sg.begin <= over || (sg.nth == 0 && sg.of > 1)) return;
  clear_counts(sh);
  if (wave >= 4) {
    prepare_chunks<T, true, false>(p, sg.begin, sg.end, sh, head, 4, wave, lane);
    return;
  }
  const int slot = slot_of(p.slots, sg.seq);
  const size_t state = state_at(p, slot, head);
  ChunkState st;
  if (sg.of == 1) {
    st.load(p.state_in && slot >= 0 ? p.state_in + state : nullptr, wave, lane);
  } else {
    // the segments of this sequence begin at workgroup idx - nth
    const size_t pair = 2 * kHead * kHead, stride = p.heads * pair;
    const float* at = split.states + (size_t)(idx - sg.nth) * stride + head * pair;
    st.load(at, wave, lane);
    for (int i = 1; i < sg.nth; ++i) st.apply(at + i * stride, at + i * stride + kHead * kHead, wave, lane);
  }
  walk_out<T>(p, sg, st, sh, head, wave, lane);
  if (p.state_out && slot >= 0 && sg.nth + 1 == sg.of) st.store(p.state_out + state, wave, lane);
}

// The first segment with its outputs, G and P of the middle ones.
template <typename T>
__global__ void __launch_bounds__(64 * kWalkWaves) time_mix_segment_kernel(TimeMix p, SegmentSplit split) {
  extern __shared__ __align__(16) uint8_t lds[];
  ChunkLds& sh = *(ChunkLds*)lds;
  const int head = blockIdx.x % p.heads, idx = blockIdx.x / p.heads;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Segment sg;
  if (!find_segment(p.seq, split, idx, sg) || sg.nth + 1 == sg.of) return;
  clear_counts(sh);
  const int walkers = sg.nth ? 8 : 4;  // the state, and the map
  if (wave >= walkers) {
    if (sg.nth == 0)
      prepare_chunks<T, true, false>(p, sg.begin, sg.end, sh, head, walkers, wave, lane);
    else
      prepare_chunks<T, false, false>(p, sg.begin, sg.end, sh, head, walkers, wave, lane);
    return;
  }
  float* to = split.states + ((size_t)idx * p.heads + head) * 2 * kHead * kHead;
  ChunkState st;
  if (sg.nth == 0) {
    const int slot = slot_of(p.slots, sg.seq);
    st.load(p.state_in && slot >= 0 ? p.state_in + state_at(p, slot, head) : nullptr, wave, lane);
    walk_out<T>(p, sg, st, sh, head, wave, lane);
    st.store(to, wave, lane);
    return;
  }
  const bool map = wave >= 4;
  const int part = wave & 3;
  if (map)
    st.identity(part, lane);
  else
    st.load(nullptr, part, lane);
  auto none = [](int, float4v) {};
  const int chunks = (sg.end - sg.begin) / kChunk;  // whole: only a last segment is ragged
  walk_chunks<T, false, false>(st, chunks, sh, part, lane, map ? 0u : ~0u, [](int) {}, none, none, [](int) { return float4v{}; });
  st.store(to + (map ? kHead * kHead : 0), part, lane);
}

namespace {
// How sequences are cut: len 0 for not at all.  A middle segment is walked
// three times over, twice by itself and once by its map, so cutting pays only
// from four segments on; they are made to fill the 256 compute units once in
// each launch, and are at least 128 tokens long.  Measured for one sequence,
// whole against cut: 32 heads, 256 tokens 29 and 38 us, 512 49 and 44, 1024 91
// and 52, 4096 340 and 127; 64 heads, 256 tokens 29 and 38, 512 50 and 46, 1024
// 93 and 66, 4096 341 and 187; 128 heads (want 2) 512 tokens 52 and 54, though
// 4096 347 and 286.  First segments of 1 to 2 times the others' length are
// within 5% of each other.
SegmentSplit segment_split(const TimeMix& p) {
  const SegmentSplit whole = {0, 0, nullptr};
  const int64_t chains = (int64_t)p.seq.nseq * p.heads;
  const int64_t mean = p.seq.tokens / p.seq.nseq;
  const int64_t want = 256 / chains;
  if (want < 4 || mean < 4 * 128) return whole;
  // each launch leaves out one segment: first + want * len tokens
  int64_t len = (2 * mean + 2 * want + 2) / (2 * want + 3);
  if (len < 128) len = 128;
  len = (len + kChunk - 1) / kChunk * kChunk;
  const int64_t segments = p.seq.tokens / len + p.seq.nseq;
  if (!p.parts || (size_t)segments * p.heads * 2 * kHead * kHead * 4 > p.parts_bytes) return whole;
  return {(int)len, (int)(len * 3 / 2 / kChunk * kChunk), p.parts};
}

// Sequences of more than `over` tokens (-1: all).
template <typename T>
hipError_t start_chunks(const TimeMix& p, int over, hipStream_t st) {
  static const hipError_t attr = allow_lds(time_mix_chunk_kernel<T>);
  static const hipError_t attr2 = allow_lds(time_mix_segment_kernel<T>);
  if (attr != hipSuccess || attr2 != hipSuccess) return attr != hipSuccess ? attr : attr2;
  const SegmentSplit split = over < 0 ? segment_split(p) : SegmentSplit{0, 0, nullptr};
  const unsigned chains = (unsigned)(split.len ? p.seq.tokens / split.len + p.seq.nseq : p.seq.nseq) * p.heads;
  if (split.len)
    hipLaunchKernelGGL(time_mix_segment_kernel<T>, dim3(chains), dim3(64 * kWalkWaves), sizeof(ChunkLds), st, p, split);
  hipLaunchKernelGGL(time_mix_chunk_kernel<T>, dim3(chains), dim3(64 * kWalkWaves), sizeof(ChunkLds), st, p, split, over);
  return hipGetLastError();
}

template <typename T>
hipError_t start_time_mix(const TimeMix& p, hipStream_t st) {
  // A chunk workgroup has a compute unit to itself and takes 8.3 us for up to
  // 16 tokens, a step workgroup 3 + 0.4 us a token, and five of those share a
  // unit (28 KB of LDS each).  Measured, steps against chunks: 1 sequence of 8
  // tokens 6.1 and 8.2 us, of 12 7.5 and 8.3, of 16 9.1 and 8.3, with 32 as with
  // 64 heads; 32 sequences with 32 heads, of 4 tokens 9.8 and 31, of 16 22 and
  // 31, of 24 31 and 38, of 32 38.5 and 38.9.
  const int64_t chains = (int64_t)p.seq.nseq * p.heads;
  const dim3 grid((unsigned)chains), block(256);
  if (p.seq.tokens <= p.seq.nseq || p.seq.tokens <= 12) {
    hipLaunchKernelGGL(time_mix_step_kernel<T>, grid, block, 0, st, p, INT_MAX);
    return hipGetLastError();
  }
  // Where the chunk workgroups would queue, the short sequences of a batch of
  // mostly short ones take steps and only the others chunks.
  constexpr int kShort = 24;
  if (chains > 256 && p.seq.tokens <= (int64_t)kShort * p.seq.nseq) {
    hipLaunchKernelGGL(time_mix_step_kernel<T>, grid, block, 0, st, p, kShort);
    const hipError_t e = hipGetLastError();
    return e != hipSuccess || p.seq.tokens <= kShort ? e : start_chunks<T>(p, kShort, st);
  }
  return start_chunks<T>(p, -1, st);
}
}  // namespace

hipError_t launch_time_mix(const TimeMix& p, bool bf16, hipStream_t st) {
  return bf16 ? start_time_mix<BF16>(p, st) : start_time_mix<F16>(p, st);
}

}  // namespace rq
