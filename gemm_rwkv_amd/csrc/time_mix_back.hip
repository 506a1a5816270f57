// Gradient of the state recurrence, in chunks of 16 tokens (time_mix_chunk.h
// for the chunk's products and the notation).
//
// Two chains run along each sequence, independent of each other: the state S
// forward, and the gradient E of the state back.  The first launch walks both
// at once, a workgroup each, and leaves for every chunk the state before it,
// D = E diag(exp L_15) after it, U and Z.  With those the chunks no longer
// depend on each other, and the second launch makes the gradients of all of
// them at once:
//
//   dQb = tril(dY U^T)   dQk = tril(dY V^T)   dAb, dAk = strictly lower Z U^T, Z V^T
//   dR = dY S + dQb B + dQk K        dA = Z S + dAb B + dAk K
//   dB = U D + dQb^T R + dAb^T A     dK = V D + dQk^T R + dAk^T A
//   dV = Qk^T dY + Ak^T Z + K D^T
//
// each times the decay that scaled its input, and for the decays
//   dL_t = R dR - B dB - K dK + (A dA)_{t+1},
//   dL_15 = ... + sum_v D o (S + U^T B + V^T K),   dlog w_t = sum_{s>=t} dL_s.
// What a token reads of itself (the diagonals of dQb and dQk) is in R dR and in
// B dB and K dK alike and no decay lies between: it is added after dL, so that
// it cancels exactly.
#include "mix.h"
#include "time_mix_chunk.h"

namespace rq {

namespace {
constexpr int kState = kHead * kHead;

// Chunk c of sequence s is number begin / 16 + s + c of all chunks: at least
// one past every chunk of the sequences before it.
__device__ __forceinline__ int first_chunk(int begin, int s) { return begin / kChunk + s; }

// The sequence of chunk number j, and its place there; false for a number
// between two sequences.
__device__ __forceinline__ bool find_chunk(const Sequences& q, int j, int& begin, int& end, int& c) {
  int lo = 0, hi = q.nseq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    seq_span(q, mid, begin, end);
    if (first_chunk(begin, mid) <= j) lo = mid; else hi = mid - 1;
  }
  seq_span(q, lo, begin, end);
  c = j - first_chunk(begin, lo);
  return c >= 0 && c < (end - begin + kChunk - 1) / kChunk;
}

// What the chains leave per chunk and head.
struct Chain {
  float* S;  // [chunks][heads][64 v][64 k]
  float* D;
  float* U;  // [chunks][heads][16 t][64 v]
  float* Z;
};
}  // namespace

// A workgroup per sequence, head and direction.  Bound by the walk's chain and,
// where all compute units have one, by what it writes: 4 sequences of 1024
// tokens and 32 heads take 124 us.  (When it took 126, 94 without writing the
// states, and 107 keeping every second chunk's, which cost the second launch
// more.)
template <typename T>
__global__ void __launch_bounds__(64 * kWalkWaves) time_mix_chains_kernel(TimeMixBack b, Chain to) {
  extern __shared__ __align__(16) uint8_t lds[];
  ChunkLds& sh = *(ChunkLds*)lds;
  const bool back = blockIdx.x & 1;
  const int chain = blockIdx.x >> 1;
  TimeMix p = b.f;
  const int head = chain % p.heads, s = chain / p.heads;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  int begin, end;
  seq_span(p.seq, s, begin, end);
  const int chunks = (end - begin + kChunk - 1) / kChunk;
  clear_counts(sh);
  if (wave >= 4) {
    if (back) {
      p.v = b.dy;
      prepare_chunks<T, false, true>(p, begin, end, sh, head, 4, wave, lane);
    } else {
      prepare_chunks<T, false, false>(p, begin, end, sh, head, 4, wave, lane);
    }
    return;
  }
  const int q = lane & 15, g = lane >> 4;
  const size_t state = ((size_t)s * p.heads + head) * kState;
  const size_t at = ((size_t)first_chunk(begin, s) * p.heads + head);
  auto out = [](int, float4v) {};
  auto steps = [](int) { return float4v{}; };
  auto rows = [&](float* base, int c, float4v u) {
    float* to = base + (at + (size_t)c * p.heads) * (kChunk * kHead) + 4 * g * kHead + 16 * wave + q;
#pragma unroll
    for (int i = 0; i < 4; ++i) to[i * kHead] = u[i];
  };
  ChunkState st;
  if (!back) {
    st.load(p.state_in ? p.state_in + state : nullptr, wave, lane);
    walk_chunks<T, false, false>(
        st, chunks, sh, wave, lane, ~0u, [&](int c) { st.store(to.S + (at + (size_t)c * p.heads) * kState, wave, lane); },
        [&](int c, float4v u) { rows(to.U, c, u); }, out, steps);
  } else {
    st.load(b.dstate_out ? b.dstate_out + state : nullptr, wave, lane);
    walk_chunks<T, false, true>(
        st, chunks, sh, wave, lane, ~0u,
        [&](int c) { st.store(to.D + (at + (size_t)(chunks - 1 - c) * p.heads) * kState, wave, lane); },
        [&](int c, float4v u) { rows(to.Z, chunks - 1 - c, u); }, out, steps);
    if (b.dstate_in) st.store(b.dstate_in + state, wave, lane);
  }
}

namespace {
constexpr int kPad = 68;  // floats of a row of decays: 16-byte writes of 16 rows spread over the banks

// Operands of a chunk's gradients: rows [16][64] in blocks of eight channels
// (row_block) and the 16x16 matrices as operands, in bf16 terms: three for
// fp32 values, NV for V and dY, which those hold exactly.
template <int NV>
struct GradLds {
  uint4 a[3][128], r[3][128], b[3][128], k[3][128], u[3][128], z[3][128], dy[NV][128], v[NV][128];
  float fall[kChunk][kPad], slope[kChunk][kPad];  // decays from the chunk's start; the sigmoid's slope
  float diag[2][kChunk];  // of dQb and dQk, which are without it below
  uint4 mr[3][64];  // (dQb, dQk)
  uint4 ma[3][64];  // (dAb, dAk)
  uint4 mb[3][64];  // (dQb^T, dAb^T)
  uint4 mk[3][64];  // (dQk^T, dAk^T)
  uint4 mv[3][64];  // (Qk^T, Ak^T)
};

// The term products that count, smallest first: those above 2^-24.
template <int NA, int NB>
__device__ __forceinline__ float4v mul_terms(const uint4* a, const uint4* b, float4v c) {
#pragma unroll
  for (int sum = 2; sum >= 0; --sum)
#pragma unroll
    for (int i = 0; i < NA; ++i)
      if (sum - i >= 0 && sum - i < NB) c = mfma32(a[i], b[sum - i], c);
  return c;
}

// X Y^T over the 64 channels of two rows' worth of operands in LDS: row 4 g + i
// of X, row q of Y.
template <int NA, int NB>
__device__ __forceinline__ float4v gram_rows(const uint4 (*x)[128], const uint4 (*y)[128], int q, int g) {
  float4v c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int at = row_block(q, 4 * h + g);
    uint4 a[NA], b[NB];
#pragma unroll
    for (int n = 0; n < NA; ++n) a[n] = x[n][at];
#pragma unroll
    for (int n = 0; n < NB; ++n) b[n] = y[n][at];
    c = mul_terms<NA, NB>(a, b, c);
  }
  return c;
}

// Stores a 16x16 result (row 4 g + i, column q) as half `half` of an operand
// whose row is q and whose slot is 4 g + i; entries with KEEP(slot - q) only.
template <typename Keep>
__device__ __forceinline__ void put_half(uint4 (*m)[64], int half, float4v x, int q, int g, int lane, Keep keep) {
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if (!keep(4 * g + i - q)) x[i] = 0.f;
  uint2 t[3];
  split4<3>(x, t);
#pragma unroll
  for (int n = 0; n < 3; ++n) ((uint2*)&m[n][lane])[half] = t[n];
}

// Entry i of four rows of an operand half (x, y words).
__device__ __forceinline__ float entry(const uint4* t, int half, int i) {
  float s = 0.f;
#pragma unroll
  for (int n = 0; n < 3; ++n) {
    const uint32_t w = half ? (i < 2 ? t[n].z : t[n].w) : (i < 2 ? t[n].x : t[n].y);
    s += BF16::up((i & 1) ? w >> 16 : w & 0xffffu);
  }
  return s;
}
}  // namespace

// The gradients of one chunk and head: four waves, of which wave w takes
// channels 16 w .. 16 w + 15.  For 4 sequences of 1024 tokens and 32 heads it
// reads the 335 MB that the chains leave and moves 220 MB of rows, in 167 us,
// 3.3 TB/s: its 65 KB of LDS (three terms of every row, so that the gradients
// are fp32's until they are rounded) leave two workgroups per compute unit to
// wait for memory.  Three, with two terms, took 134 us.
template <typename T>
__global__ void __launch_bounds__(256, 2) time_mix_grad_kernel(TimeMixBack b, Chain from) {
  constexpr int NV = ChunkHead<T, false>::kV;
  __shared__ __align__(16) GradLds<NV> sh;
  const TimeMix& p = b.f;
  const int head = blockIdx.x % p.heads, j = blockIdx.x / p.heads;
  int begin, end, c;
  if (!find_chunk(p.seq, j, begin, end, c)) return;
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int q = lane & 15, g = lane >> 4;
  const int t0 = begin + c * kChunk, n = min(kChunk, end - t0);
  const size_t at = (size_t)j * p.heads + head;

  // S and D with this wave's columns of k, and D with its rows of v
  float S[16], D[16], Dv[16];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const size_t e = at * kState + (32 * h + 8 * g + i) * kHead + 16 * wave + q;
      S[8 * h + i] = from.S[e];
      D[8 * h + i] = from.D[e];
    }
    load8f(from.D + at * kState + (16 * wave + q) * kHead + 32 * h + 8 * g, Dv + 8 * h);
  }

  // rows: token q, channels 16 w + 4 g .. + 3
  {
    const bool held = q < n;
    const size_t e = (size_t)(t0 + q) * p.ld + head * kHead + 16 * wave + 4 * g;
    const void* src[7] = {p.r, p.w, p.k, p.a, p.b, p.v, b.dy};
    uint2 raw[7];
#pragma unroll
    for (int i = 0; i < 7; ++i) {
      const uint32_t other = i == 1 ? T::kMinusInf2 : 0u;
      raw[i] = held ? *(const uint2*)((const uint16_t*)src[i] + e) : make_uint2(other, other);
    }
    const size_t er = at * (kChunk * kHead) + q * kHead + 16 * wave + 4 * g;
    const float4v u = *(const float4v*)(from.U + er), z = *(const float4v*)(from.Z + er);
    float x[4], fall[4], before[4], slope[4], grow[4];
    auto up4 = [&](int i) {
      up2<T>(raw[i].x, x);
      up2<T>(raw[i].y, x + 2);
    };
    up4(1);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float sig = sigmoid_f32(x[i]);
      slope[i] = sig * sigmoid_f32(-x[i]);  // not sig (1 - sig), which cancels as sig nears 1
      float l = -(kDecay * kLog2e) * sig;
      l += dpp<0x111>(l);
      l += dpp<0x112>(l);
      l += dpp<0x114>(l);
      l += dpp<0x118>(l);
      fall[i] = __builtin_amdgcn_exp2f(l);
      grow[i] = __builtin_amdgcn_exp2f(-l);
      before[i] = dpp_or<0x111>(1.f, fall[i]);
    }
    *(float4v*)&sh.fall[q][16 * wave + 4 * g] = float4v{fall[0], fall[1], fall[2], fall[3]};
    *(float4v*)&sh.slope[q][16 * wave + 4 * g] = float4v{slope[0], slope[1], slope[2], slope[3]};
    const int block = row_block(q, 2 * wave + (g >> 1)), half = g & 1;
    auto put3 = [&](uint4(*m)[128], float4v f) {
      uint2 t[3];
      split4<3>(f, t);
#pragma unroll
      for (int i = 0; i < 3; ++i) ((uint2*)&m[i][block])[half] = t[i];
    };
    auto put_scaled = [&](uint4(*m)[128], int i, const float* s) {
      up4(i);
      put3(m, float4v{x[0] * s[0], x[1] * s[1], x[2] * s[2], x[3] * s[3]});
    };
    put_scaled(sh.r, 0, fall);
    put_scaled(sh.k, 2, grow);
    put_scaled(sh.a, 3, before);
    put_scaled(sh.b, 4, grow);
    put3(sh.u, u);
    put3(sh.z, z);
#pragma unroll
    for (int i = 5; i < 7; ++i) {
      uint4(*m)[128] = i == 5 ? sh.v : sh.dy;
      if (NV == 1) {
        ((uint2*)&m[0][block])[half] = raw[i];
      } else {
        up4(i);
        uint2 t[2];
        split4<2>(float4v{x[0], x[1], x[2], x[3]}, t);
#pragma unroll
        for (int n = 0; n < NV; ++n) ((uint2*)&m[n][block])[half] = t[n];
      }
    }
  }
  __syncthreads();

  // the 16x16 matrices, both ways round
  auto strict = [](int d) { return d < 0; };          // slot < row
  auto upper = [](int d) { return d >= 0; };
  auto strict_upper = [](int d) { return d > 0; };
  auto put_diag = [&](float* to, float4v x) {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * g + i == q) to[q] = x[i];
  };
  if (wave == 0) {
    const float4v x = gram_rows<3, NV>(sh.u, sh.dy, q, g);
    put_diag(sh.diag[0], x);
    put_half(sh.mr, 0, x, q, g, lane, strict);
    put_half(sh.mb, 0, gram_rows<NV, 3>(sh.dy, sh.u, q, g), q, g, lane, strict_upper);
  } else if (wave == 1) {
    const float4v x = gram_rows<NV, NV>(sh.v, sh.dy, q, g);
    put_diag(sh.diag[1], x);
    put_half(sh.mr, 1, x, q, g, lane, strict);
    put_half(sh.mk, 0, gram_rows<NV, NV>(sh.dy, sh.v, q, g), q, g, lane, strict_upper);
    put_half(sh.mv, 0, gram_rows<3, 3>(sh.r, sh.k, q, g), q, g, lane, upper);
  } else if (wave == 2) {
    put_half(sh.ma, 0, gram_rows<3, 3>(sh.u, sh.z, q, g), q, g, lane, strict);
    put_half(sh.mb, 1, gram_rows<3, 3>(sh.z, sh.u, q, g), q, g, lane, strict_upper);
  } else {
    put_half(sh.ma, 1, gram_rows<NV, 3>(sh.v, sh.z, q, g), q, g, lane, strict);
    put_half(sh.mk, 1, gram_rows<3, NV>(sh.z, sh.v, q, g), q, g, lane, strict_upper);
    put_half(sh.mv, 1, gram_rows<3, 3>(sh.a, sh.k, q, g), q, g, lane, strict_upper);
  }
  __syncthreads();

  const float4v zero = {0.f, 0.f, 0.f, 0.f};
  float4v dr = zero, da = zero, db = zero, dk = zero, dv = zero;
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int row = row_block(q, 4 * h + g);
    uint4 m[3], x[3];
    auto rows = [&](const uint4(*from_)[128], int terms) {
#pragma unroll
      for (int n = 0; n < 3; ++n)
        if (n < terms) x[n] = from_[n][row];
    };
    split8<3>(S + 8 * h, m);
    rows(sh.dy, NV);
    dr = mul_terms<NV, 3>(x, m, dr);
    rows(sh.z, 3);
    da = mul_terms<3, 3>(x, m, da);
    split8<3>(D + 8 * h, m);
    rows(sh.u, 3);
    db = mul_terms<3, 3>(x, m, db);
    rows(sh.v, NV);
    dk = mul_terms<NV, 3>(x, m, dk);
    split8<3>(Dv + 8 * h, m);
    rows(sh.k, 3);
    dv = mul_terms<3, 3>(x, m, dv);
  }
  const int ch = 16 * wave + 4 * (q & 3);
  uint4 bk[3], ra[3], yz[3], m[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    bk[i] = pair(rows4(sh.b[i], g, q, ch), rows4(sh.k[i], g, q, ch));
    ra[i] = pair(rows4(sh.r[i], g, q, ch), rows4(sh.a[i], g, q, ch));
    yz[i] = pair(i < NV ? rows4(sh.dy[i < NV ? i : 0], g, q, ch) : make_uint2(0, 0), rows4(sh.z[i], g, q, ch));
  }
  // sum_v D o S and the chunk's own part of it, before dB and dK get the rest
  float last = 0.f;
#pragma unroll
  for (int i = 0; i < 16; ++i) last = fmaf(S[i], D[i], last);
  float4v R, A, B, K;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    R[i] = entry(ra, 0, i);
    A[i] = entry(ra, 1, i);
    B[i] = entry(bk, 0, i);
    K[i] = entry(bk, 1, i);
    last = fmaf(B[i], db[i], fmaf(K[i], dk[i], last));
  }
  last += __shfl_xor(last, 16);
  last += __shfl_xor(last, 32);
  auto mats = [&](const uint4(*x)[64]) {
#pragma unroll
    for (int n = 0; n < 3; ++n) m[n] = x[n][lane];
  };
  mats(sh.mr);
  dr = mul_terms<3, 3>(m, bk, dr);
  mats(sh.ma);
  da = mul_terms<3, 3>(m, bk, da);
  mats(sh.mb);
  db = mul_terms<3, 3>(m, ra, db);
  mats(sh.mk);
  dk = mul_terms<3, 3>(m, ra, dk);
  mats(sh.mv);
  dv = mul_terms<3, 3>(m, yz, dv);

  // decays: dL, then its sums from the end; lane (g, q) has tokens 4 g + i of
  // channel 16 w + q
  float4v dl = R * dr - B * db - K * dk;
  const float4v next = A * da;
  const float4v mb = *(const float4v*)&sh.diag[0][4 * g], mk = *(const float4v*)&sh.diag[1][4 * g];
  dr += mb * B + mk * K;
  db += mb * R;
  dk += mk * R;
  const float up = __shfl_down(next[0], 16);
  dl[0] += next[1];
  dl[1] += next[2];
  dl[2] += next[3];
  dl[3] += g == 3 ? last : up;
  dl[2] += dl[3];
  dl[1] += dl[2];
  dl[0] += dl[1];
  const float all = dl[0];
  float after = 0.f;
#pragma unroll
  for (int i = 1; i < 4; ++i) {
    const float x = __shfl_down(all, 16 * i);
    if (g + i < 4) after += x;
  }
  float4v dw;
  {
    const float* fall = &sh.fall[4 * g][16 * wave + q];
    const float* slope = &sh.slope[4 * g][16 * wave + q];
    float f = g ? fall[-kPad] : 1.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      dw[i] = (dl[i] + after) * (-kDecay * slope[i * kPad]);
      da[i] *= f;
      f = fall[i * kPad];
      dr[i] *= f;
      f = fall[i * kPad];
      const float grow = __builtin_amdgcn_rcpf(f);
      db[i] *= grow;
      dk[i] *= grow;
    }
  }
  // through LDS to whole rows; the row operands are done with
  __syncthreads();
  uint16_t* out = (uint16_t*)&sh.a[0][0];  // [6][16][64]
  static_assert(sizeof(sh.a) + sizeof(sh.r) >= 6 * kChunk * kHead * 2, "outputs fit");
  const float4v all6[6] = {dr, dw, dk, dv, da, db};
#pragma unroll
  for (int o = 0; o < 6; ++o)
#pragma unroll
    for (int i = 0; i < 4; ++i)
      out[(o * kChunk + 4 * g + i) * kHead + 16 * wave + q] = (uint16_t)T::down2(all6[o][i], 0.f);
  __syncthreads();
  void* dst[6] = {b.dr, b.dw, b.dk, b.dv, b.da, b.db};
#pragma unroll
  for (int o = 0; o < 6; o += 2) {
    const int which = o + (threadIdx.x >> 7), t = (threadIdx.x >> 3) & 15, c8 = threadIdx.x & 7;
    if (t < n)
      *(uint4*)((uint16_t*)(threadIdx.x >> 7 ? dst[o + 1] : dst[o]) + (size_t)(t0 + t) * p.ld + head * kHead + 8 * c8) =
          *(const uint4*)(out + (which * kChunk + t) * kHead + 8 * c8);
  }
}

namespace {
size_t chunk_slots(int64_t tokens, int64_t nseq) { return (size_t)(tokens / kChunk + nseq); }
}  // namespace

size_t time_mix_back_bytes(int64_t tokens, int64_t heads, int64_t nseq) {
  return chunk_slots(tokens, nseq) * heads * (2 * kState + 2 * kChunk * kHead) * 4;
}

namespace {
template <typename T>
hipError_t start_back(const TimeMixBack& b, hipStream_t st) {
  static const hipError_t attr = allow_lds(time_mix_chains_kernel<T>);
  if (attr != hipSuccess) return attr;
  const size_t n = chunk_slots(b.f.seq.tokens, b.f.seq.nseq) * b.f.heads;
  Chain c;
  c.S = b.f.parts;
  c.D = c.S + n * kState;
  c.U = c.D + n * kState;
  c.Z = c.U + n * kChunk * kHead;
  hipLaunchKernelGGL(time_mix_chains_kernel<T>, dim3(2u * b.f.seq.nseq * b.f.heads), dim3(64 * kWalkWaves), sizeof(ChunkLds), st, b,
                     c);
  if (b.f.seq.tokens > 0)
    hipLaunchKernelGGL(time_mix_grad_kernel<T>, dim3((unsigned)n), dim3(256), 0, st, b, c);
  return hipGetLastError();
}
}  // namespace

hipError_t launch_time_mix_back(const TimeMixBack& b, bool bf16, hipStream_t st) {
  return bf16 ? start_back<BF16>(b, st) : start_back<F16>(b, st);
}

}  // namespace rq
