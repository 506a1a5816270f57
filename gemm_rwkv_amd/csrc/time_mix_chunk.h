// The state recurrence in chunks of 16 tokens, on matrix instructions.
//
// With the decays accumulated from the chunk's start, L_t = sum_{s<=t} log w_s,
//   A_t = a_t exp(L_{t-1}),  R_t = r_t exp(L_t),  B_t = b_t exp(-L_t),
//   K_t = k_t exp(-L_t),     u_t = S_{t-1} a_t
// the chunk is five products around the state S before it:
//   U = T (A S^T + Ak V),              T = (1 - Ab)^-1
//   Y = R S^T + Qb U + Qk V
//   S' = (S + U^T B + V^T K) diag(exp L_15)
// with Ab, Ak the strictly lower parts of A B^T, A K^T and Qb, Qk the lower
// parts of R B^T, R K^T (16 x 16).  A decay is at least 0.545, so exp(-L) stays
// below 1.7e4 and every factor is far inside fp32's and bf16's exponents.
//
// Precision.  A matrix instruction multiplies bf16 exactly and adds in fp32,
// so an fp32 factor is cut into three bf16 terms that hold its 24 bits
// exactly, and a product of two such factors keeps the six term products
// above 2^-24 of it: states and outputs are as exact as fp32 before an output
// is rounded.
//
// Lanes.  l = 16 g + q.  A 16x16 result has row 4 g + i in register i and
// column q.  As the B operand of the next product, its registers are the
// slots of contraction index 4 g + i: the A operand only has to name its
// slots alike, so the whole chain from state to state moves nothing between
// lanes.  The state is held as S^T in four tiles; register i of tile n is
// channel k = 32 (n / 2) + 8 g + 4 (n % 2) + i, so that the two tiles of an
// operand hold eight consecutive channels.
#pragma once

#include "mix.h"

namespace rq {

typedef short short4v __attribute__((ext_vector_type(4)));

constexpr int kChunk = 16;

__device__ __forceinline__ float4v mfma32(uint4 a, uint4 b, float4v c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, a), __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
}
// the upper halves of two words: a bf16 pair, cut (not rounded)
__device__ __forceinline__ uint32_t high2(float lo, float hi) {
  return __builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, hi), __builtin_bit_cast(uint32_t, lo), 0x07060302u);
}
__device__ __forceinline__ float cut(float x) {
  return __builtin_bit_cast(float, __builtin_bit_cast(uint32_t, x) & 0xffff0000u);
}

// Two fp32 values as NT bf16 pairs that add up to them, eight bits each:
// NT = 3 holds fp32, NT = 2 the eleven bits of fp16, both exactly.
template <int NT>
__device__ __forceinline__ void split2(float x, float y, uint32_t* t) {
  t[0] = high2(x, y);
  x -= cut(x);
  y -= cut(y);
  t[1] = high2(x, y);
  if (NT == 2) return;
  x -= cut(x);
  y -= cut(y);
  t[2] = high2(x, y);
}

// Eight values as NT operands.
template <int NT>
__device__ __forceinline__ void split8(const float* x, uint4* t) {
  uint32_t w[4][NT];
#pragma unroll
  for (int i = 0; i < 4; ++i) split2<NT>(x[2 * i], x[2 * i + 1], w[i]);
#pragma unroll
  for (int n = 0; n < NT; ++n) t[n] = make_uint4(w[0][n], w[1][n], w[2][n], w[3][n]);
}
// Four values of a 16x16 result as NT half operands.
template <int NT>
__device__ __forceinline__ void split4(float4v x, uint2* t) {
  uint32_t w[2][NT];
  split2<NT>(x[0], x[1], w[0]);
  split2<NT>(x[2], x[3], w[1]);
#pragma unroll
  for (int n = 0; n < NT; ++n) t[n] = make_uint2(w[0][n], w[1][n]);
}

// The term products that count, smallest first: the six above 2^-24.
__device__ __forceinline__ float4v mul32(const uint4* a, const uint4* b, float4v c) {
  c = mfma32(a[0], b[2], c);
  c = mfma32(a[2], b[0], c);
  c = mfma32(a[1], b[1], c);
  c = mfma32(a[0], b[1], c);
  c = mfma32(a[1], b[0], c);
  return mfma32(a[0], b[0], c);
}

__device__ __forceinline__ uint4 pair(uint2 a, uint2 b) { return make_uint4(a.x, a.y, b.x, b.y); }

// A product over 16 tokens fills half of an instruction's 32 slots, so two
// term products go side by side: (a0, a1) with (b0, b0) and so on.  The
// 16-slot instruction takes as long and is not used: in an earlier form of
// these kernels, where 32-slot instructions went on adding to its results,
// sums came out without their last two registers, at some timings.  Why is not
// known; the instruction, the compiler's wait states and that form's own order
// are all possible.  What is kept to here: a result that another kind of matrix
// instruction adds to has been read by a vector instruction first (settled).
__device__ __forceinline__ float4v mul_tokens(const uint2* a, const uint2* b, float4v c) {
  c = mfma32(pair(a[0], a[2]), pair(b[2], b[0]), c);
  c = mfma32(pair(a[0], a[1]), pair(b[1], b[1]), c);
  return mfma32(pair(a[0], a[1]), pair(b[0], b[0]), c);
}
// the same with NV exact terms of b
template <int NV>
__device__ __forceinline__ float4v mul_values(const uint2* a, const uint2* b, float4v c) {
  c = mfma32(pair(a[2], make_uint2(0, 0)), pair(b[0], make_uint2(0, 0)), c);
  if (NV == 2) c = mfma32(pair(a[0], a[1]), pair(b[NV - 1], b[NV - 1]), c);
  return mfma32(pair(a[0], a[1]), pair(b[0], b[0]), c);
}

// One chunk's operands in LDS, prepared by one wave and read by those that
// hold the state.
struct ChunkOps {
  uint4 a[3][2][64];    // A: terms, channel halves, lanes (row q, channels 32 h + 8 g + j)
  uint4 r[3][2][64];    // R (where Y is wanted, as q)
  uint4 q[3][64];       // row q, slots j < 4: Qb at 4 g + j, j >= 4: Qk
  uint2 t[3][64];       // T: row q, slots 4 g + i
  uint2 ak[3][64];      // Ak: row q, slots 4 g + i
  uint4 b[3][16 * 8];   // B rows [16][64 channels] in blocks of eight, see row_block
  uint4 k[3][16 * 8];
  uint4 v[2][16 * 8];   // V rows, two bf16 terms (one for bf16 rows)
  float end[64];        // exp L_15 by channel
  int odd;              // what is not finite: kOddRows, kOddValues
};
constexpr int kOddRows = 1, kOddValues = 2;

// Block c (eight channels) of row t.  A transposing read takes four rows and
// two of every four channels of half a row at once; turning the halves of
// rows 2 and 3 of each four puts all of them on different banks.
__device__ __forceinline__ int row_block(int t, int c) { return t * 8 + (c ^ ((t & 2) << 1)); }

// Four rows 4 g + 0..3 of one channel per lane, as half an operand: within
// the 16 lanes of g, lane q fetches row 4 g + q / 4, four channels from ch(q % 4).
__device__ __forceinline__ uint2 rows4(const uint4* rows, int g, int q, int channel) {
  const int t = 4 * g + (q >> 2);
  const uint2* p = (const uint2*)(rows + row_block(t, channel >> 3)) + ((channel >> 2) & 1);
  typedef __attribute__((address_space(3))) short4v lds4;
  return __builtin_bit_cast(uint2, __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds4*)p));
}

// One 16-byte block of a row, or a constant past the sequence's end.
__device__ __forceinline__ uint4 block_or(uint32_t other, const void* base, size_t elem, bool held) {
  return held ? *(const uint4*)((const uint16_t*)base + elem) : make_uint4(other, other, other, other);
}

template <int CTRL>
__device__ __forceinline__ float dpp_or(float old, float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(__builtin_bit_cast(int, old), __builtin_bit_cast(int, v), CTRL,
                                                               0xf, 0xf, false));
}

// Prepares a chunk in four steps of about the same length, for the wave that
// owns it; lane 16 g + q has token q and channels 32 h + 8 g + 0..7.  Places
// past the sequence's end are neutral: a raw decay of -inf, which is a decay
// of 1, and zeros everywhere else.
//
// REV: the operands of the gradient's walk back.  With D the gradient of the
// state after the chunk times exp L_15,
//   Z = T^T (B D^T + Qb^T dY),   dS = D + Z^T A + dY^T R
// which is the forward chain with B for A, Qb^T for Ak, T^T for T, A and R for
// B and K, and dY for V (p.v is dY then, and p.k is not read).
//
// OUT: with what Y takes, R, Qb and Qk.
template <typename T, bool OUT, bool REV>
struct ChunkPrep {
  uint4 raw[6][2];  // r, w, k, v, a, b
  float fall[16], grow[16];
  uint4 at[3][2], rt[3][2], bt[3][2], kt[3][2];
  float4v ab, ak, qb, qk;

  __device__ __forceinline__ void load(const TimeMix& p, int head, int t0, int n, int lane) {
    const int q = lane & 15, g = lane >> 4;
    const bool held = q < n;
    // one address for the wave per array, one offset per lane for all; made
    // anew for each chunk, because six lane addresses kept would cost twelve
    // registers, which spill
    const size_t row = (size_t)t0 * p.ld + head * kHead;
    size_t at0 = (size_t)q * p.ld + 8 * g;
    asm volatile("" : "+v"(at0));
    const void* src[6] = {p.r, p.w, p.k, p.v, p.a, p.b};
#pragma unroll
    for (int i = 0; i < 6; ++i)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if ((OUT || REV || i != 0) && (!REV || i != 2)) raw[i][h] = block_or(i == 1 ? T::kMinusInf2 : 0u, (const uint16_t*)src[i] + row, at0 + 32 * h, held);
  }

  __device__ __forceinline__ static void up8(uint4 v, float* f) {
    up2<T>(v.x, f);
    up2<T>(v.y, f + 2);
    up2<T>(v.z, f + 4);
    up2<T>(v.w, f + 6);
  }

  // accumulated decays: a sum over the 16 lanes of a row, then 2^L and 2^-L
  __device__ __forceinline__ void decays() {
    float w[16];
    up8(raw[1][0], w);
    up8(raw[1][1], w + 8);
#pragma unroll
    for (int j = 0; j < 16; ++j) {
      float l = log2_decay(w[j]);
      l += dpp<0x111>(l);  // row_shr:1, 2, 4, 8
      l += dpp<0x112>(l);
      l += dpp<0x114>(l);
      l += dpp<0x118>(l);
      fall[j] = __builtin_amdgcn_exp2f(l);
      grow[j] = __builtin_amdgcn_exp2f(-l);
    }
  }

  __device__ __forceinline__ void factors() {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      uint4 t[3];
      float x[8], before[8];  // 2^L of the row before
#pragma unroll
      for (int j = 0; j < 8; ++j) before[j] = dpp_or<0x111>(1.f, fall[8 * h + j]);
      auto scaled = [&](int which, const float* s) {
        up8(raw[which][h], x);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] *= s[j];
      };
      scaled(4, before);
      split8<3>(x, t);
      at[0][h] = t[0]; at[1][h] = t[1]; at[2][h] = t[2];
      scaled(5, grow + 8 * h);
      split8<3>(x, t);
      bt[0][h] = t[0]; bt[1][h] = t[1]; bt[2][h] = t[2];
      if (!REV) {
        scaled(2, grow + 8 * h);
        split8<3>(x, t);
        kt[0][h] = t[0]; kt[1][h] = t[1]; kt[2][h] = t[2];
      }
      if (OUT || REV) {
        scaled(0, fall + 8 * h);
        split8<3>(x, t);
        rt[0][h] = t[0]; rt[1][h] = t[1]; rt[2][h] = t[2];
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  }

  // X Y^T over the 64 channels
  __device__ __forceinline__ static float4v gram(const uint4 (&x)[3][2], const uint4 (&y)[3][2]) {
    float4v c = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint4 a[3] = {x[0][h], x[1][h], x[2][h]}, b[3] = {y[0][h], y[1][h], y[2][h]};
      c = mul32(a, b, c);
    }
    return c;
  }

  __device__ __forceinline__ void grams() {
    ab = gram(at, bt);  // row t = 4 g + i, column s = q
    if (REV) {
      ak = gram(rt, bt);  // row t = 4 g + i, column s = q: the operand of Qb^T
      return;
    }
    ak = gram(kt, at);  // row s = 4 g + i, column t = q: already the operand of Ak
    if (!OUT) return;
    qb = gram(bt, rt);
    qk = gram(kt, rt);
  }

  __device__ __forceinline__ void put_rows(ChunkOps& o, int lane) const {
    const int q = lane & 15, g = lane >> 4;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int block = row_block(q, 4 * h + g);
#pragma unroll
      for (int n = 0; n < 3; ++n) {
        o.a[n][h][lane] = REV ? bt[n][h] : at[n][h];
        o.b[n][block] = REV ? at[n][h] : bt[n][h];
        o.k[n][block] = REV ? rt[n][h] : kt[n][h];
        if (OUT) o.r[n][h][lane] = rt[n][h];
      }
      put_v(o, block, raw[3][h], (T*)nullptr);
      if (q == 15)
#pragma unroll
        for (int j = 0; j < 8; ++j) o.end[32 * h + 8 * g + j] = fall[8 * h + j];
    }
  }
  // V rows as bf16 terms: bf16 is one; fp16's eleven bits are two, exactly
  __device__ __forceinline__ static void put_v(ChunkOps& o, int block, uint4 v, BF16*) { o.v[0][block] = v; }
  __device__ __forceinline__ static void put_v(ChunkOps& o, int block, uint4 v, F16*) {
    float x[8];
    uint4 t[2];
    up8(v, x);
    split8<2>(x, t);
    o.v[0][block] = t[0];
    o.v[1][block] = t[1];
  }

  // Rows 0..15 of a 16x16 result, each in one register of every lane group:
  // lane swaps of the halves, then of the quarters.
  __device__ __forceinline__ static void spread_rows(float4v x, float* row) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float f = x[i];  // a vector's element is not cast in place: clang takes the first one
      const uint32_t v = __builtin_bit_cast(uint32_t, f);
      const auto h = __builtin_amdgcn_permlane32_swap(v, v, false, false);  // groups 0 1 0 1, 2 3 2 3
      const auto lo = __builtin_amdgcn_permlane16_swap(h[0], h[0], false, false);
      const auto hi = __builtin_amdgcn_permlane16_swap(h[1], h[1], false, false);
      row[i] = __builtin_bit_cast(float, (uint32_t)lo[0]);
      row[4 + i] = __builtin_bit_cast(float, (uint32_t)lo[1]);
      row[8 + i] = __builtin_bit_cast(float, (uint32_t)hi[0]);
      row[12 + i] = __builtin_bit_cast(float, (uint32_t)hi[1]);
    }
  }
  // x + lane LANE of each group's v * y
  template <int LANE>
  __device__ __forceinline__ static float fma_lane(float v, float y, float x) {
    return fmaf(dpp<0x150 + LANE>(v), y, x);  // row_newbcast
  }
  template <int S, int U, bool COLUMN>
  __device__ __forceinline__ static float substitute(const float* ab, const float* row, float x) {
    // row form: T[q][s] += T[q][u] Ab[u][s], u from 15 down to s + 1; column
    // form: T[s][q] += Ab[s][u] T[u][q], u from 0 up to s - 1
    if constexpr (COLUMN) {
      if constexpr (U < S) return substitute<S, U + 1, true>(ab, row, fma_lane<U>(ab[S], row[U], x));
    } else {
      if constexpr (U > S) return substitute<S, U - 1, false>(ab, row, fma_lane<S>(ab[U], row[U], x));
    }
    return x;
  }
  template <int S, bool COLUMN>
  __device__ __forceinline__ static void substitute_all(const float* ab, float* row, int q) {
    row[S] = substitute<S, COLUMN ? 0 : 15, COLUMN>(ab, row, q == S ? 1.f : 0.f);
    if constexpr (COLUMN && S < 15) substitute_all<S + 1, true>(ab, row, q);
    if constexpr (!COLUMN && S > 0) substitute_all<S - 1, false>(ab, row, q);
  }
  __device__ __forceinline__ static float4v pick4(const float* x, int g) {
    float4v r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[i], b = x[4 + i], c = x[8 + i], d = x[12 + i];
      const float lo = g & 1 ? b : a, hi = g & 1 ? d : c;
      r[i] = g & 2 ? hi : lo;
    }
    return r;
  }

  // T = (1 - Ab)^-1 from T = 1 + T Ab: lane q has row q, and column s follows
  // from the columns to its right (REV: T = 1 + Ab T, lane q has column q, and
  // row s follows from the rows above).  Substitution, because the powers of
  // Ab grow and cancel where neighbouring tokens share a direction.
  __device__ __forceinline__ void solve(ChunkOps& o, int lane) const {
    const int q = lane & 15, g = lane >> 4;
    float row[16], abr[16];
    spread_rows(ab, abr);
    substitute_all<REV ? 0 : 15, REV>(abr, row, q);
    uint2 t[3];
    split4<3>(pick4(row, g), t);
#pragma unroll
    for (int n = 0; n < 3; ++n) o.t[n][lane] = t[n];
    // slot s = 4 g + i of row t = q
    float4v k = ak;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (REV ? 4 * g + i < q : 4 * g + i >= q) k[i] = 0.f;
    split4<3>(k, t);
#pragma unroll
    for (int n = 0; n < 3; ++n) o.ak[n][lane] = t[n];
    if (!OUT) return;
    // every row of A, B and K is in ab and ak
    float zero = 0.f;
    uint32_t values = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) zero += ab[i] + ak[i];
    zero *= 0.f;
#pragma unroll
    for (int h = 0; h < 2; ++h)
      values |= T::not_finite2(raw[3][h].x) | T::not_finite2(raw[3][h].y) | T::not_finite2(raw[3][h].z) | T::not_finite2(raw[3][h].w);
    const int odd = (__builtin_amdgcn_ballot_w64(zero != zero) ? kOddRows : 0) | (__builtin_amdgcn_ballot_w64(values != 0) ? kOddValues : 0);
    if (lane == 0) o.odd = odd;
    float4v qbm = qb, qkm = qk;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (4 * g + i > q) qbm[i] = qkm[i] = 0.f;
    uint2 b[3], c[3];
    split4<3>(qbm, b);
    split4<3>(qkm, c);
#pragma unroll
    for (int n = 0; n < 3; ++n) o.q[n][lane] = make_uint4(b[n].x, b[n].y, c[n].x, c[n].y);
  }
};

// The state's side of a chunk: sixteen channels of v per wave (16 wave + q),
// S^T in four tiles.
struct ChunkState {
  float4v X[4];

  __device__ __forceinline__ static int channel(int n, int g) { return 32 * (n >> 1) + 8 * g + 4 * (n & 1); }

  __device__ __forceinline__ void load(const float* state, int wave, int lane) {
    const int q = lane & 15, g = lane >> 4;
#pragma unroll
    for (int n = 0; n < 4; ++n)
      X[n] = state ? *(const float4v*)(state + (16 * wave + q) * kHead + channel(n, g)) : float4v{0.f, 0.f, 0.f, 0.f};
  }
  __device__ __forceinline__ void store(float* state, int wave, int lane) const {
    const int q = lane & 15, g = lane >> 4;
#pragma unroll
    for (int n = 0; n < 4; ++n) *(float4v*)(state + (16 * wave + q) * kHead + channel(n, g)) = X[n];
  }
  // rows of the identity, for the map from the state before a segment to the
  // one after it
  __device__ __forceinline__ void identity(int wave, int lane) {
    const int q = lane & 15, g = lane >> 4;
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) X[n][i] = channel(n, g) + i == 16 * wave + q ? 1.f : 0.f;
  }

  // Passes the state through vector moves, which wait for whatever wrote it.
  __device__ __forceinline__ void settled() {
#pragma unroll
    for (int n = 0; n < 4; ++n)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float x = X[n][i];
        X[n][i] = dpp<0xe4>(x);  // quad_perm 0,1,2,3: as it is
      }
    __builtin_amdgcn_sched_barrier(0);
  }

  // S <- S P + G with P, G [64][64] in fp32, on fp32 matrix instructions:
  // register i of tile n is the slot of contraction channel(n, g) + i.
  __device__ __forceinline__ void apply(const float* G, const float* P, int wave, int lane) {
    const int q = lane & 15, g = lane >> 4;
    ChunkState to;
    to.load(G, wave, lane);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float* row = P + 32 * (m >> 1) + 8 * (q >> 2) + 4 * (m & 1) + (q & 3);
#pragma unroll
      for (int n = 0; n < 4; ++n)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          to.X[m] = __builtin_amdgcn_mfma_f32_16x16x4f32(row[(channel(n, g) + i) * kHead], X[n][i], to.X[m], 0, 0, 0);
    }
    *this = to;
    settled();
  }
};

// The operands that a chunk starts with; with REV also what scales the state
// before it.
template <typename T, bool REV>
struct ChunkHead {
  static constexpr int kV = __is_same(T, BF16) ? 1 : 2;  // terms of V
  uint4 a[2][3];
  uint2 ak[3], v[kV], t[3];
  float4v end[4];
  int odd;

  // values: all ones, or 0 to take V for zeros (the map alone)
  __device__ __forceinline__ void fetch(const ChunkOps& o, int wave, int lane, uint32_t values) {
    const int q = lane & 15, g = lane >> 4;
    odd = o.odd;  // first, because it is looked at first
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < 3; ++n) a[h][n] = o.a[n][h][lane];
#pragma unroll
    for (int n = 0; n < 3; ++n) ak[n] = o.ak[n][lane];
#pragma unroll
    for (int n = 0; n < kV; ++n) {
      v[n] = rows4(o.v[n], g, q, 16 * wave + 4 * (q & 3));
      v[n].x &= values;
      v[n].y &= values;
    }
#pragma unroll
    for (int n = 0; n < 3; ++n) t[n] = o.t[n][lane];
    if (REV)
#pragma unroll
      for (int n = 0; n < 4; ++n) end[n] = *(const float4v*)&o.end[ChunkState::channel(n, g)];
  }
};

// The state as operands of the next products: three terms.
__device__ __forceinline__ void split_half(const ChunkState& st, int h, uint4* x) {
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[i] = st.X[2 * h][i];
    f[4 + i] = st.X[2 * h + 1][i];
  }
  split8<3>(f, x);
}

// Instruction mixes for the scheduler: N times one matrix instruction and then
// so many of the others.
template <int N, int READS, int VALU>
__device__ __forceinline__ void interleave() {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (READS) __builtin_amdgcn_sched_group_barrier(0x100, READS, 0);
    if (VALU) __builtin_amdgcn_sched_group_barrier(0x002, VALU, 0);
  }
}

// The columns (channels of v, of this wave's sixteen) in which a lane has `on`.
__device__ __forceinline__ uint32_t columns(bool on) {
  uint64_t m = __builtin_amdgcn_ballot_w64(on);
  m |= m >> 32;
  return (uint32_t)(m | m >> 16) & 0xffffu;
}

// Whether what is not finite in a chunk would reach the outputs of tokens before
// it: the triangular products multiply what a later token has with zeros, which
// makes NaN of it.  In a column whose state is not finite already none of the
// outputs is, in whatever way they are summed.  (R reaches its own row only.)
template <typename T, bool REV>
__device__ __forceinline__ bool leaks(const ChunkState& st, const ChunkHead<T, REV>& hd, int odd) {
  uint32_t hurt = 0, held = 0;
#pragma unroll
  for (int n = 0; n < ChunkHead<T, REV>::kV; ++n) hurt |= BF16::not_finite2(hd.v[n].x) | BF16::not_finite2(hd.v[n].y);
#pragma unroll
  for (int n = 0; n < 4; ++n)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float s = st.X[n][i];
      held |= (__builtin_bit_cast(uint32_t, s) & 0x7f800000u) == 0x7f800000u;
    }
  return (((odd & kOddRows) ? 0xffffu : columns(hurt != 0)) & ~columns(held != 0)) != 0;
}

// A chunk's n tokens one after the other, for one that leaks: Y as chunk_step
// lays it out.  Rows come straight from memory.
template <typename T>
__device__ __forceinline__ float4v step_tokens(const TimeMix& p, int head, int t0, int n, ChunkState& st, int wave, int lane) {
  asm volatile("" : "+v"(lane));  // nothing of this is kept in registers over the chunks
  const int q = lane & 15, g = lane >> 4;
  float4v y = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 1
  for (int t = 0; t < n; ++t) {
    const size_t row = (size_t)(t0 + t) * p.ld + head * kHead;
    auto four = [&](const void* from, int m) {  // the channels of tile m that this lane has
      const uint2 v = *(const uint2*)((const uint16_t*)from + row + ChunkState::channel(m, g));
      float f[4];
      up2<T>(v.x, f);
      up2<T>(v.y, f + 2);
      return float4v{f[0], f[1], f[2], f[3]};
    };
    auto over_groups = [](float x) {
      x += __shfl_xor(x, 16);
      return x + __shfl_xor(x, 32);
    };
    const float v = T::up(((const uint16_t*)p.v)[row + 16 * wave + q]);
    float u = 0.f, out = 0.f;
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float4v a = four(p.a, m);
#pragma unroll
      for (int i = 0; i < 4; ++i) u = fmaf(st.X[m][i], a[i], u);
    }
    u = over_groups(u);
#pragma unroll
    for (int m = 0; m < 4; ++m) {
      const float4v w = four(p.w, m), b = four(p.b, m), k = four(p.k, m), r = four(p.r, m);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        st.X[m][i] = fmaf(st.X[m][i], __builtin_amdgcn_exp2f(log2_decay(w[i])), fmaf(u, b[i], v * k[i]));
        out = fmaf(st.X[m][i], r[i], out);
      }
    }
    out = over_groups(out);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t == 4 * g + i) y[i] = out;
  }
  return y;
}

// Takes the state over a chunk.  OUT: Y (row t = 4 g + i, column v = q).  REV:
// back over it.  save(U) takes U, or Z, as Y is laid out.  x: the state as
// operands, made again at the end; with REV the state is scaled by the next
// chunk's `end` before that.
//
// What bounds it: one wave's chain from state to state.  Its products are
// about 950 cycles of the matrix unit; cutting results into terms and fetching
// 30 KB of operands each take about as long, a fetch some 15 cycles of the
// wave's issue and no more than fifteen in flight.  So the three are mixed by
// hand, instruction by instruction: B, K and `end` between the products with A
// and R, the next chunk's head (`next`) and the cutting of each half of the
// new state between the products of its update.  Measured: 1.33 us a chunk (one
// sequence of 4096 tokens, 32 heads), 1.36 with every second compute unit at
// work (128 heads).  What Y alone takes in two terms in place of three would
// save 0.1 of it and leave fp16 outputs 1.2e-4 of their norm from those of fp32
// operations, now 1.2e-5.
template <typename T, bool OUT, bool REV, typename Next, typename Save>
__device__ __forceinline__ float4v chunk_step(ChunkState& st, uint4 (*x)[3], const ChunkOps& o, ChunkHead<T, REV>& hd,
                                              int lane, Next next, Save save) {
  const int q = lane & 15, g = lane >> 4;
  constexpr int NV = ChunkHead<T, REV>::kV;
  const float4v zero = {0.f, 0.f, 0.f, 0.f};
  uint4 r[2][3], qq[3];
  if (OUT) {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < 3; ++n) r[h][n] = o.r[n][h][lane];
#pragma unroll
    for (int n = 0; n < 3; ++n) qq[n] = o.q[n][lane];
  }
  __builtin_amdgcn_sched_barrier(0);
  // A S^T + Ak V, R S^T
  uint2 b[4][3], k[4][3];
  float4v end[4];
#pragma unroll
  for (int n = 0; n < 4; ++n) {
#pragma unroll
    for (int j = 0; j < 3; ++j) {
      b[n][j] = rows4(o.b[j], g, q, ChunkState::channel(n, q & 3));
      k[n][j] = rows4(o.k[j], g, q, ChunkState::channel(n, q & 3));
    }
    if (!REV) end[n] = *(const float4v*)&o.end[ChunkState::channel(n, g)];
  }
  float4v y = zero;
  const float4v u0 = mul32(hd.a[0], x[0], zero);
  float4v u = mul_values<NV>(hd.ak, hd.v, mul32(hd.a[1], x[1], zero));
  if (OUT)
#pragma unroll
    for (int h = 0; h < 2; ++h) y = mul32(r[h], x[h], y);
  interleave<(12 + NV + 1 + (OUT ? 12 : 0)), (OUT ? 1 : 2), 0>();
  __builtin_amdgcn_sched_barrier(0);
  uint2 s[3];
  u += u0;
  split4<3>(u, s);
  u = mul_tokens(hd.t, s, zero);
  split4<3>(u, s);
  save(u);
  uint4 uv[3];
#pragma unroll
  for (int n = 0; n < 3; ++n) uv[n] = pair(s[n], n < NV ? hd.v[n < NV ? n : 0] : make_uint2(0, 0));
  __builtin_amdgcn_sched_barrier(0);
  next();
  // S' = (S + U^T B + V^T K) diag(end), Y = R S^T + Q (U, V)
#pragma unroll
  for (int n = 0; n < 4; ++n) {
    uint4 c[3];
#pragma unroll
    for (int j = 0; j < 3; ++j) c[j] = pair(b[n][j], k[n][j]);
    st.X[n] = mul32(c, uv, st.X[n]) * (REV ? hd.end[n] : end[n]);
    if (n & 1) split_half(st, n >> 1, x[n >> 1]);
  }
  if (OUT) y = mul32(qq, uv, y);
  interleave<12, 1, 0>();
  interleave<(12 + (OUT ? 6 : 0)), 0, 4>();
  __builtin_amdgcn_sched_barrier(0);
  if (OUT)
    // cut here, between the products, and not where the loop's two entries meet
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int n = 0; n < 3; ++n) asm volatile("" : "+v"(x[h][n].x), "+v"(x[h][n].y), "+v"(x[h][n].z), "+v"(x[h][n].w));
  return y;
}

// A workgroup that walks a run of chunks: waves 0-3 hold the state, sixteen
// channels of v each, and take it from chunk to chunk (where the run's map is
// wanted too, waves 4-7 hold that); the other waves prepare the chunks'
// operands ahead of them, in turn, in LDS buffers.  Two counters per buffer
// order them: `ready` chunks written, and `done` one per chunk and walking
// wave.  Every wait is for a count that the other side reaches by
// itself: a buffer's chunk c waits for the readers of chunk c - kBuffers, who
// wait for nothing later than it.
constexpr int kBuffers = 4;
constexpr int kWalkWaves = 12;

struct ChunkLds {
  ChunkOps ops[kBuffers];
  int ready[kBuffers], done[kBuffers];
};

__device__ __forceinline__ void clear_counts(ChunkLds& sh) {
  if (threadIdx.x < kBuffers) sh.ready[threadIdx.x] = sh.done[threadIdx.x] = 0;
  __syncthreads();
}
__device__ __forceinline__ int count_of(int* count) {
  return __builtin_amdgcn_readfirstlane(__hip_atomic_load(count, __ATOMIC_ACQUIRE, __HIP_MEMORY_SCOPE_WORKGROUP));
}
__device__ __forceinline__ void wait_for(int* count, int want) {
  while (count_of(count) < want) __builtin_amdgcn_s_sleep(1);
}
// The LDS does a wave's operations in their order, so what the wave has read
// or written before is done when the count changes; only the compiler has to
// be kept from moving them.
__device__ __forceinline__ void signal(int* count, int lane) {
  asm volatile("" ::: "memory");
  if (lane == 0) __hip_atomic_fetch_add(count, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
  asm volatile("" ::: "memory");
}

// The side of preparing wave `wave`, which comes after `walkers` others: the
// chunks of tokens begin..end, from the last to the first with REV.
template <typename T, bool OUT, bool REV>
__device__ __forceinline__ void prepare_chunks(const TimeMix& p, int begin, int end, ChunkLds& sh, int head, int walkers, int wave,
                                               int lane) {
  const int chunks = (end - begin + kChunk - 1) / kChunk;
  ChunkPrep<T, OUT, REV> prep;
  for (int c = wave - walkers; c < chunks; c += kWalkWaves - walkers) {
    ChunkOps& o = sh.ops[c % kBuffers];
    const int t = begin + (REV ? chunks - 1 - c : c) * kChunk;
    prep.load(p, head, t, min(kChunk, end - t), lane);
    prep.decays();
    // without these the scheduler mixes the stages and needs more registers
    __builtin_amdgcn_sched_barrier(0);
    prep.factors();
    __builtin_amdgcn_sched_barrier(0);
    prep.grams();
    __builtin_amdgcn_sched_barrier(0);
    wait_for(&sh.done[c % kBuffers], c / kBuffers * walkers);
    prep.put_rows(o, lane);
    __builtin_amdgcn_sched_barrier(0);
    prep.solve(o, lane);
    signal(&sh.ready[c % kBuffers], lane);
  }
}

// A walking wave's side: its part of a state over the run, or of the map
// (values 0).  In the c-th chunk of the walk: before(c) with the state at hand
// (multiplied by `end` with REV), save(c, U or Z), and, with OUT, out(c, Y) and
// steps(c), which takes the state over the chunk token by token.
template <typename T, bool OUT, bool REV, typename Before, typename Save, typename Out, typename Steps>
__device__ __forceinline__ void walk_chunks(ChunkState& st, int chunks, ChunkLds& sh, int wave, int lane, uint32_t values,
                                            Before before, Save save, Out out, Steps steps) {
  ChunkHead<T, REV> hd;
  uint4 x[2][3];
  int c = 0;
  while (c < chunks) {
    wait_for(&sh.ready[c % kBuffers], c / kBuffers + 1);
    hd.fetch(sh.ops[c % kBuffers], wave, lane, values);
    if (REV)
#pragma unroll
      for (int n = 0; n < 4; ++n) st.X[n] *= hd.end[n];
#pragma unroll
    for (int h = 0; h < 2; ++h) split_half(st, h, x[h]);
    bool whole = true;
    for (; c < chunks; ++c) {
      if (OUT) {
        const int odd = __builtin_amdgcn_readfirstlane(hd.odd);
        if (__builtin_expect(odd != 0, 0) && leaks(st, hd, odd)) {
          whole = false;
          break;
        }
      }
      const int n = c + 1;
      const ChunkOps& o = sh.ops[c % kBuffers];
      before(c);
      // looked at early, so that the answer is here when it is needed
      const int seen = __hip_atomic_load(&sh.ready[n % kBuffers], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
      const float4v y = chunk_step<T, OUT, REV>(
          st, x, o, hd, lane,
          [&] {
            const int want = n < chunks ? n / kBuffers + 1 : 0;
            if (__builtin_amdgcn_readfirstlane(seen) < want) wait_for(&sh.ready[n % kBuffers], want);
            asm volatile("" ::: "memory");
            // (past the last chunk whatever the buffer holds, for nothing)
            hd.fetch(sh.ops[n % kBuffers], wave, lane, values);
            if (REV && n >= chunks)
#pragma unroll
              for (int i = 0; i < 4; ++i) hd.end[i] = float4v{1.f, 1.f, 1.f, 1.f};
          },
          [&](float4v u) { save(c, u); });
      signal(&sh.done[c % kBuffers], lane);
      if (OUT) out(c, y);
    }
    // out of the loop, so that it costs the others no registers
    if (!whole) {
      const float4v y = steps(c);
      signal(&sh.done[c % kBuffers], lane);
      out(c, y);
      ++c;
    }
  }
}

template <typename K>
hipError_t allow_lds(K* kernel) {
  return hipFuncSetAttribute((const void*)kernel, hipFuncAttributeMaxDynamicSharedMemorySize, sizeof(ChunkLds));
}

}  // namespace rq
