// Internal launchers and device helpers of the operators between an RWKV-7
// layer's projections: the shifted norm (shift_norm.hip), the state recurrence
// (time_mix.hip, time_mix_back.hip), the head norm and gate (head_gate.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "device_common.h"
#include "runs.h"

namespace rq {

constexpr int kHead = 64;  // channels per head

// Sequences in a run of tokens: offsets cu[nseq + 1], or null for nseq
// sequences of `len` tokens each.
struct Sequences {
  const int32_t* cu;
  int nseq;
  int len;
  int tokens;
};

// Where sequence i keeps its state: slots[i], or i itself without a slot map;
// -1 for a slot outside the array.
struct Slots {
  const int32_t* map;
  int count;
};

// ---- norm, shift and mixtures (shift_norm.hip) ------------------------------
struct ShiftNorm {
  const void* x;      // [tokens][ld]
  const void* delta;  // [tokens][ld] or null
  float alpha;
  int width, ld;
  Sequences seq;
  Slots slots;
  const float* gamma;
  const float* beta;
  float eps;
  const float* mu;  // [nmix][width]
  int nmix;
  const void* shift_in;  // [slots][width] or null
  void* shift_out;       // or null
  void* x_out;           // [tokens][ld] or null
  void* out;             // [nmix][tokens][ldo]
  int ldo;
};
hipError_t launch_shift_norm(const ShiftNorm& p, bool bf16, hipStream_t st);

struct ShiftNormBack {
  const void* x;
  float alpha;
  int width, ld;
  Sequences seq;
  const float* gamma;
  const float* beta;
  float eps;
  const float* mu;
  int nmix;
  const void* shift_in;   // [nseq][width] or null
  const void* dout;       // [nmix][tokens][ldo]
  int ldo;
  const void* dx_out;     // [tokens][ld] or null
  const void* dshift_out; // [nseq][width] or null
  void* dx;               // [tokens][ld]
  void* ddelta;           // [tokens][ld] or null
  void* dshift_in;        // [nseq][width] or null
  float* dgamma;
  float* dbeta;
  float* dmu;             // [nmix][width]
  float* parts;           // workspace of parts_bytes, or null
  size_t parts_bytes;
};
hipError_t launch_shift_norm_back(const ShiftNormBack& p, bool bf16, hipStream_t st);

// Sums rows 0..count-1 of parts, [count][n0 + n1 + n2], into three arrays of
// n0, n1 and n2 (multiples of four), in a fixed order (head_gate.hip).
struct SumTargets {
  float* out[3];
  int n[3];
};
hipError_t launch_sum_parts(const float* parts, int count, const SumTargets& to, hipStream_t st);

// ---- head norm, bonus and gate (head_gate.hip) ------------------------------
struct HeadGate {
  const void *y, *r, *k, *v, *g;  // [tokens][ld]
  int tokens, heads, ld;
  const float *gamma, *beta, *u;  // [64 heads]
  float eps;
  void* out;  // [tokens][ldo]
  int ldo;
};
hipError_t launch_head_gate(const HeadGate& p, bool bf16, hipStream_t st);

struct HeadGateBack {
  HeadGate f;        // out unused
  const void* dout;  // [tokens][ld], as every gradient
  void *dy, *dr, *dk, *dv, *dg;
  float *dgamma, *dbeta, *du;
  float* parts;
  size_t parts_bytes;
};
hipError_t launch_head_gate_back(const HeadGateBack& p, bool bf16, hipStream_t st);

// ---- state recurrence (time_mix.hip, time_mix_back.hip) ---------------------
struct TimeMix {
  const void *r, *w, *k, *v, *a, *b;  // [tokens][ld]
  int heads, ld;
  Sequences seq;
  Slots slots;
  const float* state_in;  // [slots][heads][64][64] or null
  float* state_out;       // or null
  void* y;                // [tokens][ldy]
  int ldy;
  float* parts;
  size_t parts_bytes;
};
hipError_t launch_time_mix(const TimeMix& p, bool bf16, hipStream_t st);

struct TimeMixBack {
  TimeMix f;                // y, state_out unused; slots are the sequences
  const void* dy;           // [tokens][ld]
  const float* dstate_out;  // [nseq][heads][64][64] or null
  void *dr, *dw, *dk, *dv, *da, *db;
  float* dstate_in;  // or null
};
hipError_t launch_time_mix_back(const TimeMixBack& p, bool bf16, hipStream_t st);
// workspace bytes that launch_time_mix_back needs (past the split counters)
size_t time_mix_back_bytes(int64_t tokens, int64_t heads, int64_t nseq);

#if defined(__HIPCC__)
// ---- device helpers ----------------------------------------------------------

// 16-bit element types: widening is exact, narrowing rounds to nearest even
struct F16 {
  static constexpr uint32_t kMinusInf2 = 0xfc00fc00u;
  // nonzero if one of two values is an infinity or NaN: its exponent's carry
  static __device__ __forceinline__ uint32_t not_finite2(uint32_t v) { return ((v & 0x7fff7fffu) + 0x04000400u) & 0x80008000u; }
  static __device__ __forceinline__ float up(uint32_t lo16) {
    return (float)__builtin_bit_cast(_Float16, (uint16_t)lo16);
  }
  static __device__ __forceinline__ uint32_t down2(float a, float b) {
    half2v h = {(_Float16)a, (_Float16)b};
    return __builtin_bit_cast(uint32_t, h);
  }
};
struct BF16 {
  static constexpr uint32_t kMinusInf2 = 0xff80ff80u;
  static __device__ __forceinline__ uint32_t not_finite2(uint32_t v) { return ((v & 0x7fff7fffu) + 0x00800080u) & 0x80008000u; }
  static __device__ __forceinline__ float up(uint32_t lo16) { return __builtin_bit_cast(float, lo16 << 16); }
  static __device__ __forceinline__ uint32_t down2(float a, float b) {
    typedef __bf16 bf2 __attribute__((ext_vector_type(2)));
    bf2 h = {(__bf16)a, (__bf16)b};
    return __builtin_bit_cast(uint32_t, h);
  }
};

template <typename T>
__device__ __forceinline__ void up2(uint32_t v, float* f) {
  f[0] = T::up(v & 0xffffu);
  f[1] = T::up(v >> 16);
}

template <typename T>
__device__ __forceinline__ void load8(const void* base, size_t elem, float* f) {
  const uint4 v = *(const uint4*)((const uint16_t*)base + elem);
  up2<T>(v.x, f);
  up2<T>(v.y, f + 2);
  up2<T>(v.z, f + 4);
  up2<T>(v.w, f + 6);
}

template <typename T>
__device__ __forceinline__ uint4 pack8(const float* f) {
  return make_uint4(T::down2(f[0], f[1]), T::down2(f[2], f[3]), T::down2(f[4], f[5]), T::down2(f[6], f[7]));
}

template <typename T>
__device__ __forceinline__ void store8(void* base, size_t elem, const float* f) {
  *(uint4*)((uint16_t*)base + elem) = pack8<T>(f);
}

__device__ __forceinline__ void load8f(const float* p, float* f) {
  *(float4*)f = *(const float4*)p;
  *(float4*)(f + 4) = *(const float4*)(p + 4);
}

template <int CTRL>
__device__ __forceinline__ float dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_update_dpp(0, __builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}

// Sum over the 16 lanes of a row; every lane gets the same bits (the adds of
// each step pair the same two values).
__device__ __forceinline__ float row_sum(float v) {
  v += dpp<0x128>(v);  // row_ror:8
  v += dpp<0x124>(v);
  v += dpp<0x122>(v);
  v += dpp<0x121>(v);
  return v;
}

// Sum over aligned groups of 8 lanes: quads, then the mirrored half row.
__device__ __forceinline__ float oct_sum(float v) {
  v += dpp<0xb1>(v);   // quad_perm 1,0,3,2
  v += dpp<0x4e>(v);   // quad_perm 2,3,0,1
  v += dpp<0x141>(v);  // row_half_mirror
  return v;
}

__device__ __forceinline__ float wave_sum(float v) {
  v = row_sum(v);
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

// [begin, end) of sequence i; offsets outside 0..tokens or falling are
// clamped, so that every token index the kernels form is in range.
__device__ __forceinline__ void seq_span(const Sequences& s, int i, int& begin, int& end) {
  if (s.cu) {
    begin = min(max(s.cu[i], 0), s.tokens);
    end = min(max(s.cu[i + 1], begin), s.tokens);
  } else {
    begin = i * s.len;
    end = begin + s.len;
  }
}

// The last sequence that begins at or before token t.
__device__ __forceinline__ int seq_of(const Sequences& s, int t) {
  if (!s.cu) return s.len > 0 ? min(t / s.len, s.nseq - 1) : 0;
  int lo = 0, hi = s.nseq - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (s.cu[mid] <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ int slot_of(const Slots& s, int i) {
  const int j = s.map ? s.map[i] : i;
  return j >= 0 && j < s.count ? j : -1;
}

// RWKV-7's decay: log2 w = -exp(-1/2) log2(e) sigmoid(raw), so that w is in
// (0.545, 1).  Both functions below are single instructions of 1 ulp.
constexpr float kDecay = 0.6065306597126334f;
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float sigmoid_f32(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-kLog2e * x));
}
__device__ __forceinline__ float log2_decay(float raw) { return -(kDecay * kLog2e) * sigmoid_f32(raw); }
#endif

}  // namespace rq
