// One token per row of logits z:
//
//   w_i = exp((z_i - max z) / T)
//
// in the order of falling z, equal ones by rising index: the first top_k stay;
// of those the shortest prefix that holds top_p of their mass; of those the
// ones with w_i >= min_p.  The token is the first of the kept ones, by index,
// whose cumulative mass exceeds u times the kept mass.
//
// Every filter keeps a prefix of that order, so what is kept is known by its
// last member, a key (the float's bits in the order of its values) and an
// index, and nothing is sorted.  That member is found by counting: a histogram
// of 2048 classes of z, then of the digits of the keys in the one class that
// the border falls into.  A token changes when an error moves any of the
// borders between kept tokens over u, and there may be 65536 of them, so
// weights are fp64 to 2^-47, the draw's sums fp64 in a fixed order, and the
// histograms integers, in units small enough that they fit 64 bits: no order
// of the atomic adds changes a bit.
//
// A workgroup has a row.
#include "mix.h"
#include "next_token.h"

namespace rq {

namespace {

constexpr int kBins = 2048;
constexpr uint32_t kAll = 0;  // a key below every key: nothing is cut
constexpr float kMinusInf = -__builtin_huge_valf();

// 2^y to 2^-47 of its value (Taylor's series of exp(r ln 2), |r| <= 1/2); 0 far below.
__device__ __forceinline__ double pow2(double y) {
  y = fmax(y, -1100.0);
  const double n = __builtin_rint(y), r = (y - n) * 0.69314718055994530942;
  double p = 1.0 / 39916800.0;
  p = __builtin_fma(p, r, 1.0 / 3628800.0);
  p = __builtin_fma(p, r, 1.0 / 362880.0);
  p = __builtin_fma(p, r, 1.0 / 40320.0);
  p = __builtin_fma(p, r, 1.0 / 5040.0);
  p = __builtin_fma(p, r, 1.0 / 720.0);
  p = __builtin_fma(p, r, 1.0 / 120.0);
  p = __builtin_fma(p, r, 1.0 / 24.0);
  p = __builtin_fma(p, r, 1.0 / 6.0);
  p = __builtin_fma(p, r, 0.5);
  p = __builtin_fma(p, r, 1.0);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_amdgcn_ldexp(p, (int)n);
}

// Keys: unsigned numbers in the order of the floats; +0 and -0 are one.
__device__ __forceinline__ uint32_t key_of(float z) {
  const uint32_t b = __builtin_bit_cast(uint32_t, z + 0.f);
  return b ^ ((uint32_t)((int)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ float of_key(uint32_t k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

struct F32 {};
template <typename T>
__device__ __forceinline__ float up1(const void* row, int i) {
  return T::up(((const uint16_t*)row)[i]);
}
template <>
__device__ __forceinline__ float up1<F32>(const void* row, int i) {
  return ((const float*)row)[i];
}
template <typename T>
__device__ __forceinline__ void up8(const void* row, int at, float* z) {
  load8<T>(row, (size_t)at, z);
}
template <>
__device__ __forceinline__ void up8<F32>(const void* row, int at, float* z) {
  load8f((const float*)row + at, z);
}

// The cut: what comes after (key, index) in the order is out.
struct Cut {
  uint32_t key;
  int index;
  __device__ __forceinline__ bool keeps(uint32_t k, int i) const { return k > key || (k == key && i <= index); }
};

template <typename T, int NT>
struct Row {
  static constexpr int W = NT / 64;
  const void* z;
  int vocab;
  float top;        // the largest logit
  double rate;      // log2(e) / T
  int shift;        // a weight's unit in the histograms is 2^-shift
  // shared memory
  unsigned long long* hist;  // [kBins]; also the draw's sums
  unsigned long long* wsum;  // [W + 4]

  // The 8 logits from 8 v on, NaN and places past the row's end as -inf.
  __device__ __forceinline__ void get(int v, float* f) const {
    if (8 * v + 8 <= vocab) {
      up8<T>(z, 8 * v, f);
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = f[e] == f[e] ? f[e] : kMinusInf;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = 8 * v + e < vocab ? up1<T>(z, 8 * v + e) : kMinusInf;
        f[e] = x == x ? x : kMinusInf;
      }
    }
  }
  // f(z, index) for every logit, this thread's share of it
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    const int vecs = (vocab + 7) >> 3;
    for (int v = threadIdx.x; v < vecs; v += NT) {
      float x[8];
      get(v, x);
#pragma unroll
      for (int e = 0; e < 8; ++e) f(x[e], 8 * v + e);
    }
  }
  // Whether a logit has a weight at all: beside +inf only +inf has.
  __device__ __forceinline__ bool alive(float x) const {
    return x > kMinusInf && (top < __builtin_huge_valf() || x == top);
  }
  __device__ __forceinline__ double weight(float x) const {
    return x == top ? 1.0 : alive(x) ? pow2(((double)x - (double)top) * rate) : 0.0;
  }
  __device__ __forceinline__ unsigned long long units(float x) const {
    // rounded by the add: its sum's last bit is a unit
    return __builtin_bit_cast(unsigned long long, __builtin_amdgcn_ldexp(weight(x), shift) + 0x1p52) & 0xfffffffffffffull;
  }

  // First bin at which the histogram's running sum reaches target (>= 1), and
  // the sum before it; bin kBins where it never does.  total: of all bins.
  __device__ void reach(unsigned long long target, int& bin, unsigned long long& before, unsigned long long& total) const {
    constexpr int PER = kBins / NT;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    unsigned long long h[PER], mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine += h[i] = hist[tid * PER + i];
    unsigned long long run = mine;
#pragma unroll
    for (int o = 1; o < 64; o <<= 1) {
      const unsigned long long n = __shfl_up(run, o);
      if (lane >= o) run += n;
    }
    if (lane == 63) wsum[wave] = run;
    if (tid == 0) wsum[W] = kBins, wsum[W + 1] = 0;
    __syncthreads();
    unsigned long long at = run - mine;
    total = 0;
    for (int i = 0; i < W; ++i) {
      if (i < wave) at += wsum[i];
      total += wsum[i];
    }
    if (at < target && at + mine >= target) {
#pragma unroll
      for (int i = 0; i < PER; ++i) {
        if (at < target && at + h[i] >= target) wsum[W] = tid * PER + i, wsum[W + 1] = at;
        at += h[i];
      }
    }
    __syncthreads();
    bin = (int)wsum[W];
    before = wsum[W + 1];
    __syncthreads();
  }
  __device__ void clear() const {
    for (int i = threadIdx.x; i < kBins; i += NT) hist[i] = 0;
    __syncthreads();
  }

  // The first index (in index order) at which the running sum of f(z, index)
  // exceeds target, or share * the whole sum where target < 0.
  template <typename F>
  __device__ int walk(F f, double target, double share, double& whole) const {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int vecs = (vocab + 7) >> 3, turns = (vecs + NT - 1) / NT;
    double* sums = (double*)hist;  // [turns][W] <= kBins
    for (int t = 0; t < turns; ++t) {
      const int v = t * NT + tid;
      double s = 0;
      if (v < vecs) {
        float x[8];
        get(v, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) s += f(x[e], 8 * v + e);
      }
#pragma unroll
      for (int o = 32; o; o >>= 1) s += __shfl_xor(s, o);
      if (lane == 0) sums[t * W + wave] = s;
    }
    __syncthreads();
    // one wave finds the 512 logits that hold the place, then the place
    if (wave == 0) {
      const int slots = turns * W, per = (slots + 63) / 64;
      double mine = 0;
      for (int i = lane * per; i < min(slots, (lane + 1) * per); ++i) mine += sums[i];
      double run = mine;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double n = __shfl_up(run, o);
        if (lane >= o) run += n;
      }
      const double total = __shfl(run, 63);
      const double goal = target < 0 ? share * total : target;
      // the first lane whose part passes the goal, else the last with any mass
      uint64_t hit = __ballot(mine > 0 && run > goal), any = __ballot(mine > 0);
      int slot = 0;
      double at = 0;
      if (any) {
        const int l = hit ? __builtin_ctzll(hit) : 63 - __builtin_clzll(any);
        at = __shfl(run - mine, l);
        slot = -1;
        for (int i = l * per; i < min(slots, (l + 1) * per); ++i) {
          const double s = sums[i];
          if (s <= 0) continue;
          if (slot >= 0) at += sums[slot];
          slot = i;
          if (at + s > goal) break;
        }
      }
      // slot: 64 vectors, one per lane
      const int v = (slot / W) * NT + (slot % W) * 64 + lane;
      float x[8];
      double w[8], own = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 0;
      if (v < vecs) {
        get(v, x);
#pragma unroll
        for (int e = 0; e < 8; ++e) own += w[e] = f(x[e], 8 * v + e);
      }
      run = own;
#pragma unroll
      for (int o = 1; o < 64; o <<= 1) {
        const double n = __shfl_up(run, o);
        if (lane >= o) run += n;
      }
      hit = __ballot(own > 0 && at + run > goal);
      any = __ballot(own > 0);
      int found = -1;
      if (any) {
        const int l = hit ? __builtin_ctzll(hit) : 63 - __builtin_clzll(any);
        double here = at + (run - own);
        int best = -1;
        bool past = false;
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          if (w[e] > 0 && !past) best = 8 * v + e;
          here += w[e];
          past = past || (w[e] > 0 && here > goal);
        }
        found = __shfl(best, l);
      }
      if (lane == 0) {
        wsum[W] = (unsigned long long)(long long)found;
        wsum[W + 1] = __builtin_bit_cast(unsigned long long, total);
      }
    }
    __syncthreads();
    const int found = (int)(long long)wsum[W];
    whole = __builtin_bit_cast(double, wsum[W + 1]);
    __syncthreads();
    return found;
  }

  // Tightens the cut to the shortest prefix that holds `count` logits (MASS
  // false) or the share p of the mass that the cut keeps so far (MASS).  low:
  // the smallest logit with a weight.
  template <bool MASS>
  __device__ void select(double amount, float low, float temperature, Cut& cut) const {
    auto measure = [&](float x) -> unsigned long long { return MASS ? units(x) : 1ull; };
    // classes of equal width, over what can matter: 2^-64 of the best and
    // more, or every logit
    const float d = top - low;
    const float wide = MASS ? fminf(45.f * temperature, d) : d;
    const float scale = wide > 0.f && wide < 3e38f ? (float)kBins / wide : 0.f;
    const bool flat = !(scale < 3e38f);
    auto klass = [&](float x) -> int {
      const float at = flat ? 0.f : (top - x) * scale;
      return x == top ? 0 : (int)fminf(at, (float)(kBins - 1));
    };
    clear();
    each([&](float x, int i) {
      if (alive(x) && cut.keeps(key_of(x), i)) {
        const unsigned long long w = measure(x);
        if (w) atomicAdd(&hist[klass(x)], w);
      }
    });
    __syncthreads();
    int bin;
    unsigned long long before, total, sum;
    unsigned long long goal = 1;
    if constexpr (MASS) {
      // the total first
      reach(~0ull, bin, before, total);
      goal = (unsigned long long)__builtin_ceil(amount * (double)total);
      if (goal < 1) goal = 1;
    } else {
      goal = (unsigned long long)amount;
    }
    reach(goal, bin, before, total);
    if (bin >= kBins) return;  // fewer than that are left
    const int in = bin;
    // the digits of the class's keys, from the first in which they differ
    uint32_t lo = ~0u, hi = 0;
    each([&](float x, int i) {
      const uint32_t k = key_of(x);
      if (alive(x) && cut.keeps(k, i) && klass(x) == in && measure(x)) lo = min(lo, k), hi = max(hi, k);
    });
#pragma unroll
    for (int o = 32; o; o >>= 1) {
      lo = min(lo, (uint32_t)__shfl_xor((int)lo, o));
      hi = max(hi, (uint32_t)__shfl_xor((int)hi, o));
    }
    if ((threadIdx.x & 63) == 0) wsum[threadIdx.x >> 6] = (unsigned long long)lo << 32 | hi;
    __syncthreads();
    for (int i = 0; i < W; ++i) lo = min(lo, (uint32_t)(wsum[i] >> 32)), hi = max(hi, (uint32_t)wsum[i]);
    __syncthreads();
    unsigned long long ties = 0;
    for (;;) {
      const int bits = lo == hi ? 0 : 32 - __builtin_clz(lo ^ hi);
      const int drop = bits > 11 ? bits - 11 : 0;
      const uint32_t base = drop + 11 < 32 ? lo >> (drop + 11) << (drop + 11) : 0;
      clear();
      each([&](float x, int i) {
        const uint32_t k = key_of(x);
        if (k >= lo && k <= hi && alive(x) && cut.keeps(k, i) && klass(x) == in) {
          const unsigned long long w = measure(x);
          if (w) atomicAdd(&hist[kBins - 1 - ((k - base) >> drop)], w);
        }
      });
      __syncthreads();
      unsigned long long add;
      reach(goal - before, bin, add, sum);
      before += add;
      ties = hist[bin];
      __syncthreads();
      const uint32_t digit = base + ((uint32_t)(kBins - 1 - bin) << drop);
      lo = max(lo, digit);
      hi = min(hi, digit + ((1u << drop) - 1));
      if (drop == 0) break;
    }
    // lo is the border's key; of its equals the first `want` stay
    const unsigned long long each_ = measure(of_key(lo));
    const unsigned long long want = (goal - before + each_ - 1) / each_;
    if (want * each_ >= ties) {  // all of them
      if (lo != cut.key) cut.index = 0x7fffffff;
      cut.key = lo;
      return;
    }
    const Cut was = cut;
    double whole;
    const int last = walk([&](float x, int i) { return key_of(x) == lo && was.keeps(lo, i) ? 1.0 : 0.0; },
                          (double)(want - 1), 0.0, whole);
    cut.key = lo;
    cut.index = last;
  }
};

template <typename T, int NT>
__global__ void __launch_bounds__(NT) sample_kernel(Sample p) {
  constexpr int W = NT / 64;
  __shared__ unsigned long long hist[kBins];
  __shared__ unsigned long long wsum[W + 4];
  const int row = blockIdx.x, tid = threadIdx.x;
  constexpr int kBytes = __is_same(T, F32) ? 4 : 2;
  Row<T, NT> r;
  r.z = (const char*)p.logits + (size_t)row * p.ld * kBytes;
  r.vocab = p.vocab;
  r.hist = hist;
  r.wsum = wsum;
  r.shift = min(51, 62 - (32 - __builtin_clz(p.vocab)));  // a weight is below 2^52, the histogram's sum below 2^63
  float hi = kMinusInf, lo = __builtin_huge_valf();
  r.each([&](float x, int) {
    hi = fmaxf(hi, x);
    lo = fminf(lo, x > kMinusInf ? x : lo);
  });
#pragma unroll
  for (int o = 32; o; o >>= 1) {
    hi = fmaxf(hi, __shfl_xor(hi, o));
    lo = fminf(lo, __shfl_xor(lo, o));
  }
  if ((tid & 63) == 0)
    wsum[tid >> 6] = (unsigned long long)__builtin_bit_cast(uint32_t, hi) << 32 | __builtin_bit_cast(uint32_t, lo);
  __syncthreads();
  for (int i = 0; i < W; ++i) {
    hi = fmaxf(hi, __builtin_bit_cast(float, (uint32_t)(wsum[i] >> 32)));
    lo = fminf(lo, __builtin_bit_cast(float, (uint32_t)wsum[i]));
  }
  __syncthreads();
  if (!(hi > kMinusInf)) {  // nothing to draw
    if (tid == 0) {
      p.token[row] = -1;
      if (p.logprob) p.logprob[row] = kMinusInf;
    }
    return;
  }
  r.top = hi;
  const float temperature = p.temperature ? p.temperature[row] : 1.f;
  const bool greedy = !(temperature > 0.f);
  Cut cut = {kAll, 0};
  r.rate = greedy ? 0.0 : 1.44269504088896340736 / (double)temperature;
  if (greedy) {
    double whole;
    const int at = r.walk([&](float x, int) { return x == hi ? 1.0 : 0.0; }, 0.0, 0.0, whole);
    if (tid == 0) {
      p.token[row] = at;
      if (p.logprob) p.logprob[row] = 0.f;
    }
    return;
  }
  if (hi == __builtin_huge_valf()) lo = hi;
  const int k = p.top_k ? p.top_k[row] : 0;
  if (k > 0 && k < p.vocab) r.template select<false>((double)k, lo, temperature, cut);
  const float top_p = p.top_p ? p.top_p[row] : 1.f;
  if (top_p < 1.f) r.template select<true>((double)fmaxf(top_p, 0.f), lo, temperature, cut);
  const float min_p = p.min_p ? p.min_p[row] : 0.f;
  const double least = min_p > 0.f ? (double)fminf(min_p, 1.f) : 0.0;
  const float u = p.u[row];
  const double share = u > 0.f ? (double)fminf(u, 0x1.fffffep-1f) : 0.0;
  double whole;
  const int at = r.walk(
      [&](float x, int i) {
        if (!cut.keeps(key_of(x), i)) return 0.0;
        const double w = r.weight(x);
        return w >= least ? w : 0.0;
      },
      -1.0, share, whole);
  if (tid == 0) {
    p.token[row] = at;
    if (p.logprob) p.logprob[row] = (float)log(r.weight(up1<T>(r.z, at)) / whole);
  }
}

template <typename T>
hipError_t launch_type(const Sample& p, hipStream_t st) {
  if (p.vocab <= 4096)
    hipLaunchKernelGGL((sample_kernel<T, 256>), dim3(p.rows), dim3(256), 0, st, p);
  else
    hipLaunchKernelGGL((sample_kernel<T, 1024>), dim3(p.rows), dim3(1024), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_sample(const Sample& p, int type, hipStream_t st) {
  switch (type) {
    case OUT_F16: return launch_type<F16>(p, st);
    case OUT_BF16: return launch_type<BF16>(p, st);
    default: return launch_type<F32>(p, st);
  }
}

}  // namespace rq
