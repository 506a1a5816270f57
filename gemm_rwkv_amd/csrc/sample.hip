// One token per row of logits z:
//
//   w_i = exp((z_i - max z) / T)
//
// in the order of falling z, equal ones by rising index: the first top_k stay;
// of those the shortest prefix that holds top_p of their mass; of those the
// ones with w_i >= min_p.  The token is the first of the kept ones, by index,
// whose cumulative mass exceeds u times the kept mass.
//
// A token changes when an error moves any border between kept tokens over u's
// place, and there may be 65536 of them, so weights are fp64 to 2^-46 and sums
// fp64 in a fixed order: that, some 20 fp64 operations a logit, and the row's way
// through one compute unit are what bounds the draw.
//
// Every filter keeps a prefix of that order, and the row is never sorted.
//   - top_k up to 256: the r-th largest of the threads' own maxima in each wave,
//     the least over the waves, is passed by at least top_k logits and by few
//     more; those go to a list of up to 512.
//   - Otherwise a histogram over 4096 classes of z, of counts for top_k, of
//     weights for top_p, tells the class that the border falls into, and the
//     class's own logits, or all up to it if they are few, go to the list.
//   - A list is ranked by comparing all pairs.  One that holds all that is kept
//     is filtered and drawn from; one of a border's class gives the cut, a key
//     (the float's bits in the order of its values) and an index, that the draw
//     over the row goes by.
//   - A class with more than 512 members (equal logits, most of all) is told
//     apart by histograms of its keys' digits.
// Histograms are of integers (counts, or weights in units of 2^-shift that fit
// 64 bits), so the order of the atomic adds changes no bit.
//
// A workgroup has a row; its waves own consecutive parts of it, 8 logits a lane
// and turn.  One row of 65536 in fp16 (128 KB) takes 15.9 us with top_k 50, top_p
// and min_p (4 for the largest, 5 for the list, 5 to rank and draw), 21.6 with no
// filter (13 for the weights' sums, 3 to find the place), 41 with top_p alone
// (20 for the histogram, 7 to fetch the border's class, then the draw), 44 with
// top_k 5000.  509 rows of 50277 in bf16 take 41 with no filter, 1.2 TB/s, of which
// the weights' instructions are some 13; the rest is the pass for the largest
// logit before them, and two workgroups to a compute unit that take the same
// passes at the same time.  509 rows of 65536 in fp16 take 123 with top_p alone:
// the draw's walk makes a weight of every logit, also of those past the cut.
#include "mix.h"
#include "next_token.h"

namespace rq {

namespace {

constexpr int kBins = 4096;
constexpr int kParts = 8;       // sums that four lanes keep of their turns
constexpr int kList = 512;      // logits of the short list
constexpr int kListTopK = 256;  // the largest top_k that maxima are asked for
constexpr float kMinusInf = -__builtin_huge_valf(), kInf = __builtin_huge_valf();
// Weights below 2^-990 count as 0.  Those, -inf, NaN and places past the row's end
// are made 2^-1015: 2^20 of them are nothing still, and no sum that holds the
// largest logit's 1 sees them.
constexpr double kNothing = 0x1p-990, kFloor = -1015;

// p r + c with c in scalar registers (as a plain fma it becomes two instructions,
// c copied to where the sum is made).
__device__ __forceinline__ double horner(double p, double r, double c) {
  asm("v_fma_f64 %0, %1, %2, %3" : "=v"(p) : "v"(p), "v"(r), "s"(c));
  return p;
}

// 2^(d rate), above 2^-1022, by Taylor's series in the part r of d rate past the
// nearest whole number.  The first term left out is 2^-46.7 of the value at r = -1/2,
// beside some 2^-52 of rounding.
__device__ __forceinline__ double pow2(double d, double rate) {
  constexpr double kRound = 0x1.8p52;  // with it added, the whole number is in the low bits
  const double a = __builtin_fma(d, rate, kRound), r = __builtin_fma(d, rate, -(a - kRound));
  double p = __builtin_fma(4.44553827187081e-10, r, 7.054911620801121e-09);  // ln(2)^k / k!, k = 11, 10, ...
  p = horner(p, r, 1.0178086009239696e-07);
  p = horner(p, r, 1.3215486790144305e-06);
  p = horner(p, r, 1.5252733804059838e-05);
  p = horner(p, r, 0.00015403530393381606);
  p = horner(p, r, 0.0013333558146428441);
  p = horner(p, r, 0.009618129107628477);
  p = horner(p, r, 0.055504108664821576);
  p = horner(p, r, 0.2402265069591007);
  p = horner(p, r, 0.6931471805599453);
  p = __builtin_fma(p, r, 1.0);
  return __builtin_bit_cast(double, __builtin_bit_cast(uint64_t, p) + ((uint64_t)(uint32_t)__builtin_bit_cast(uint64_t, a) << 52));
}
// The larger, or the one that is no NaN.  (fmax would first see to signalling NaN.)
__device__ __forceinline__ double larger(double d, double floor) {
  asm("v_max_f64 %0, %1, %2" : "=v"(d) : "v"(d), "s"(floor));
  return d;
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
struct Vec {  // 8 logits as they lie in memory
  typedef uint16_t Raw;
  static constexpr Raw kNone = (Raw)T::kMinusInf2;
  uint4 v;
  __device__ __forceinline__ void load(const void* row, int at) { v = *(const uint4*)((const uint16_t*)row + at); }
  __device__ __forceinline__ void none() { v = make_uint4(T::kMinusInf2, T::kMinusInf2, T::kMinusInf2, T::kMinusInf2); }
  static __device__ __forceinline__ float one(const void* row, int at) { return T::up(((const uint16_t*)row)[at]); }
  __device__ __forceinline__ void up(float* z) const {
    up2<T>(v.x, z);
    up2<T>(v.y, z + 2);
    up2<T>(v.z, z + 4);
    up2<T>(v.w, z + 6);
  }
};
template <>
struct Vec<F32> {
  typedef float Raw;
  static constexpr Raw kNone = kMinusInf;
  float4 a, b;
  __device__ __forceinline__ void load(const void* row, int at) {
    a = *(const float4*)((const float*)row + at);
    b = *(const float4*)((const float*)row + at + 4);
  }
  __device__ __forceinline__ void none() { a = b = make_float4(kMinusInf, kMinusInf, kMinusInf, kMinusInf); }
  static __device__ __forceinline__ float one(const void* row, int at) { return ((const float*)row)[at]; }
  __device__ __forceinline__ void up(float* z) const {
    z[0] = a.x, z[1] = a.y, z[2] = a.z, z[3] = a.w, z[4] = b.x, z[5] = b.y, z[6] = b.z, z[7] = b.w;
  }
};

// The float after x (finite, or -inf).
__device__ __forceinline__ float after(float x) {
  if (x == 0.f) return __builtin_bit_cast(float, 1u);
  const int b = __builtin_bit_cast(int, x);
  return __builtin_bit_cast(float, b < 0 ? b - 1 : b + 1);
}

// The cut: what comes after (z, index) in the order is out.
struct Cut {
  float z = kMinusInf;
  int index = 0x7fffffff;
  __device__ __forceinline__ bool none() const { return z == kMinusInf; }
  // What the logits of the vector from `at` on have to reach, all of them alike
  // except in the one vector that holds the index.
  __device__ __forceinline__ float bar(int at) const { return at <= index ? z : after(z); }
  __device__ __forceinline__ bool split(int at) const { return at <= index && index < at + 7; }
  // f(e, whether l[e] stays)
  template <typename F>
  __device__ __forceinline__ void each(const float* l, int at, F f) const {
    const float b = bar(at);
    if (split(at)) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f(e, l[e] >= bar(at + e));
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) f(e, l[e] >= b);
    }
  }
  __device__ __forceinline__ bool keeps(float x, int i) const { return x >= bar(i); }
};

template <int NT>
struct Shared {
  static constexpr int W = NT / 64;
  union {
    unsigned long long hist[kBins];
    double part[kParts][NT / 4];
    struct {
      // key and ~index: larger comes first; a border's class in the second half
      alignas(16) unsigned long long order[2 * kList];
      unsigned long long sorted[kList];
      double weight[kList];  // in the order
      double partial[NT];
      int rank[kList];
    } list;
  };
  uint4 tail[2];  // the row's last logits past whole vectors, filled up with -inf
  unsigned long long wave[W];
  unsigned long long said[2];
  double kept;
  int lanes[W];  // of each wave, those that have a logit
  int count[2], least;
};

// (a reference kept in a struct would lose that it is to LDS)
template <int NT>
__device__ __forceinline__ Shared<NT>& shared_of() {
  __shared__ Shared<NT> s;
  return s;
}

// Sum over each four lanes / the wave.
template <int CTRL>
__device__ __forceinline__ double dpp_d(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v);
  const uint32_t lo = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)b, CTRL, 0xf, 0xf, true);
  const uint32_t hi = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)(uint32_t)(b >> 32), CTRL, 0xf, 0xf, true);
  return __builtin_bit_cast(double, (uint64_t)hi << 32 | lo);
}
__device__ __forceinline__ double quad_sum(double v) {
  v += dpp_d<0xb1>(v);  // quad_perm 1,0,3,2
  return v + dpp_d<0x4e>(v);
}
__device__ __forceinline__ double across_quads(double v) {
#pragma unroll
  for (int o = 32; o > 2; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
__device__ __forceinline__ double sum_of(double v) {
#pragma unroll
  for (int o = 32; o; o >>= 1) v += __shfl_xor(v, o);
  return v;
}
// The wave's largest.
__device__ __forceinline__ float wave_most(float v) {
  v = fmaxf(v, dpp<0x128>(v));  // row_ror 8, 4, 2, 1
  v = fmaxf(v, dpp<0x124>(v));
  v = fmaxf(v, dpp<0x122>(v));
  v = fmaxf(v, dpp<0x121>(v));
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
// Sum over this lane and those before it.
template <typename N>
__device__ __forceinline__ N running(N v) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const N n = __shfl_up(v, o);
    if (lane >= o) v += n;
  }
  return v;
}

// A value that every lane has alike, for a scalar register.
template <typename N>
__device__ __forceinline__ N uniform(N v) {
  if constexpr (sizeof(N) == 8) {
    const uint64_t b = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)b);
    const uint32_t hi = (uint32_t)__builtin_amdgcn_readfirstlane((int)(uint32_t)(b >> 32));
    return __builtin_bit_cast(N, (uint64_t)hi << 32 | lo);
  } else {
    return __builtin_bit_cast(N, __builtin_amdgcn_readfirstlane(__builtin_bit_cast(int, v)));
  }
}

template <typename T, int NT>
struct Row {
  static constexpr int W = NT / 64;
  const void* z;
  int vocab, turns;
  float top, low;  // the largest logit, the smallest that is finite
  bool infinite;   // the largest is +inf: it counts as 0 and all else as -inf
  double rate;     // log2(e) / T
  double floor;    // kFloor / rate
  double scale;    // units of the histograms in a weight of 1

  static __device__ __forceinline__ Shared<NT>& shared() { return shared_of<NT>(); }

  __device__ __forceinline__ int first_vec() const { return (int)(threadIdx.x >> 6) * turns * 64 + (int)(threadIdx.x & 63); }
  // The 8 logits of vector v, places past the row's end as -inf.  (Any load is
  // of a whole vector; a row of fewer than 8 has none.)
  __device__ __forceinline__ Vec<T> fetch(int v) const {
    Vec<T> x;
    const int whole = vocab >> 3;
    if (whole > 0) {
      x.load(z, 8 * min(v, whole - 1));
      if (v >= whole) x.none();
    } else {
      x.none();
    }
    if (v == whole) x.load(shared().tail, 0);
    return x;
  }
  __device__ __forceinline__ void open(const Vec<T>& x, float* f) const {
    x.up(f);
    if (infinite)
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = f[e] == kInf ? 0.f : kMinusInf;
  }
  // f(8 logits, index of the first) for this thread's part of the row, AHEAD
  // vectors loaded at once: four where f is short, one, with the next on its
  // way, where it is long enough to wait behind.
  template <int AHEAD, typename F>
  __device__ __forceinline__ void vectors(F f) const {
    const int v0 = first_vec();
    if constexpr (AHEAD == 1) {
      Vec<T> next = fetch(v0);
#pragma unroll 1
      for (int t = 0; t < turns; ++t) {
        const Vec<T> x = next;
        next = fetch(v0 + 64 * (t + 1));
        float l[8];
        open(x, l);
        f(l, 8 * (v0 + 64 * t));
      }
    } else {
      // (turns past the last one read the next wave's part: its logits are left out)
#pragma unroll 1
      for (int t = 0; t < turns; t += AHEAD) {
        Vec<T> x[AHEAD];
#pragma unroll
        for (int a = 0; a < AHEAD; ++a) x[a] = fetch(v0 + 64 * (t + a));
#pragma unroll
        for (int a = 0; a < AHEAD; ++a)
          if (t + a < turns) {
            float l[8];
            open(x[a], l);
            f(l, 8 * (v0 + 64 * (t + a)));
          }
      }
    }
  }
  template <typename F>
  __device__ __forceinline__ void each(F f) const {
    vectors<1>([&](const float* l, int at) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f(l[e], at + e);
    });
  }
  __device__ __forceinline__ double weight(float x) const { return pow2(larger((double)x - (double)top, floor), rate); }
  // rounded by the add: its sum's last bit is a unit
  __device__ __forceinline__ unsigned long long units(float x) const {
    return __builtin_bit_cast(unsigned long long, __builtin_fma(weight(x), scale, 0x1p52)) & 0xfffffffffffffull;
  }

  // A logit's class, and what it adds to the class's bin.  It goes by half the
  // distance from the top, which fp32 holds whatever two finite logits are.
  __device__ __forceinline__ float half_below(float x) const { return __builtin_fmaf(-0.5f, x, 0.5f * top); }
  __device__ __forceinline__ int klass_of(float x, float per) const {
    return per < 3e38f ? (int)fminf(half_below(x) * per, (float)(kBins - 1)) : x == top ? 0 : 1;
  }
  __device__ __forceinline__ unsigned long long measure(bool mass, float x) const {
    return mass ? units(x) : x > kMinusInf ? 1ull : 0ull;
  }

  // The first index (in index order) at which the running sum of what f(8 logits,
  // index of the first, e) gives for the e-th exceeds target, or share * the
  // whole sum where target < 0.
  template <typename F>
  __device__ __forceinline__ int walk(F f, double target, double share, double& whole) const {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int group = (turns + kParts - 1) / kParts;  // turns to a part
    double mine = 0, now = 0;
    int part = 0, left = group;
    auto keep = [&]() {
      now = quad_sum(now);
      if ((tid & 3) == 0) shared().part[part][tid >> 2] = now;
      ++part;
      mine += now;
      now = 0;
    };
    vectors<1>([&](const float* l, int at) {
      double v = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) v += f(l[e], at, e);
      now += v;
      if (--left == 0) {
        keep();
        left = group;
      }
    });
    if (left != group) keep();
    const int parts = part;
    mine = across_quads(mine);
    if (lane == 0) shared().wave[wave] = __builtin_bit_cast(unsigned long long, mine);
    if (tid == 0) shared().said[0] = ~0ull;
    __syncthreads();
    // the wave whose part of the row passes the goal, else the last with any mass
    const double theirs = lane < W ? __builtin_bit_cast(double, shared().wave[lane & (W - 1)]) : 0.0;
    const double upto = running(theirs);
    const double total = __shfl(upto, 63);
    const double goal = target < 0 ? share * total : target;
    const uint64_t any = __ballot(theirs > kNothing), hit = __ballot(theirs > kNothing && upto > goal);
    const int at_wave = hit ? __builtin_ctzll(hit) : any ? 63 - __builtin_clzll(any) : -1;
    if (wave == at_wave) {
      // its part, then the turn, the lane and the logit, each the same way
      double sums[kParts], at = __shfl(upto - theirs, at_wave), run = at;
#pragma unroll
      for (int i = 0; i < kParts; ++i) sums[i] = i < parts ? shared().part[i][tid >> 2] : 0.0;
#pragma unroll
      for (int i = 0; i < kParts; ++i) sums[i] = across_quads(sums[i]);
      int at_part = 0;
      bool past = false;
#pragma unroll
      for (int i = 0; i < kParts; ++i) {
        if (sums[i] > kNothing && !past) {
          at_part = i;
          at = run;
          past = run + sums[i] > goal;
        }
        run += sums[i];
      }
      run = at;
      int found = -1;
#pragma unroll 1
      for (int t = at_part * group; t < min(turns, (at_part + 1) * group); ++t) {
        const int v = first_vec() + 64 * t;
        float l[8];
        open(fetch(v), l);
        double w[8], own = 0;
#pragma unroll
        for (int e = 0; e < 8; ++e) own += w[e] = f(l[e], 8 * v, e);
        const double upto = running(own);
        const uint64_t any = __ballot(own > kNothing), hit = __ballot(own > kNothing && run + upto > goal);
        if (any) {
          const int holder = hit ? __builtin_ctzll(hit) : 63 - __builtin_clzll(any);
          double here = run + (upto - own);
          int best = -1;
          bool past = false;
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            if (w[e] > kNothing && !past) best = 8 * v + e;
            here += w[e];
            past = past || (w[e] > kNothing && here > goal);
          }
          found = __shfl(best, holder);
          if (hit) break;
        }
        run += __shfl(upto, 63);
      }
      if (lane == 0) shared().said[0] = (unsigned long long)(long long)found;
    }
    __syncthreads();
    whole = uniform(total);
    const int found = uniform((int)shared().said[0]);
    __syncthreads();
    return found;
  }

  // First bin at which the histogram's running sum reaches goal(its total) (>= 1),
  // and the sum before it; bin kBins where it never does.
  template <typename G>
  __device__ __forceinline__ void reach(G goal_of, int& bin, unsigned long long& before) const {
    constexpr int PER = kBins / NT;
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    unsigned long long mine = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) mine += shared().hist[tid * PER + i];
    const unsigned long long run = running(mine);
    if (lane == 63) shared().wave[wave] = run;
    if (tid == 0) shared().said[0] = kBins, shared().said[1] = 0;
    __syncthreads();
    unsigned long long at = run - mine, total = 0;
    for (int i = 0; i < W; ++i) {
      if (i < wave) at += shared().wave[i];
      total += shared().wave[i];
    }
    const unsigned long long goal = goal_of(uniform(total));
    if (at < goal && at + mine >= goal) {
#pragma unroll 1
      for (int i = 0; i < PER; ++i) {
        const unsigned long long h = shared().hist[tid * PER + i];
        if (at + h >= goal) {
          shared().said[0] = tid * PER + i, shared().said[1] = at;
          break;
        }
        at += h;
      }
    }
    __syncthreads();
    bin = uniform((int)shared().said[0]);
    before = uniform(shared().said[1]);
    __syncthreads();
  }
  __device__ __forceinline__ void clear() const {
    for (int i = threadIdx.x; i < kBins; i += NT) shared().hist[i] = 0;
    __syncthreads();
  }

  // order[base ..] of n members, ranked into sorted[], with their weights.  Every
  // pair is compared: thread (i, share) has its share of the others.
  __device__ __forceinline__ void rank(int base, int n) const {
    const int tid = threadIdx.x;
    unsigned long long* order = shared().list.order + base;
    for (int i = tid; i < kList; i += NT) shared().list.rank[i] = 0;
    if (tid == 0 && (n & 1)) order[n] = 0;
    __syncthreads();
    int width = 64;
    while (width < n && width < NT) width <<= 1;
    const int shares = NT / width, share = tid / width;
    for (int i = tid & (width - 1); i < n; i += width) {
      const unsigned long long own = order[i];
      int before = 0;
      // two to a read; a place past the list holds 0, which is before nothing
#pragma unroll 4
      for (int j = 2 * share; j < n; j += 2 * shares) {
        const ulonglong2 o = *(const ulonglong2*)(order + j);
        before += (int)(o.x > own) + (int)(o.y > own);
      }
      if (before) atomicAdd(&shared().list.rank[i], before);
    }
    __syncthreads();
    for (int i = tid; i < n; i += NT) {
      const int place = shared().list.rank[i];
      shared().list.sorted[place] = order[i];
      shared().list.weight[place] = weight(of_key((uint32_t)(order[i] >> 32)));
    }
    __syncthreads();
  }

  // Draws from order[0 .. n), which holds all that is kept: the first top_k (0:
  // all), of those the prefix that reaches goal (or, where goal < 0 and top_p <
  // 1, top_p of their mass), of those w >= least.
  __device__ __forceinline__ int draw_short(int n, int top_k, float top_p, double goal, double least, double share,
                                            double& kept) const {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    if (tid == 0) shared().least = 0x7fffffff;
    rank(0, n);
    // filters, by one wave: eight in a row to a lane
    if (wave == 0) {
      const int stay = top_k ? min(top_k, n) : n;
      constexpr int PER = kList / 64;
      double w[PER], own = 0;
#pragma unroll
      for (int e = 0; e < PER; ++e) own += w[e] = lane * PER + e < stay ? shared().list.weight[lane * PER + e] : 0.0;
      const double upto = running(own);
      if (goal < 0) goal = (double)fmaxf(top_p, 0.f) * __shfl(upto, 63);
      double at = upto - own;
      int held = 0;
#pragma unroll
      for (int e = 0; e < PER; ++e) {
        const int place = lane * PER + e;
        held += place < stay && (place == 0 || ((!(top_p < 1.f) || at < goal) && w[e] >= least && w[e] > kNothing));
        at += w[e];
      }
#pragma unroll
      for (int o = 32; o; o >>= 1) held += __shfl_xor(held, o);
      double in = 0;
#pragma unroll
      for (int e = 0; e < PER; ++e) in += lane * PER + e < held ? w[e] : 0.0;
      in = sum_of(in);
      if (lane == 0) shared().said[0] = (unsigned)held, shared().kept = in;
    }
    __syncthreads();
    const int held = (int)shared().said[0];
    kept = shared().kept;
    // each kept one's mass before it in index order; the order of the list fixes
    // the order of the sums
    int width = 64;
    while (width < held && width < NT) width <<= 1;
    const int pieces = NT / width, piece = tid / width;
    for (int a = tid & (width - 1); a < held; a += width) {
      double before = 0;
      const uint32_t own = (uint32_t)shared().list.sorted[a];  // ~index
#pragma unroll 4
      for (int j = piece; j < held; j += pieces) before += (uint32_t)shared().list.sorted[j] > own ? shared().list.weight[j] : 0.0;
      if (pieces > 1) {
        shared().list.partial[tid] = before;
      } else if (before + shared().list.weight[a] > share * kept) {
        atomicMin(&shared().least, (int)~own);
      }
    }
    __syncthreads();
    if (pieces > 1 && tid < held) {
      double before = 0;
      for (int j = 0; j < pieces; ++j) before += shared().list.partial[j * width + tid];
      if (before + shared().list.weight[tid] > share * kept) atomicMin(&shared().least, (int)~(uint32_t)shared().list.sorted[tid]);
    }
    __syncthreads();
    int token = shared().least;
    __syncthreads();
    if (token == 0x7fffffff) {  // rounding left u's place past the last one
      token = 0;
      for (int j = 0; j < held; ++j) token = max(token, (int)~(uint32_t)shared().list.sorted[j]);
    }
    return token;
  }

  // The logits that reach the wanted number's bar, onto the list.  most: this
  // thread's largest.  How many; more than kList are not all there.
  __device__ __forceinline__ int list_best(float most, int want) const {
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    // each wave's share goes by its lanes that have a logit; a last wave whose part
    // is cut short, and its maxima low, is not asked, where others are there
    const int full = ((vocab + 7) >> 3) / (64 * turns), asked = full ? full : W;
    const int lanes = wave < asked ? shared().lanes[wave] : 0;
    int all = 0;
    for (int i = 0; i < asked; ++i) all += shared().lanes[i];
    all = max(all, 1);
    const int quota = (want * lanes + all - 1) / all;
    // the quota-th largest: the largest taken out quota - 1 times, or from about 8
    // on (0.2 us each) the lanes sorted (1.8 us)
    float v = most, mine;
    if (quota <= 8) {
      mine = wave_most(v);
#pragma unroll 1
      for (int i = 1; i < quota; ++i) {
        if (lane == __builtin_ctzll(__ballot(v == mine))) v = kMinusInf;
        mine = wave_most(v);
      }
    } else {
#pragma unroll
      for (int k = 2; k <= 64; k <<= 1)
#pragma unroll
        for (int o = k >> 1; o; o >>= 1) {
          const float n = __shfl_xor(v, o);
          const bool larger = ((lane & k) == 0) == ((lane & o) == 0);  // this lane keeps the larger of the two
          v = larger ? fmaxf(v, n) : fminf(v, n);
        }
      mine = __shfl(v, min(quota, 64) - 1);
    }
    if (lane == 0) shared().wave[wave] = __builtin_bit_cast(uint32_t, lanes == 0 ? kInf : quota > lanes ? kMinusInf : mine);
    if (tid == 0) shared().count[0] = 0;
    __syncthreads();
    float bar = kInf;
    for (int i = 0; i < W; ++i) bar = fminf(bar, __builtin_bit_cast(float, (uint32_t)shared().wave[i]));
    auto take = [&](const float* l, int at) {
      float m = l[0];
#pragma unroll
      for (int e = 1; e < 8; ++e) m = fmaxf(m, l[e]);
      if (!(m >= bar) || !(m > kMinusInf)) return;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (l[e] >= bar && l[e] > kMinusInf) {
          const int place = atomicAdd(&shared().count[0], 1);
          if (place < kList) shared().list.order[place] = (unsigned long long)key_of(l[e]) << 32 | (uint32_t)~(at + e);
        }
    };
    vectors<4>(take);
    __syncthreads();
    const int n = uniform(shared().count[0]);
    __syncthreads();
    return n;
  }

  // The border of the shortest prefix of what the cut keeps that holds `amount`
  // logits or, where mass, that share of its mass.  Returns how many
  // logits, all up to the border's class, are on the list, goal then being the
  // mass to reach; or 0, the cut being tightened to the border (or left alone
  // where there are no more than `amount`).
  __device__ __forceinline__ int select(bool mass, double amount, float temperature, Cut& cut, double& goal_out) const {
    const int tid = threadIdx.x;
    // classes of equal width, over what can matter: 2^-64 of the best and
    // more, or every logit (in halves, as half_below() is); where that is too
    // little to divide, two: the largest ones and the others
    const float wide = mass ? fminf(22.5f * temperature, half_below(low)) : half_below(low);
    const float per = wide > 0.f ? (float)kBins / wide : kInf;
    const bool flat = !(per < 3e38f);
    const Cut was = cut;
    auto klass = [&](float x) { return klass_of(x, per); };
    clear();
    auto add = [&](auto of) {
      vectors<1>([&](const float* l, int at) {
        was.each(l, at, [&](int e, bool stays) {
          const unsigned long long w = of(l[e]);
          if (w && stays) atomicAdd(&shared().hist[klass(l[e])], w);
        });
      });
    };
    if (mass)
      add([&](float x) { return units(x); });
    else
      add([&](float x) { return x > kMinusInf ? 1ull : 0ull; });
    __syncthreads();
    int bin;
    unsigned long long before, goal = 1;
    reach(
        [&](unsigned long long total) {
          if (mass) {
            goal = max((unsigned long long)__builtin_ceil(amount * (double)total), 1ull);
            goal_out = amount * (double)total / scale;
          } else {
            goal = (unsigned long long)amount;
          }
          return goal;
        },
        bin, before);
    if (bin >= kBins) return 0;
    const int in = bin;
    const unsigned long long held = uniform(shared().hist[in]);
    // the class's members in the second half of the list, those before it in the
    // first, until a wave sees that they are too many
    if (tid == 0) shared().count[0] = shared().count[1] = 0;
    __syncthreads();
    // values between which the class lies, past any rounding of klass()
    const float around = fmaxf(wide, 0.5f * fabsf(top)) * 0x1p-20f;
    const float below = flat ? kMinusInf : 2.f * (0.5f * top - ((float)in + 1.f) / per - around);
    float above = kInf;
    bool full = false;
    vectors<1>([&](const float* l, int at) {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const bool near = l[e] >= below && l[e] <= above;
        if (__ballot(near) == 0) continue;
        const int c = klass(l[e]);
        const bool stays = near && c <= in && l[e] > kMinusInf && was.keeps(l[e], at + e);
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const bool mine = stays && (c == in) == (half == 1);
          const uint64_t who = __ballot(mine);
          if (who == 0 || (half == 0 && full)) continue;
          int place = 0;
          if ((tid & 63) == __builtin_ctzll(who)) place = atomicAdd(&shared().count[half], __popcll(who));
          place = __shfl(place, __builtin_ctzll(who)) + __popcll(who & ((1ull << (tid & 63)) - 1));
          if (mine && place < kList)
            shared().list.order[half * kList + place] = (unsigned long long)key_of(l[e]) << 32 | (uint32_t)~(at + e);
          if (half == 0 && __ballot(mine && place >= kList)) {
            full = true;
            if (!flat) above = 2.f * (0.5f * top - (float)in / per + around);
          }
        }
      }
    });
    __syncthreads();
    const int less = uniform(shared().count[0]), same = uniform(shared().count[1]);
    __syncthreads();
    if (less + same <= kList) {
      if (less < kList)
        for (int i = tid; i < same; i += NT) shared().list.order[less + i] = shared().list.order[kList + i];
      __syncthreads();
      return less + same;
    }
    if (same <= kList) {
      rank(kList, same);
      if (tid < 64) {
        constexpr int PER = kList / 64;
        unsigned long long own = 0, w[PER];
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          const int place = tid * PER + e;
          own += w[e] = place < same ? measure(mass, of_key((uint32_t)(shared().list.sorted[place] >> 32))) : 0;
        }
        unsigned long long at = before + running(own) - own;
#pragma unroll
        for (int e = 0; e < PER; ++e) {
          if (at < goal && at + w[e] >= goal) shared().said[0] = shared().list.sorted[tid * PER + e];
          at += w[e];
        }
      }
      __syncthreads();
      const unsigned long long at = uniform(shared().said[0]);
      cut.z = of_key((uint32_t)(at >> 32));
      cut.index = (int)~(uint32_t)at;
      __syncthreads();
      return 0;
    }
    narrow(mass, per, was, in, before, goal, held, cut);
    return 0;
  }

  // The border among a class's `held`, which the list has no room for, `before`
  // being the sum of the classes before it and `goal` the one to reach: by
  // histograms of the digits of the members' keys, from the first in which they
  // differ.
  __device__ __forceinline__ void narrow(bool mass, float per, const Cut& was, int in, unsigned long long before,
                                         unsigned long long goal, unsigned long long held, Cut& cut) const {
    const int tid = threadIdx.x;
    unsigned long long ties = held;
    auto member = [&](float x, int i) { return x > kMinusInf && klass_of(x, per) == in && was.keeps(x, i); };
    uint32_t lo = ~0u, hi = 0;
    each([&](float x, int i) {
      const uint32_t k = key_of(x);
      if (member(x, i) && measure(mass, x)) lo = min(lo, k), hi = max(hi, k);
    });
#pragma unroll
    for (int o = 32; o; o >>= 1) {
      lo = min(lo, (uint32_t)__shfl_xor((int)lo, o));
      hi = max(hi, (uint32_t)__shfl_xor((int)hi, o));
    }
    if ((tid & 63) == 0) shared().wave[tid >> 6] = (unsigned long long)lo << 32 | hi;
    __syncthreads();
    for (int i = 0; i < W; ++i) lo = min(lo, (uint32_t)(shared().wave[i] >> 32)), hi = max(hi, (uint32_t)shared().wave[i]);
    lo = uniform(lo), hi = uniform(hi);
    __syncthreads();
    constexpr int kDigit = 12;
    static_assert(1 << kDigit == kBins, "a digit has a bin");
    for (int digits = 0; lo != hi && digits < (32 + kDigit - 1) / kDigit; ++digits) {
      const int bits = 32 - __builtin_clz(lo ^ hi);
      const int drop = bits > kDigit ? bits - kDigit : 0;
      const uint32_t base = drop + kDigit < 32 ? lo >> (drop + kDigit) << (drop + kDigit) : 0;
      clear();
      each([&](float x, int i) {
        const uint32_t k = key_of(x);
        if (k >= lo && k <= hi && member(x, i)) {
          const unsigned long long w = measure(mass, x);
          if (w) atomicAdd(&shared().hist[kBins - 1 - ((k - base) >> drop)], w);
        }
      });
      __syncthreads();
      int bin;
      unsigned long long add;
      reach([&](unsigned long long) { return goal - before; }, bin, add);
      before += add;
      ties = uniform(shared().hist[bin]);
      __syncthreads();
      const uint32_t digit = base + ((uint32_t)(kBins - 1 - bin) << drop);
      lo = max(lo, digit);
      hi = min(hi, digit + ((1u << drop) - 1));
      if (drop == 0) break;
    }
    // lo is the border's key; of its equals the first `want` stay
    const float border = of_key(lo);
    const unsigned long long one = measure(mass, border);
    const unsigned long long want = (goal - before + one - 1) / one;
    if (want * one >= ties) {  // all of them
      if (border != cut.z) cut.index = 0x7fffffff;
    } else {
      double whole;
      cut.index = walk([&](float x, int at, int e) { return x == border && was.keeps(x, at + e) ? 1.0 : 0.0; },
                       (double)(want - 1), 0.0, whole);
    }
    cut.z = border;
  }
};

// The token of a row that has one to draw, and the kept mass.  most: this
// thread's largest logit.
template <typename T, int NT>
__device__ __forceinline__ int draw(const Row<T, NT>& r, const Sample& p, int row, float temperature, float most, double& whole) {
  int k = p.top_k ? p.top_k[row] : 0;
  if (k < 0 || k >= p.vocab) k = 0;
  const float top_p = p.top_p ? p.top_p[row] : 1.f;
  const float min_p = p.min_p ? p.min_p[row] : 0.f;
  const double least = min_p > 0.f ? (double)fminf(min_p, 1.f) : 0.0;
  const float u = p.u[row];
  const double share = u > 0.f ? (double)fminf(u, 0x1.fffffep-1f) : 0.0;
  int n = 0, want = k;
  double goal = -1.0;
  Cut cut;
  if (k > 0 && k <= kListTopK) n = r.list_best(most, k);
  const bool listed = n > 0 && n <= kList;
  // the border of top_k, then that of top_p
#pragma unroll 1
  for (int pass = listed || k == 0; pass < (listed ? 1 : 2); ++pass) {
    const bool mass = pass == 1;
    if (mass && !(top_p < 1.f)) break;
    n = r.select(mass, mass ? (double)fmaxf(top_p, 0.f) : (double)k, temperature, cut, goal);
    if (n > 0) {
      if (mass) want = 0;  // the list goes by the mass, and holds what top_k left
      break;
    }
  }
  if (n > 0) return r.draw_short(n, want, top_p, want ? -1.0 : goal, least, share, whole);
  if (cut.none() && !(least > 0.0)) return r.walk([&](float x, int, int) { return r.weight(x); }, -1.0, share, whole);
  const float beyond = after(cut.z);
  return r.walk(
      [&](float x, int at, int e) {
        const double w = r.weight(x);
        return x >= (at + e <= cut.index ? cut.z : beyond) && w >= least ? w : 0.0;
      },
      -1.0, share, whole);
}

template <typename T, int NT>
__global__ void __launch_bounds__(NT, 4) sample_kernel(Sample p) {
  constexpr int W = NT / 64;
  Shared<NT>& s = shared_of<NT>();
  const int row = blockIdx.x, tid = threadIdx.x;
  typedef typename Vec<T>::Raw Raw;
  const Raw* z = (const Raw*)p.logits + (size_t)row * p.ld;
  if (tid < 8) ((Raw*)s.tail)[tid] = (p.vocab & ~7) + tid < p.vocab ? z[(p.vocab & ~7) + tid] : Vec<T>::kNone;
  __syncthreads();
  // a weight is below 2^52 units, the histogram's sum below 2^63
  const int shift = min(51, 62 - (32 - __builtin_clz(p.vocab)));
  Row<T, NT> r = {z, p.vocab, (((p.vocab + 7) >> 3) + NT - 1) / NT, 0.f, 0.f, false, 0.0, 0.0, __builtin_amdgcn_ldexp(1.0, shift)};
  // the largest and smallest logit, past NaN
  float most = kMinusInf, low = kInf;
  auto see = [&](float x) {
    most = fmaxf(most, x);
    low = fminf(low, x);
  };
  r.template vectors<16 / sizeof(Raw)>([&](const float* l, int at) {
    if (at + 8 > p.vocab) return;
#pragma unroll
    for (int e = 0; e < 8; ++e) see(l[e]);
  });
  // the thread that owns the last few
  const int last = p.vocab >> 3;
  if (tid == last / (64 * r.turns) * 64 + (last & 63))
    for (int i = p.vocab & ~7; i < p.vocab; ++i) see(Vec<T>::one(z, i));
  const int lanes = __popcll(__ballot(most > kMinusInf));
  float hi = wave_most(most), lo = -wave_most(-low);
  if ((tid & 63) == 0) {
    s.wave[tid >> 6] = (unsigned long long)__builtin_bit_cast(uint32_t, lo) << 32 | __builtin_bit_cast(uint32_t, hi);
    s.lanes[tid >> 6] = lanes;
  }
  __syncthreads();
  for (int i = 0; i < W; ++i) {
    hi = fmaxf(hi, __builtin_bit_cast(float, (uint32_t)s.wave[i]));
    lo = fminf(lo, __builtin_bit_cast(float, (uint32_t)(s.wave[i] >> 32)));
  }
  __syncthreads();
  if (!(hi > kMinusInf)) {  // nothing to draw
    if (tid == 0) {
      p.token[row] = -1;
      if (p.logprob) p.logprob[row] = kMinusInf;
    }
    return;
  }
  hi = uniform(hi);
  const float temperature = p.temperature ? p.temperature[row] : 1.f;
  if (!(temperature > 0.f)) {  // the first of the largest
    int at = 0x7fffffff;
    if (most == hi)
      r.template vectors<4>([&](const float* l, int first) {
#pragma unroll
        for (int e = 0; e < 8; ++e) at = l[e] == hi ? min(at, first + e) : at;
      });
#pragma unroll
    for (int o = 32; o; o >>= 1) at = min(at, __shfl_xor(at, o));
    if ((tid & 63) == 0) s.wave[tid >> 6] = (unsigned)at;
    __syncthreads();
    for (int i = 0; i < W; ++i) at = min(at, (int)s.wave[i]);
    if (tid == 0) {
      p.token[row] = at;
      if (p.logprob) p.logprob[row] = 0.f;
    }
    return;
  }
  // (an infinite temperature's: any two finite logits weigh the same)
  r.rate = fmax(1.44269504088896340736 / (double)temperature, 0x1p-960);
  r.floor = kFloor / r.rate;
  if (hi == kInf) {
    r.infinite = true;
    most = most == kInf ? 0.f : kMinusInf;
    const int with = __popcll(__ballot(most == 0.f));
    if ((tid & 63) == 0) s.lanes[tid >> 6] = with;
    __syncthreads();  // (the row's waves all come here; list_best() reads every wave's number)
    hi = 0.f;
  }
  if (!(lo > kMinusInf)) {  // the smallest finite one
    float least = kInf;
    r.template vectors<1>([&](const float* l, int) {
#pragma unroll
      for (int e = 0; e < 8; ++e) least = l[e] > kMinusInf ? fminf(least, l[e]) : least;
    });
    least = -wave_most(-least);
    if ((tid & 63) == 0) s.wave[tid >> 6] = __builtin_bit_cast(uint32_t, least);
    __syncthreads();
    lo = kInf;
    for (int i = 0; i < W; ++i) lo = fminf(lo, __builtin_bit_cast(float, (uint32_t)s.wave[i]));
    __syncthreads();
  }
  r.top = uniform(hi);
  r.low = uniform(lo);
  double whole;
  const int at = draw(r, p, row, temperature, most, whole);
  if (tid == 0) {
    p.token[row] = at;
    if (p.logprob) {
      const float x = r.infinite ? hi : Vec<T>::one(z, max(at, 0));  // (a row with a largest logit has a token)
      p.logprob[row] = (float)log(r.weight(x) / whole);
    }
  }
}

template <typename T>
hipError_t launch_type(const Sample& p, hipStream_t st) {
  // Up to a row for each of 256 compute units, the row's own time counts: 16 waves.
  // Past that two workgroups of 8 overlap on a unit (one's reads and barriers with
  // the other's arithmetic).  Rows of 65536 in fp16, in us with 8 and 16 waves: 256
  // rows 30 and 28 with no filter, 24 and 23 with top_k 50, 95 and 69 with top_p
  // alone, 79 and 64 with a mixture; 300 rows 42 and 47, 27 and 36, 109 and 95, 95
  // and 75; 509 rows 47 and 51, 31 and 39, 122 and 127, 98 and 94; 900 rows 80 and
  // 96, 53 and 74, 187 and 207, 133 and 146.
  if (p.rows > 256)
    hipLaunchKernelGGL((sample_kernel<T, 512>), dim3(p.rows), dim3(512), 0, st, p);
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
