// The norm over each head's 64 outputs of the state recurrence, the bonus and
// the gate, and their gradient:
//
//   z = (y - mean) rstd gamma + beta + (sum_j r_j k_j u_j) v,   out = z g
//
// with mean and variance over a head's 64 channels.  One pass over five rows
// in and one out (backward: six and five); eight lanes hold a head, eight
// channels each, so the three sums are three lane exchanges and nothing goes
// through LDS.  Bound by memory: 8192 tokens of width 2560 take 50 us, 5.0 TB/s,
// what a copy reaches; 32 tokens of width 4096 2.6 us, a launch.
#include "mix.h"

namespace rq {

// One thread: eight channels of `rows` tokens.  blockDim 256 covers 2048
// channels of one row.
template <typename T>
__global__ void __launch_bounds__(256) head_gate_kernel(HeadGate p, int rows) {
  const int c = (blockIdx.y * 256 + threadIdx.x) * 8;
  const int width = p.heads * kHead;
  if (c >= width) return;  // whole heads: a group of eight lanes leaves together
  float gamma[8], beta[8], u[8];
  load8f(p.gamma + c, gamma);
  load8f(p.beta + c, beta);
  load8f(p.u + c, u);
  const int t0 = blockIdx.x * rows, t1 = run_end(p.tokens, t0, rows);
  for (int t = t0; t < t1; ++t) {
    const size_t at = (size_t)t * p.ld + c;
    float y[8], r[8], k[8], v[8], g[8];
    load8<T>(p.y, at, y);
    load8<T>(p.r, at, r);
    load8<T>(p.k, at, k);
    load8<T>(p.v, at, v);
    load8<T>(p.g, at, g);
    float sum = 0.f, bonus = 0.f, sq = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      sum += y[i];
      bonus = fmaf(r[i] * k[i], u[i], bonus);
    }
    const float mean = oct_sum(sum) * (1.f / kHead);
    bonus = oct_sum(bonus);
#pragma unroll
    for (int i = 0; i < 8; ++i) sq = fmaf(y[i] - mean, y[i] - mean, sq);
    const float rstd = rsqrtf(oct_sum(sq) * (1.f / kHead) + p.eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = fmaf(bonus, v[i], fmaf((y[i] - mean) * rstd, gamma[i], beta[i])) * g[i];
    store8<T>(p.out, (size_t)t * p.ldo + c, y);
  }
}

hipError_t launch_head_gate(const HeadGate& p, bool bf16, hipStream_t st) {
  const int width = p.heads * kHead;
  const int cols = (width / 8 + 255) / 256;
  const int rows = gate_rows(p.tokens);
  const dim3 grid(run_count(p.tokens, rows), cols);
  if (bf16)
    hipLaunchKernelGGL(head_gate_kernel<BF16>, grid, dim3(256), 0, st, p, rows);
  else
    hipLaunchKernelGGL(head_gate_kernel<F16>, grid, dim3(256), 0, st, p, rows);
  return hipGetLastError();
}

// Backward.  With z and n = (y - mean) rstd as above and dz = dout g:
//   dg = dout z, dv = dz bonus, db = sum_j dz_j v_j, dr = db k u, dk = db r u,
//   dn = dz gamma, dy = (dn - mean(dn) - n mean(dn n)) rstd,
//   dgamma = sum_t dz n, dbeta = sum_t dz, du = sum_t db r k.
// A wave covers 512 channels, the workgroup's four waves every fourth of its
// rows; the parameter gradients stay in registers, are added across the waves
// in LDS and written as one row of partial sums per workgroup, so their order
// is fixed.  Bound by memory: 4096 tokens of width 2048 in bf16 take 39 to 44
// us, 4.2 to 4.7 TB/s, and the sums of the partial rows 5 us more.
template <typename T>
__global__ void __launch_bounds__(256, 4) head_gate_back_kernel(HeadGateBack b, int rows) {
  const HeadGate& p = b.f;
  __shared__ float red[4][24][64];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int width = p.heads * kHead;
  const int c = (blockIdx.y * 64 + lane) * 8;
  const bool on = c < width;
  float dgamma[8] = {}, dbeta[8] = {}, du[8] = {};
  if (on) {
    float gamma[8], beta[8], u[8];
    load8f(p.gamma + c, gamma);
    load8f(p.beta + c, beta);
    load8f(p.u + c, u);
    const int t1 = run_end(p.tokens, blockIdx.x * rows, rows);
    for (int t = blockIdx.x * rows + wave; t < t1; t += 4) {
      const size_t at = (size_t)t * p.ld + c;
      float y[8], r[8], k[8], v[8], g[8], d[8];
      load8<T>(p.y, at, y);
      load8<T>(p.r, at, r);
      load8<T>(p.k, at, k);
      load8<T>(p.v, at, v);
      load8<T>(p.g, at, g);
      load8<T>(b.dout, at, d);
      float sum = 0.f, bonus = 0.f, sq = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sum += y[i];
        bonus = fmaf(r[i] * k[i], u[i], bonus);
      }
      const float mean = oct_sum(sum) * (1.f / kHead);
      bonus = oct_sum(bonus);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        y[i] -= mean;
        sq = fmaf(y[i], y[i], sq);
      }
      const float rstd = rsqrtf(oct_sum(sq) * (1.f / kHead) + p.eps);
      float dn[8], dg[8], dv[8], db = 0.f, m1 = 0.f, m2 = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float n = y[i] * rstd;
        const float dz = d[i] * g[i];
        dg[i] = d[i] * fmaf(bonus, v[i], fmaf(n, gamma[i], beta[i]));
        dv[i] = dz * bonus;
        db = fmaf(dz, v[i], db);
        dn[i] = dz * gamma[i];
        m1 += dn[i];
        m2 = fmaf(dn[i], n, m2);
        dgamma[i] = fmaf(dz, n, dgamma[i]);
        dbeta[i] += dz;
        y[i] = n;
      }
      db = oct_sum(db);
      m1 = oct_sum(m1) * (1.f / kHead);
      m2 = oct_sum(m2) * (1.f / kHead);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        dn[i] = (dn[i] - m1 - y[i] * m2) * rstd;
        du[i] = fmaf(db * r[i], k[i], du[i]);
        const float bu = db * u[i], kk = k[i];
        k[i] = bu * r[i];
        r[i] = bu * kk;
      }
      store8<T>(b.dy, at, dn);
      store8<T>(b.dr, at, r);
      store8<T>(b.dk, at, k);
      store8<T>(b.dv, at, dv);
      store8<T>(b.dg, at, dg);
    }
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    red[wave][i][lane] = dgamma[i];
    red[wave][8 + i][lane] = dbeta[i];
    red[wave][16 + i][lane] = du[i];
  }
  __syncthreads();
  // parts[workgroup][3][width], or the gradients themselves with one workgroup
  const int c0 = blockIdx.y * 512;
  for (int e = threadIdx.x; e < 3 * 512; e += 256) {
    const int which = e / 512, col = e % 512;
    if (c0 + col >= width) continue;
    const int j = which * 8 + col % 8, l = col / 8;
    const float s = ((red[0][j][l] + red[1][j][l]) + red[2][j][l]) + red[3][j][l];
    if (gridDim.x == 1)
      (which == 0 ? b.dgamma : which == 1 ? b.dbeta : b.du)[c0 + col] = s;
    else
      b.parts[((size_t)blockIdx.x * 3 + which) * width + c0 + col] = s;
  }
}

// Sums `count` rows of partial sums into up to three outputs, one after the
// other in a row.  64 columns per workgroup, four per thread; 64 groups of
// rows side by side, so that eight rows in flight per thread are all there is
// to wait for; added in a fixed order.
__global__ void __launch_bounds__(1024) sum_parts_kernel(const float* __restrict__ parts, int count, int n, SumTargets to) {
  __shared__ float4v red[64][17];
  const int c4 = threadIdx.x & 15, grp = threadIdx.x >> 4;
  const int col = blockIdx.x * 64 + 4 * c4;
  float4v s = {0.f, 0.f, 0.f, 0.f};
  if (col < n) {
    const float* at = parts + col;
    int i = grp;
    for (; i + 7 * 64 < count; i += 8 * 64) {
      float4v v[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) v[k] = *(const float4v*)(at + (size_t)(i + 64 * k) * n);
#pragma unroll
      for (int k = 0; k < 8; ++k) s += v[k];
    }
    for (; i < count; i += 64) s += *(const float4v*)(at + (size_t)i * n);
  }
  red[grp][c4] = s;
  __syncthreads();
  if (threadIdx.x < 256) {
    // four threads per four columns, sixteen groups each
    const int part = threadIdx.x >> 6, e = threadIdx.x & 63;
    float t = 0.f;
    for (int k = 0; k < 16; ++k) t += red[16 * part + k][e >> 2][e & 3];
    red[16 * part][e >> 2][e & 3] = t;
  }
  __syncthreads();
  if (threadIdx.x < 64 && blockIdx.x * 64 + threadIdx.x < n) {
    const int e = threadIdx.x;
    const float t = ((red[0][e >> 2][e & 3] + red[16][e >> 2][e & 3]) + red[32][e >> 2][e & 3]) + red[48][e >> 2][e & 3];
    int c = blockIdx.x * 64 + e;
    if (c < to.n[0]) {
      to.out[0][c] = t;
    } else if ((c -= to.n[0]) < to.n[1]) {
      to.out[1][c] = t;
    } else {
      to.out[2][c - to.n[1]] = t;
    }
  }
}

hipError_t launch_sum_parts(const float* parts, int count, const SumTargets& to, hipStream_t st) {
  const int n = to.n[0] + to.n[1] + to.n[2];
  hipLaunchKernelGGL(sum_parts_kernel, dim3((n + 63) / 64), dim3(1024), 0, st, parts, count, n, to);
  return hipGetLastError();
}

hipError_t launch_head_gate_back(const HeadGateBack& b, bool bf16, hipStream_t st) {
  const HeadGate& p = b.f;
  const int width = p.heads * kHead;
  const int cols = (width + 511) / 512;
  // rows per workgroup: about 1024 workgroups, at least 16 rows each, and no
  // more partial sums than the workspace holds
  int64_t groups = run_count(p.tokens, 16);
  const int64_t want = (1024 + cols - 1) / cols;
  if (groups > want) groups = want;
  const int64_t fit = b.parts ? (int64_t)(b.parts_bytes / ((size_t)width * 12)) : 0;
  if (groups > fit) groups = fit;
  if (groups < 1) groups = 1;
  const int rows = run_rows(p.tokens, (int)groups);
  if (p.tokens > 0) groups = run_count(p.tokens, rows);
  const dim3 grid((unsigned)groups, cols);
  if (bf16)
    hipLaunchKernelGGL(head_gate_back_kernel<BF16>, grid, dim3(256), 0, st, b, rows);
  else
    hipLaunchKernelGGL(head_gate_back_kernel<F16>, grid, dim3(256), 0, st, b, rows);
  hipError_t e = hipGetLastError();
  if (groups == 1 || e != hipSuccess) return e;
  return launch_sum_parts(b.parts, (int)groups, {{b.dgamma, b.dbeta, b.du}, {width, width, width}}, st);
}

}  // namespace rq
