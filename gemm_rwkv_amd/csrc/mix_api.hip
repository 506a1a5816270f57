// C ABI of the operators between an RWKV-7 layer's projections
// (include/rq.h): argument checks, then one launch or two on the caller's
// stream.
#include <hip/hip_runtime.h>
#include <string.h>

#include "kernels.h"
#include "mix.h"
#include "rq.h"
#include "validate.h"

using rqv::Span;

namespace {

constexpr int64_t kMostWidth = 8192;  // a row is held in the registers of one workgroup
constexpr int64_t kMostMix = 8;
constexpr int64_t kMostGrid = (int64_t)1 << 21;  // workgroups of one launch

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

int hip_status(hipError_t e) { return e == hipSuccess ? RQ_OK : RQ_ERR_HIP; }

Span bytes_span(const void* p, size_t n) {
  Span s;
  s.lo = (uintptr_t)p;
  s.hi = p ? s.lo + n : s.lo;
  return s;
}

// What a call reads and writes; no output may overlap anything else, except
// one that is exactly the input it may replace.
struct Buffers {
  static constexpr int kMost = 32;
  Span in[kMost], out[kMost];
  const void* same[kMost];  // the input that out[i] may replace
  int nin = 0, nout = 0;
  int status = RQ_OK;

  void fail(int st) {
    if (status == RQ_OK) status = st;
  }
  bool pointer(const void* p, bool needed) {
    if (!p) {
      if (needed) fail(RQ_ERR_NULL);
      return false;
    }
    if (!rqv::aligned16(p)) fail(RQ_ERR_ALIGN);
    return true;
  }
  void read(const void* p, size_t n, bool needed = true) {
    if (pointer(p, needed)) in[nin++] = bytes_span(p, n);
  }
  void write(const void* p, size_t n, bool needed = true, const void* may_be = nullptr) {
    if (!pointer(p, needed)) return;
    same[nout] = may_be;
    out[nout++] = bytes_span(p, n);
  }
  // 16-bit rows [m][ld], n used per row
  // no rows may be no array: an empty tensor's address is null
  void read_rows(const void* p, int64_t m, int64_t n, int64_t ld, bool needed = true) {
    if (pointer(p, needed && m > 0)) in[nin++] = rqv::act_span(p, m, n, ld, 2);
  }
  void write_rows(const void* p, int64_t m, int64_t n, int64_t ld, bool needed = true) {
    if (!pointer(p, needed && m > 0)) return;
    same[nout] = nullptr;
    out[nout++] = rqv::act_span(p, m, n, ld, 2);
  }
  // int32 indices
  void read_index(const void* p, int64_t n) {
    if (!p) return;
    if (!aligned4(p)) fail(RQ_ERR_ALIGN);
    in[nin++] = bytes_span(p, (size_t)n * 4);
  }
  int check(const void* ws, size_t ws_bytes) {
    if (status != RQ_OK) return status;
    for (int i = 0; i < nout; ++i) {
      for (int j = 0; j < nin; ++j)
        if (rqv::overlaps(out[i], in[j]) && !(same[i] && in[j].lo == (uintptr_t)same[i] && out[i].lo == in[j].lo))
          return RQ_ERR_ALIAS;
      for (int j = i + 1; j < nout; ++j)
        if (rqv::overlaps(out[i], out[j])) return RQ_ERR_ALIAS;
    }
    if (ws) {
      if (!rqv::aligned16(ws)) return RQ_ERR_ALIGN;
      const Span w = bytes_span(ws, ws_bytes);
      for (int i = 0; i < nin; ++i)
        if (rqv::overlaps(w, in[i])) return RQ_ERR_ALIAS;
      for (int i = 0; i < nout; ++i)
        if (rqv::overlaps(w, out[i])) return RQ_ERR_ALIAS;
    }
    return RQ_OK;
  }
};

// The workspace past the split counters, which these operators leave alone.
float* parts_of(void* ws, size_t ws_bytes, size_t& n) {
  n = ws && ws_bytes > rq::kSplitCounterBytes ? ws_bytes - rq::kSplitCounterBytes : 0;
  return n ? (float*)((uint8_t*)ws + rq::kSplitCounterBytes) : nullptr;
}

int check_type(int dtype) { return dtype == RQ_F16 || dtype == RQ_BF16 ? RQ_OK : RQ_ERR_FORMAT; }

int check_ld(int64_t rows, int64_t width, int64_t ld) {
  if (ld < width || ld >= rqv::kMaxDim || rows * ld >= ((int64_t)1 << 40)) return RQ_ERR_SHAPE;
  return ld % 8 ? RQ_ERR_ALIGN : RQ_OK;
}

int check_heads(int64_t tokens, int64_t heads, int64_t ld) {
  if (tokens < 0 || tokens >= rqv::kMaxDim - 64 || heads < 1 || heads > (1 << 20)) return RQ_ERR_SHAPE;
  return check_ld(tokens, heads * rq::kHead, ld);
}

int check_seqs(int64_t tokens, const void* cu, int64_t nseq) {
  if (nseq < 0 || nseq >= kMostGrid || (tokens > 0 && nseq == 0)) return RQ_ERR_SHAPE;
  if (!cu && nseq > 0 && tokens % nseq != 0) return RQ_ERR_SHAPE;
  return RQ_OK;
}

rq::Sequences sequences(const int32_t* cu, int64_t nseq, int64_t tokens) {
  rq::Sequences s;
  s.cu = cu;
  s.nseq = (int)nseq;
  s.len = nseq ? (int)(tokens / nseq) : 0;
  s.tokens = (int)tokens;
  return s;
}

// slots [nseq] into an array of nslots states; without a map, sequence i is slot i
int check_slots(const void* slots, int64_t nslots, int64_t nseq, bool used) {
  if (!used) return RQ_OK;
  if (nslots < 0 || nslots >= kMostGrid || (!slots && nslots < nseq)) return RQ_ERR_SHAPE;
  return RQ_OK;
}

bool eps_ok(float eps) { return eps >= 0.f && eps <= 1e30f; }

constexpr size_t kStateBytes = (size_t)rq::kHead * rq::kHead * 4;

}  // namespace

extern "C" {

int rq_time_mix(int dtype, const void* r, const void* w, const void* k, const void* v, const void* a, const void* b,
                int64_t tokens, int64_t heads, int64_t ld, const int32_t* cu, int64_t nseq, const float* state_in,
                float* state_out, const int32_t* slots, int64_t nslots, void* y, int64_t ldy, void* workspace,
                size_t workspace_bytes, void* stream) {
  int st;
  if ((st = check_type(dtype)) != RQ_OK) return st;
  if ((st = check_heads(tokens, heads, ld)) != RQ_OK) return st;
  if ((st = check_seqs(tokens, cu, nseq)) != RQ_OK) return st;
  if ((st = check_slots(slots, nslots, nseq, state_in || state_out)) != RQ_OK) return st;
  const int64_t width = heads * rq::kHead;
  if ((st = check_ld(tokens, width, ldy)) != RQ_OK) return st;
  if (nseq * heads >= kMostGrid || (state_in || state_out ? nslots * heads : 0) >= ((int64_t)1 << 40)) return RQ_ERR_SHAPE;
  Buffers io;
  const void* rows[6] = {r, w, k, v, a, b};
  for (int i = 0; i < 6; ++i) io.read_rows(rows[i], tokens, width, ld);
  const size_t states = (size_t)(nslots * heads) * kStateBytes;
  io.read(state_in, states, false);
  io.read_index(cu, nseq + 1);
  io.read_index(slots, nseq);
  io.write(state_out, states, false, state_in);
  io.write_rows(y, tokens, width, ldy);
  if ((st = io.check(workspace, workspace_bytes)) != RQ_OK) return st;
  if (nseq == 0 || (tokens == 0 && !state_out)) return RQ_OK;
  rq::TimeMix p;
  memset(&p, 0, sizeof(p));
  p.r = r; p.w = w; p.k = k; p.v = v; p.a = a; p.b = b;
  p.heads = (int)heads;
  p.ld = (int)ld;
  p.seq = sequences(cu, nseq, tokens);
  p.slots.map = slots;
  p.slots.count = (int)nslots;
  p.state_in = state_in;
  p.state_out = state_out;
  p.y = y;
  p.ldy = (int)ldy;
  p.parts = parts_of(workspace, workspace_bytes, p.parts_bytes);
  return hip_status(rq::launch_time_mix(p, dtype == RQ_BF16, (hipStream_t)stream));
}

size_t rq_time_mix_backward_bytes(int64_t tokens, int64_t heads, int64_t nseq) {
  if (tokens < 0 || tokens >= rqv::kMaxDim || heads < 1 || heads > (1 << 20) || nseq < 0 || nseq >= kMostGrid) return 0;
  return rq::kSplitCounterBytes + rq::time_mix_back_bytes(tokens, heads, nseq);
}

int rq_time_mix_backward(int dtype, const void* r, const void* w, const void* k, const void* v, const void* a,
                         const void* b, int64_t tokens, int64_t heads, int64_t ld, const int32_t* cu, int64_t nseq,
                         const float* state_in, const void* dy, const float* dstate_out, void* dr, void* dw, void* dk,
                         void* dv, void* da, void* db, float* dstate_in, void* workspace, size_t workspace_bytes,
                         void* stream) {
  int st;
  if ((st = check_type(dtype)) != RQ_OK) return st;
  if ((st = check_heads(tokens, heads, ld)) != RQ_OK) return st;
  if ((st = check_seqs(tokens, cu, nseq)) != RQ_OK) return st;
  if (nseq * heads >= kMostGrid || (tokens / 16 + nseq) * heads >= ((int64_t)1 << 24)) return RQ_ERR_SHAPE;
  const int64_t width = heads * rq::kHead;
  Buffers io;
  const void* rows[7] = {r, w, k, v, a, b, dy};
  for (int i = 0; i < 7; ++i) io.read_rows(rows[i], tokens, width, ld);
  void* grads[6] = {dr, dw, dk, dv, da, db};
  for (int i = 0; i < 6; ++i) io.write_rows(grads[i], tokens, width, ld);
  const size_t states = (size_t)(nseq * heads) * kStateBytes;
  io.read(state_in, states, false);
  io.read(dstate_out, states, false);
  io.read_index(cu, nseq + 1);
  io.write(dstate_in, states, false);
  if ((st = io.check(workspace, workspace_bytes)) != RQ_OK) return st;
  if (nseq == 0 || (tokens == 0 && !dstate_in)) return RQ_OK;
  rq::TimeMixBack p;
  memset(&p, 0, sizeof(p));
  p.f.r = r; p.f.w = w; p.f.k = k; p.f.v = v; p.f.a = a; p.f.b = b;
  p.f.heads = (int)heads;
  p.f.ld = (int)ld;
  p.f.seq = sequences(cu, nseq, tokens);
  p.f.slots.count = (int)nseq;
  p.f.state_in = state_in;
  p.f.parts = parts_of(workspace, workspace_bytes, p.f.parts_bytes);
  if (p.f.parts_bytes < rq::time_mix_back_bytes(tokens, heads, nseq)) return RQ_ERR_WORKSPACE;
  p.dy = dy;
  p.dstate_out = dstate_out;
  p.dr = dr; p.dw = dw; p.dk = dk; p.dv = dv; p.da = da; p.db = db;
  p.dstate_in = dstate_in;
  return hip_status(rq::launch_time_mix_back(p, dtype == RQ_BF16, (hipStream_t)stream));
}

int rq_shift_norm(int dtype, const void* x, const void* delta, float alpha, int64_t tokens, int64_t width, int64_t ld,
                  const int32_t* cu, int64_t nseq, const float* gamma, const float* beta, float eps, const float* mu,
                  int64_t nmix, const void* shift_in, void* shift_out, const int32_t* slots, int64_t nslots,
                  void* x_out, void* out, int64_t ldo, void* stream) {
  int st;
  if ((st = check_type(dtype)) != RQ_OK) return st;
  if (tokens < 0 || tokens >= rqv::kMaxDim - 64 || width < 8 || width > kMostWidth || nmix < 1 || nmix > kMostMix)
    return RQ_ERR_SHAPE;
  if (width % 8) return RQ_ERR_ALIGN;
  if ((st = check_ld(tokens, width, ld)) != RQ_OK) return st;
  if ((st = check_ld(tokens * nmix, width, ldo)) != RQ_OK) return st;
  if ((st = check_seqs(tokens, cu, nseq)) != RQ_OK) return st;
  if ((st = check_slots(slots, nslots, nseq, shift_in || shift_out)) != RQ_OK) return st;
  if (!eps_ok(eps)) return RQ_ERR_VALUE;
  Buffers io;
  io.read_rows(x, tokens, width, ld);
  io.read_rows(delta, tokens, width, ld, false);
  const size_t params = (size_t)width * 4;
  io.read(gamma, params);
  io.read(beta, params);
  io.read(mu, params * nmix);
  const size_t shifts = (size_t)nslots * width * 2;
  io.read(shift_in, shifts, false);
  io.read_index(cu, nseq + 1);
  io.read_index(slots, nseq);
  io.write(shift_out, shifts, false, shift_in);
  io.write_rows(x_out, tokens, width, ld, false);
  io.write_rows(out, tokens * nmix, width, ldo);
  if ((st = io.check(nullptr, 0)) != RQ_OK) return st;
  if (nseq == 0 || (tokens == 0 && !shift_out)) return RQ_OK;
  rq::ShiftNorm p;
  memset(&p, 0, sizeof(p));
  p.x = x;
  p.delta = delta;
  p.alpha = alpha;
  p.width = (int)width;
  p.ld = (int)ld;
  p.seq = sequences(cu, nseq, tokens);
  p.slots.map = slots;
  p.slots.count = (int)nslots;
  p.gamma = gamma;
  p.beta = beta;
  p.eps = eps;
  p.mu = mu;
  p.nmix = (int)nmix;
  p.shift_in = shift_in;
  p.shift_out = shift_out;
  p.x_out = x_out;
  p.out = out;
  p.ldo = (int)ldo;
  return hip_status(rq::launch_shift_norm(p, dtype == RQ_BF16, (hipStream_t)stream));
}

int rq_shift_norm_backward(int dtype, const void* x, float alpha, int64_t tokens, int64_t width, int64_t ld,
                           const int32_t* cu, int64_t nseq, const float* gamma, const float* beta, float eps,
                           const float* mu, int64_t nmix, const void* shift_in, const void* dout, int64_t ldo,
                           const void* dx_out, const void* dshift_out, void* dx, void* ddelta, void* dshift_in,
                           float* dgamma, float* dbeta, float* dmu, void* workspace, size_t workspace_bytes,
                           void* stream) {
  int st;
  if ((st = check_type(dtype)) != RQ_OK) return st;
  if (tokens < 0 || tokens >= rqv::kMaxDim - 64 || width < 8 || width > kMostWidth || nmix < 1 || nmix > kMostMix)
    return RQ_ERR_SHAPE;
  if (width % 8) return RQ_ERR_ALIGN;
  if ((st = check_ld(tokens, width, ld)) != RQ_OK) return st;
  if ((st = check_ld(tokens * nmix, width, ldo)) != RQ_OK) return st;
  if ((st = check_seqs(tokens, cu, nseq)) != RQ_OK) return st;
  if (!eps_ok(eps)) return RQ_ERR_VALUE;
  Buffers io;
  const size_t params = (size_t)width * 4, shifts = (size_t)nseq * width * 2;
  io.read_rows(x, tokens, width, ld);
  io.read(gamma, params);
  io.read(beta, params);
  io.read(mu, params * nmix);
  io.read(shift_in, shifts, false);
  io.read_rows(dout, tokens * nmix, width, ldo);
  io.read_rows(dx_out, tokens, width, ld, false);
  io.read(dshift_out, shifts, false);
  io.read_index(cu, nseq + 1);
  io.write_rows(dx, tokens, width, ld);
  io.write_rows(ddelta, tokens, width, ld, false);
  io.write(dshift_in, shifts, false);
  io.write(dgamma, params);
  io.write(dbeta, params);
  io.write(dmu, params * nmix);
  if ((st = io.check(workspace, workspace_bytes)) != RQ_OK) return st;
  rq::ShiftNormBack p;
  memset(&p, 0, sizeof(p));
  p.x = x;
  p.alpha = alpha;
  p.width = (int)width;
  p.ld = (int)ld;
  p.seq = sequences(cu, nseq, tokens);
  p.gamma = gamma;
  p.beta = beta;
  p.eps = eps;
  p.mu = mu;
  p.nmix = (int)nmix;
  p.shift_in = shift_in;
  p.dout = dout;
  p.ldo = (int)ldo;
  p.dx_out = dx_out;
  p.dshift_out = dshift_out;
  p.dx = dx;
  p.ddelta = ddelta;
  p.dshift_in = dshift_in;
  p.dgamma = dgamma;
  p.dbeta = dbeta;
  p.dmu = dmu;
  p.parts = parts_of(workspace, workspace_bytes, p.parts_bytes);
  return hip_status(rq::launch_shift_norm_back(p, dtype == RQ_BF16, (hipStream_t)stream));
}

int rq_head_gate(int dtype, const void* y, const void* r, const void* k, const void* v, const void* g, int64_t tokens,
                 int64_t heads, int64_t ld, const float* gamma, const float* beta, float eps, const float* u, void* out,
                 int64_t ldo, void* stream) {
  int st;
  if ((st = check_type(dtype)) != RQ_OK) return st;
  if ((st = check_heads(tokens, heads, ld)) != RQ_OK) return st;
  const int64_t width = heads * rq::kHead;
  if ((st = check_ld(tokens, width, ldo)) != RQ_OK) return st;
  if (!eps_ok(eps)) return RQ_ERR_VALUE;
  Buffers io;
  const void* rows[5] = {y, r, k, v, g};
  for (int i = 0; i < 5; ++i) io.read_rows(rows[i], tokens, width, ld);
  const size_t params = (size_t)width * 4;
  io.read(gamma, params);
  io.read(beta, params);
  io.read(u, params);
  io.write_rows(out, tokens, width, ldo);
  if ((st = io.check(nullptr, 0)) != RQ_OK) return st;
  if (tokens == 0) return RQ_OK;
  rq::HeadGate p;
  p.y = y; p.r = r; p.k = k; p.v = v; p.g = g;
  p.tokens = (int)tokens;
  p.heads = (int)heads;
  p.ld = (int)ld;
  p.gamma = gamma;
  p.beta = beta;
  p.u = u;
  p.eps = eps;
  p.out = out;
  p.ldo = (int)ldo;
  return hip_status(rq::launch_head_gate(p, dtype == RQ_BF16, (hipStream_t)stream));
}

int rq_head_gate_backward(int dtype, const void* y, const void* r, const void* k, const void* v, const void* g,
                          int64_t tokens, int64_t heads, int64_t ld, const float* gamma, const float* beta, float eps,
                          const float* u, const void* dout, void* dy, void* dr, void* dk, void* dv, void* dg,
                          float* dgamma, float* dbeta, float* du, void* workspace, size_t workspace_bytes,
                          void* stream) {
  int st;
  if ((st = check_type(dtype)) != RQ_OK) return st;
  if ((st = check_heads(tokens, heads, ld)) != RQ_OK) return st;
  const int64_t width = heads * rq::kHead;
  if (!eps_ok(eps)) return RQ_ERR_VALUE;
  Buffers io;
  const void* rows[6] = {y, r, k, v, g, dout};
  for (int i = 0; i < 6; ++i) io.read_rows(rows[i], tokens, width, ld);
  void* grads[5] = {dy, dr, dk, dv, dg};
  for (int i = 0; i < 5; ++i) io.write_rows(grads[i], tokens, width, ld);
  const size_t params = (size_t)width * 4;
  io.read(gamma, params);
  io.read(beta, params);
  io.read(u, params);
  io.write(dgamma, params);
  io.write(dbeta, params);
  io.write(du, params);
  if ((st = io.check(workspace, workspace_bytes)) != RQ_OK) return st;
  rq::HeadGateBack p;
  memset(&p, 0, sizeof(p));
  p.f.y = y; p.f.r = r; p.f.k = k; p.f.v = v; p.f.g = g;
  p.f.tokens = (int)tokens;
  p.f.heads = (int)heads;
  p.f.ld = (int)ld;
  p.f.gamma = gamma;
  p.f.beta = beta;
  p.f.u = u;
  p.f.eps = eps;
  p.dout = dout;
  p.dy = dy; p.dr = dr; p.dk = dk; p.dv = dv; p.dg = dg;
  p.dgamma = dgamma;
  p.dbeta = dbeta;
  p.du = du;
  p.parts = parts_of(workspace, workspace_bytes, p.parts_bytes);
  return hip_status(rq::launch_head_gate_back(p, dtype == RQ_BF16, (hipStream_t)stream));
}

}  // extern "C"
