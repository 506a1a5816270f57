// What a call of the C ABI reads and writes: pointers, alignment and overlaps
// (host C++ only).
#pragma once

#include "validate.h"

namespace rqv {

inline bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

inline Span bytes_span(const void* p, size_t n) {
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
    if (!aligned16(p)) fail(RQ_ERR_ALIGN);
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
    if (pointer(p, needed && m > 0)) in[nin++] = act_span(p, m, n, ld, 2);
  }
  void write_rows(const void* p, int64_t m, int64_t n, int64_t ld, bool needed = true, const void* may_be = nullptr) {
    if (!pointer(p, needed && m > 0)) return;
    same[nout] = may_be;
    out[nout++] = act_span(p, m, n, ld, 2);
  }
  // 32-bit values, one per row or sequence
  void read_index(const void* p, int64_t n, bool needed = false) {
    if (!p) {
      if (needed) fail(RQ_ERR_NULL);
      return;
    }
    if (!aligned4(p)) fail(RQ_ERR_ALIGN);
    in[nin++] = bytes_span(p, (size_t)n * 4);
  }
  void write_index(const void* p, int64_t n, bool needed) {
    if (!p) {
      if (needed) fail(RQ_ERR_NULL);
      return;
    }
    if (!aligned4(p)) fail(RQ_ERR_ALIGN);
    same[nout] = nullptr;
    out[nout++] = bytes_span(p, (size_t)n * 4);
  }
  int check(const void* ws, size_t ws_bytes) {
    if (status != RQ_OK) return status;
    for (int i = 0; i < nout; ++i) {
      for (int j = 0; j < nin; ++j)
        if (overlaps(out[i], in[j]) && !(same[i] && in[j].lo == (uintptr_t)same[i] && out[i].lo == in[j].lo))
          return RQ_ERR_ALIAS;
      for (int j = i + 1; j < nout; ++j)
        if (overlaps(out[i], out[j])) return RQ_ERR_ALIAS;
    }
    if (ws) {
      if (!aligned16(ws)) return RQ_ERR_ALIGN;
      const Span w = bytes_span(ws, ws_bytes);
      for (int i = 0; i < nin; ++i)
        if (overlaps(w, in[i])) return RQ_ERR_ALIAS;
      for (int i = 0; i < nout; ++i)
        if (overlaps(w, out[i])) return RQ_ERR_ALIAS;
    }
    return RQ_OK;
  }
};

}  // namespace rqv
