// What the entry points' argument checks share (sequence.cpp, attention.cpp).  Host code.
#pragma once
#include <hip/hip_runtime.h>

#include <cstdint>
#include <exception>
#include <string>

#include "sequence.h"

namespace {

using sc::report;

inline sc_status fail(sc_status s, const char* msg) { return (sc_status)report(s, msg); }

// Runs an entry point's body; no exception leaves it.
template <class F>
sc_status guarded(F body) {
  try {
    report(SC_OK, "");
    return body();
  } catch (const std::exception&) {
    return SC_ENOMEM;
  }
}

inline int64_t size_of(int dtype) { return dtype == SC_F32 ? 4 : 2; }

// A strided tensor of `outer` blocks of `rows` rows of `len` contiguous values of `es` bytes.
struct View {
  const void* p;
  int64_t outer, rows, len, outer_stride, row_stride, es;
  int64_t last() const {  // values up to the last one's end
    return (outer - 1) * outer_stride + (rows - 1) * row_stride + len;
  }
  bool empty() const { return !p || outer <= 0 || rows <= 0 || len <= 0; }
};

constexpr int64_t kMaxStride = 1LL << 40;  // values; a tensor's whole span is held below 1e17 as well

inline bool strides_ok(const View& v) {
  if (v.outer_stride < 0 || v.row_stride < 0 || v.outer_stride > kMaxStride || v.row_stride > kMaxStride) return false;
  // the span in bytes stays far inside 64 bits
  return (long double)v.outer * v.outer_stride + (long double)v.rows * v.row_stride + v.len < 1e17L;
}

// Whether two of the tensor's values share an address.
inline bool self_overlaps(const View& v) {
  if (v.empty()) return false;
  const int64_t os = v.outer_stride, rs = v.row_stride;
  const bool blocks = (v.rows == 1 || rs >= v.len) && (v.outer == 1 || os >= (v.rows - 1) * rs + v.len);
  const bool rows = (v.outer == 1 || os >= v.len) && (v.rows == 1 || rs >= (v.outer - 1) * os + v.len);
  return !blocks && !rows;
}

// Whether two tensors may share an address: their spans meet, and they are not two channel ranges
// of one tensor (equal strides, each block's rows inside the other's gap).
inline bool overlap(const View& a, const View& b) {
  if (a.empty() || b.empty()) return false;
  const intptr_t a0 = (intptr_t)a.p, b0 = (intptr_t)b.p;
  if (a0 + a.last() * a.es <= b0 || b0 + b.last() * b.es <= a0) return false;
  if (a.es == b.es && a.outer_stride == b.outer_stride && a.outer_stride > 0) {
    const int64_t period = a.outer_stride * a.es;
    const int64_t wa = ((a.rows - 1) * a.row_stride + a.len) * a.es, wb = ((b.rows - 1) * b.row_stride + b.len) * b.es;
    const int64_t off = (((int64_t)b0 - (int64_t)a0) % period + period) % period;  // b's block after a's
    if (off >= wa && off + wb <= period) return false;
  }
  return true;
}

inline bool misaligned(const void* p, int64_t to) { return ((uintptr_t)p & (uintptr_t)(to - 1)) != 0; }

inline sc_status launched(int e) {
  if (e == (int)hipSuccess) return SC_OK;
  return (sc_status)report(SC_EDEVICE, std::string("kernel launch failed: ") + hipGetErrorString((hipError_t)e));
}

// CUs of the current device (256 where there is none: sizes can be asked for without a GPU).
inline int device_cus() {
  int dev = 0, cus = 0;
  if (hipGetDevice(&dev) != hipSuccess ||
      hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus < 1) {
    (void)hipGetLastError();
    return 256;
  }
  return cus;
}

}  // namespace
