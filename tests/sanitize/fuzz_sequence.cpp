// Drives the sequence operators' entry points (sequence.cpp) with seeded random argument structures,
// most of them wrong somewhere, with the launchers replaced: a call that passes the checks must be one
// that the kernels could run (the launcher re-derives the spans and sees that nothing overflows or
// overlaps), and no check may overflow, read memory or throw.
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <string>

#include "sequence.h"

namespace {
std::mt19937_64 rng;
int failed = 0, launched = 0;
std::string message;

int64_t pick(std::initializer_list<int64_t> v) { return *(v.begin() + rng() % v.size()); }
bool rare() { return rng() % 24 == 0; }

void check(bool ok, const char* what) {
  if (!ok) {
    failed++;
    std::printf("failed: %s\n", what);
  }
}

// [lo, hi) of a strided tensor, as exact numbers
struct Span {
  __int128 lo, hi;
};
Span span(const void* p, int64_t outer, int64_t rows, int64_t len, int64_t os, int64_t rs, int64_t es) {
  const __int128 at = (uintptr_t)p;
  return {at, at + es * ((__int128)(outer - 1) * os + (__int128)(rows - 1) * rs + len)};
}
bool apart(Span a, Span b) { return a.hi <= b.lo || b.hi <= a.lo; }
}  // namespace

namespace sc {
int report(int status, const std::string& msg) {
  message = msg;
  return status;
}
int launch_causal_conv(const sc_causal_conv& a, void*) {
  launched++;
  const int64_t es = a.dtype == SC_F32 ? 4 : 2;
  check(a.K >= 1 && a.K <= 8 && a.B >= 1 && a.D >= 1 && a.L >= 0, "conv sizes");
  check(a.weight && !((uintptr_t)a.weight & 3), "conv weight");
  if (a.L) {
    const Span out = span(a.out, a.B, a.D, a.L, a.out_batch, a.out_channel, es);
    check(apart(out, span(a.weight, 1, 1, (int64_t)a.D * a.K, 0, 0, 4)), "conv out and weight");
    if (a.x_batch != a.out_batch) check(apart(out, span(a.x, a.B, a.D, a.L, a.x_batch, a.x_channel, es)), "conv out and x");
    if (a.final_state && a.K > 1)
      check(apart(out, span(a.final_state, 1, a.num_slots, (int64_t)a.D * (a.K - 1), 0, a.final_stride, es)), "conv out and state");
  }
  return 0;
}
int launch_selective_scan(const sc_selective_scan& a, int, void*) {
  launched++;
  check(a.N >= 1 && a.N <= 256 && a.D % a.G == 0 && a.B >= 1, "scan sizes");
  if (a.L) check(apart(span(a.out, a.B, a.D, a.L, a.out_batch, a.out_channel, a.dtype == SC_F32 ? 4 : 2),
                       span(a.A, 1, 1, (int64_t)a.D * a.N, 0, 0, 4)), "scan out and A");
  const int64_t need = a.L ? scan_workspace(a, 256) : 0;
  check(!need || (a.workspace && a.workspace_bytes >= need && !((uintptr_t)a.workspace & 15)), "scan workspace");
  return 0;
}
int launch_adapter(const sc_adapter& a, int, void*) {
  launched++;
  check(a.R >= 1 && a.R <= 128 && a.B >= 1 && a.L >= 1 && a.index, "adapter sizes");
  check(!(((uintptr_t)a.down | (uintptr_t)a.up) & 15), "adapter weights");
  return 0;
}
int64_t scan_workspace(const sc_selective_scan& a, int) { return a.L > 256 ? (int64_t)a.B * a.D * (a.N + 1) * 4 : 0; }
int64_t adapter_workspace(const sc_adapter& a, int) { return a.L < 8 ? 0 : (int64_t)a.B * a.R * a.L * 4; }
}  // namespace sc

namespace {
// an address of its own gigabyte, now and then somewhere else, misaligned or NULL
template <class P>
P at(int i) {
  uintptr_t p = (uintptr_t)(i + 1) << 30;
  if (rare()) p = (uintptr_t)(rng() % 16 + 1) << 30;
  if (rare()) p += rng() % 4096;
  if (rare()) p = 0;
  return (P)p;
}
// a product, held inside 60 bits
int64_t times(int64_t a, int64_t b, int64_t c = 1) {
  const __int128 v = (__int128)a * b * c, most = (__int128)1 << 60;
  return (int64_t)(v > most ? most : v < -most ? -most : v);
}
int64_t stride(int64_t usual) {
  if (!rare()) return usual;
  return pick({0, 1, -1, usual - 1, usual + 1, 2 * usual, 1LL << 31, 1LL << 40, 1LL << 41, INT64_MAX, INT64_MIN});
}
int32_t size(int64_t most) {
  if (rare()) return (int32_t)pick({-1, 0, 1, INT32_MAX, INT32_MIN, 1 << 20, 1 << 30});
  return (int32_t)(rng() % most) + 1;
}
}  // namespace

int main(int argc, char** argv) {
  const int rounds = argc > 1 ? std::atoi(argv[1]) : 20000;
  rng.seed(7);
  for (int r = 0; r < rounds; r++) {
    int64_t bytes;
    {
      sc_causal_conv a{at<const void*>(0), at<void*>(1), at<const float*>(2), at<const float*>(3), at<const void*>(4), at<void*>(5),
                       rng() % 2 ? at<const int32_t*>(6) : nullptr, rng() % 2 ? at<const int32_t*>(7) : nullptr};
      a.dtype = (int32_t)pick({0, 1, 2, 2, 1, 0, 3}), a.B = size(6), a.D = size(40), a.L = size(300), a.K = size(8);
      a.x_channel = stride(a.L), a.x_batch = stride(times(a.D, a.L, pick({1, 2}))), a.out_channel = stride(a.L);
      a.out_batch = stride(times(a.D, a.L)), a.num_slots = rare() ? size(9) : 8;
      a.initial_stride = stride(times(a.D, (int64_t)a.K - 1)), a.final_stride = stride(times(a.D, (int64_t)a.K - 1));
      a.flags = (uint32_t)pick({0, 1, 1, 1, 2}), a.reserved = rare();
      const sc_status s = sparseconv_causal_conv(&a, nullptr);
      check(s == SC_OK ? message.empty() : !message.empty(), "conv message");
    }
    {
      sc_selective_scan a{at<const void*>(0), at<const void*>(1), rng() % 2 ? at<const void*>(2) : nullptr, at<const void*>(3),
                          at<const void*>(4), at<void*>(5), at<const float*>(6), at<const float*>(7), at<const float*>(8),
                          at<const float*>(9), at<float*>(10), rng() % 2 ? at<const int32_t*>(11) : nullptr,
                          rng() % 2 ? at<const int32_t*>(12) : nullptr, at<void*>(13), (int64_t)pick({1 << 20, 1 << 28, 0})};
      a.dtype = (int32_t)pick({0, 1, 2, 0, 1, 2, -1}), a.B = size(4), a.G = size(2), a.D = rare() ? size(40) : (int32_t)times(a.G, size(20));
      a.L = size(600), a.N = size(40), a.num_slots = rare() ? size(9) : 8, a.flags = (uint32_t)pick({0, 2, 2, 2, 1});
      a.x_channel = a.dt_channel = a.z_channel = a.out_channel = stride(a.L);
      a.x_batch = a.dt_batch = a.z_batch = a.out_batch = stride(times(a.D, a.L));
      a.b_state = a.c_state = stride(a.L), a.b_group = a.c_group = stride(times(a.N, a.L));
      a.b_batch = a.c_batch = stride(times(a.G, a.N, a.L));
      a.initial_stride = stride(times(a.D, a.N)), a.final_stride = stride(times(a.D, a.N));
      (void)sparseconv_selective_scan_workspace(&a, &bytes);
      const sc_status s = sparseconv_selective_scan(&a, nullptr);
      check(s == SC_OK ? message.empty() : !message.empty(), "scan message");
    }
    {
      sc_adapter a{at<const void*>(0), at<const void*>(1), at<void*>(2), at<const void*>(3), at<const void*>(4),
                   at<const float*>(5), at<const int32_t*>(6), at<void*>(7), (int64_t)pick({1 << 20, 1 << 28, 0})};
      a.dtype = (int32_t)pick({0, 1, 2, 0, 1, 2, 9}), a.B = size(5), a.C = size(80), a.M = size(80), a.L = size(200), a.R = size(64);
      a.adapters = size(4), a.reserved = rare();
      a.x_channel = a.base_channel = a.out_channel = stride(a.L), a.x_batch = stride(times(a.C, a.L));
      a.base_batch = a.out_batch = stride(times(a.M, a.L));
      (void)sparseconv_adapter_workspace(&a, &bytes);
      const sc_status s = sparseconv_adapter_apply(&a, nullptr);
      check(s == SC_OK ? message.empty() : !message.empty(), "adapter message");
    }
  }
  std::printf("launched %d, failed checks %d\n", launched, failed);
  return failed != 0 || launched < rounds / 4;
}
