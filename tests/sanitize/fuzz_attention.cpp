// Drives the attention operators' entry points (attention.cpp) with seeded random argument structures, most of them wrong
// somewhere, with the launchers replaced: a call that passes the checks must fit a launch (the plans are made as the
// launchers make them) and its outputs' exact bytes must not meet an input's, and no check may overflow, read memory
// or throw.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <string>
#include <vector>

#include "attention.h"
#include "attention_plan.h"

namespace {
std::mt19937_64 rng;
int failed = 0, launched = 0;
std::string message;

int64_t pick(std::initializer_list<int64_t> v) { return *(v.begin() + rng() % v.size()); }
bool rare() { return rng() % 32 == 0; }

void check(bool ok, const char* what) {
  if (!ok) {
    failed++;
    std::printf("failed: %s\n", what);
  }
}

// The runs of bytes of a strided tensor, as long as there are few.
struct Run {
  __int128 lo, hi;
};
typedef std::vector<Run> Runs;
Runs runs(const void* p, int64_t outer, int64_t rows, int64_t len, int64_t os, int64_t rs, int64_t es) {
  Runs r;
  if (!p || len <= 0) return r;
  for (int64_t o = 0; o < outer && r.size() < 4000; o++)
    for (int64_t i = 0; i < rows && r.size() < 4000; i++) {
      const __int128 at = (__int128)(uintptr_t)p + (__int128)es * ((__int128)o * os + (__int128)i * rs);
      r.push_back({at, at + (__int128)es * len});
    }
  return r;
}
// (a tensor's own runs may overlap where it is read; sorted by their beginning, the farthest end so far decides)
void apart(Runs a, Runs b, const char* what) {
  auto less = [](const Run& x, const Run& y) { return x.lo < y.lo; };
  std::sort(a.begin(), a.end(), less);
  std::sort(b.begin(), b.end(), less);
  __int128 a_end = INT64_MIN, b_end = INT64_MIN;
  for (size_t i = 0, j = 0; i < a.size() || j < b.size();) {
    if (j == b.size() || (i < a.size() && a[i].lo <= b[j].lo)) {
      if (a[i].lo < b_end) return check(false, what);
      a_end = std::max(a_end, a[i++].hi);
    } else {
      if (b[j].lo < a_end) return check(false, what);
      b_end = std::max(b_end, b[j++].hi);
    }
  }
}
void alone(Runs a, const char* what) {
  std::sort(a.begin(), a.end(), [](const Run& x, const Run& y) { return x.lo < y.lo; });
  for (size_t i = 1; i < a.size(); i++)
    if (a[i].lo < a[i - 1].hi) return check(false, what);
}
}  // namespace

namespace sc {
int report(int status, const std::string& msg) {
  message = msg;
  return status;
}
int launch_paged_attention(const sc_paged_attention& a, int cus, void*) {
  launched++;
  const AttendPlan p = attend_plan(a, cus);
  check(p.splits >= 1 && p.splits <= 32 && p.tiles >= 1 && p.nt >= 1, "attend plan");
  check((int64_t)a.B * a.G * p.groups() * 256 < kGridThreads && attend_rows(a, p) < (1LL << 40), "attend grid");
  check(attend_rows(a, p) >= (int64_t)a.B * a.H * a.L, "attend rows");
  const int64_t need = attend_workspace(a, cus), es = a.dtype == SC_F32 ? 4 : 2, os = a.flags ? 4 : es;
  check(!need || (a.workspace && a.workspace_bytes >= need && !((uintptr_t)a.workspace & 15)), "attend workspace");
  if ((int64_t)a.B * a.H * a.D > 2000) return 0;
  const Runs out = runs(a.out, a.B, (int64_t)a.H * a.D, a.L, a.out_batch, a.out_channel, os);
  alone(out, "attend out itself");
  apart(out, runs(a.q, a.B, (int64_t)a.H * a.D, a.L, a.q_batch, a.q_channel, es), "attend out and q");
  const int64_t per = (int64_t)a.G * a.P * a.D;
  apart(out, runs(a.k_pages, a.pages, 1, per, a.k_page, 0, es), "attend out and keys");
  apart(out, runs(a.v_pages, a.pages, 1, per, a.v_page, 0, es), "attend out and values");
  apart(out, runs(a.table, a.B, 1, a.width, a.table_batch, 0, 4), "attend out and table");
  return 0;
}
int launch_cache_append(const sc_cache_append& a, int cus, void*) {
  launched++;
  const AppendPlan p = append_plan(a, cus);
  check(p.groups >= 1 && p.groups * 256 < kGridThreads, "append grid");
  check(p.few || (p.chunk >= 1 && (int64_t)p.turners * p.chunk >= (a.q ? a.H : 0) + a.G && (int64_t)p.sharers * p.chunk >= a.G), "append plan");
  const int64_t es = a.dtype == SC_F32 ? 4 : 2, cs = a.cache_dtype == SC_F32 ? 4 : 2, per = (int64_t)a.G * a.P * a.D;
  if ((int64_t)a.B * a.H * a.D > 2000) return 0;
  const Runs kp = runs(a.k_pages, a.pages, 1, per, a.k_page, 0, cs), vp = runs(a.v_pages, a.pages, 1, per, a.v_page, 0, cs);
  apart(kp, vp, "append keys and values");
  alone(kp, "append keys themselves");
  for (const Runs& in : {runs(a.k, a.B, (int64_t)a.G * a.D, a.L, a.k_batch, a.k_channel, es),
                         runs(a.v, a.B, (int64_t)a.G * a.D, a.L, a.v_batch, a.v_channel, es),
                         runs(a.table, a.B, 1, a.width, a.table_batch, 0, 4), runs(a.past, 1, 1, a.B, 0, 0, 4)}) {
    apart(in, kp, "append input and keys");
    apart(in, vp, "append input and values");
    if (a.q) apart(in, runs(a.q_out, a.B, (int64_t)a.H * a.D, a.L, a.q_out_batch, a.q_out_channel, cs), "append input and q_out");
  }
  if (a.q) {
    const Runs out = runs(a.q_out, a.B, (int64_t)a.H * a.D, a.L, a.q_out_batch, a.q_out_channel, cs);
    alone(out, "append q_out itself");
    if (a.q != a.q_out) apart(out, runs(a.q, a.B, (int64_t)a.H * a.D, a.L, a.q_batch, a.q_channel, es), "append q_out and q");
    else check(es == cs && a.q_batch == a.q_out_batch && a.q_channel == a.q_out_channel, "append in place");
  }
  return 0;
}
int launch_cache_copy(const sc_cache_copy& a, void*) {
  launched++;
  check((int64_t)a.outer * a.count * ceil_div(a.page_bytes, kCopyBytes) * 256 < kGridThreads, "copy grid");
  if ((int64_t)a.outer * a.pages < 300) alone(runs(a.pool, a.outer, a.pages, a.page_bytes, a.outer_stride, a.page_stride, 1), "pool itself");
  return 0;
}
int launch_residual_norm(const sc_residual_norm& a, int cus, void*) {
  launched++;
  const NormPlan p = norm_plan(a, cus);
  check((int64_t)a.B * p.tiles * 1024 < kGridThreads && p.tiles >= 1, "norm grid");
  if (p.form == kNormPrompt) {
    const int V = a.dtype == SC_F32 ? 4 : 8;
    check((int64_t)p.pass * (p.threads >> p.lp_shift) >= a.C && (int64_t)p.tiles * (V << p.lp_shift) >= a.L, "norm plan");
  }
  if (p.form == kNormToken) check(p.threads * 8 >= a.C && a.L == 1, "norm plan");
  const int64_t es = a.dtype == SC_F32 ? 4 : 2;
  if ((int64_t)a.B * a.C > 2000) return 0;
  const Runs x = runs(a.x, a.B, a.C, a.L, a.x_batch, a.x_channel, es), y = runs(a.y, a.B, a.C, a.L, a.y_batch, a.y_channel, es);
  const Runs g = runs(a.gate, a.B, a.C, a.gate_position ? a.L : 1, a.gate_batch, a.gate_channel, es);
  const Runs s = runs(a.sum, a.B, a.C, a.L, a.sum_batch, a.sum_channel, es), o = runs(a.out, a.B, a.C, a.L, a.out_batch, a.out_channel, es);
  alone(s, "sum itself");
  alone(o, "norm out itself");
  apart(s, o, "sum and out");
  apart(s, y, "sum and y");
  apart(o, x, "norm out and x");
  apart(s, g, "sum and gate");
  apart(o, g, "norm out and gate");
  if (a.sum != a.x) apart(s, x, "sum and x");
  if (a.out != a.y) apart(o, y, "norm out and y");
  return 0;
}
}  // namespace sc

namespace {
template <class P>
P at(int i) {
  uintptr_t p = (uintptr_t)(i + 1) << 30;
  if (rare()) p = (uintptr_t)(rng() % 14 + 1) << 30;
  if (rare()) p += rng() % 4096;
  if (rare()) p = 0;
  return (P)p;
}
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
  rng.seed(11);
  for (int r = 0; r < rounds; r++) {
    {
      sc_paged_attention a{at<const void*>(0), at<void*>(1), at<const void*>(2), at<const void*>(3), at<const int32_t*>(4),
                           at<const int32_t*>(5), rng() % 2 ? at<const int32_t*>(6) : nullptr, rng() % 2 ? at<const int32_t*>(7) : nullptr,
                           rng() % 2 ? at<const float*>(8) : nullptr, at<void*>(9), (int64_t)pick({1 << 30, 1 << 20, 0})};
      a.dtype = (int32_t)pick({0, 1, 2, 0, 1, 2, 3}), a.B = size(5), a.G = size(3), a.H = rare() ? size(9) : (int32_t)times(a.G, size(4));
      a.D = rare() ? size(300) : (int32_t)pick({8, 16, 40}), a.L = rng() % 3 ? size(40) : 1, a.P = rare() ? size(300) : (int32_t)pick({16, 32, 64, 256});
      a.width = size(60), a.pages = size(9), a.window = rare() ? size(9) : 0, a.flags = rng() % 4 == 0, a.reserved = rare();
      a.scale = 0.5f, a.cap = rng() % 2 ? 3.0f : 0.0f;
      a.q_channel = stride(a.L), a.q_batch = stride(times(times(a.H, a.D), a.L, pick({1, 2})));
      a.out_channel = stride(a.L), a.out_batch = stride(times(a.H, a.D, a.L));
      const int64_t per = times(a.G, times(a.P, a.D));
      a.k_page = stride(per), a.v_page = stride(per), a.table_batch = stride(a.width);
      int64_t bytes;
      (void)sparseconv_paged_attention_workspace(&a, &bytes);
      const sc_status s = sparseconv_paged_attention(&a, nullptr);
      check(s == SC_OK ? message.empty() : !message.empty(), "attend message");
    }
    {
      sc_cache_append a{rng() % 4 ? at<const void*>(0) : nullptr, at<void*>(1), at<const void*>(2), at<const void*>(3), at<void*>(4), at<void*>(5),
                        at<const double*>(6), rng() % 2 ? at<const int32_t*>(7) : nullptr, rng() % 2 ? at<const int32_t*>(8) : nullptr,
                        at<const int32_t*>(9), at<const int32_t*>(10), rng() % 2 ? at<const int32_t*>(11) : nullptr};
      a.dtype = (int32_t)pick({0, 1, 2, 0, 0, 3}), a.cache_dtype = rng() % 4 ? a.dtype : (int32_t)pick({0, 1, 2});
      if (rng() % 8 == 0) a.q_out = const_cast<void*>(a.q);
      a.B = size(5), a.G = size(3), a.H = size(8), a.D = rare() ? size(300) : (int32_t)pick({8, 16, 40}), a.L = size(40);
      a.P = (int32_t)pick({16, 64, 256}), a.width = size(9), a.pages = size(9), a.pairs = rare() ? size(40) : a.D / 2, a.num_axes = size(3);
      a.flags = rng() % 2, a.reserved = rare();
      a.q_channel = stride(a.L), a.q_batch = stride(times(times(a.H, a.D), a.L)), a.q_out_channel = stride(a.L);
      a.q_out_batch = stride(times(a.H, a.D, a.L)), a.k_channel = a.v_channel = stride(a.L);
      a.k_batch = a.v_batch = stride(times(times(a.G, a.D), a.L));
      const int64_t per = times(a.G, times(a.P, a.D));
      a.k_page = stride(per), a.v_page = stride(per), a.table_batch = stride(a.width);
      if (rng() % 8 == 0 && per > 0 && per < (1 << 24)) a.v_pages = static_cast<char*>(a.k_pages) + per * (a.cache_dtype ? 2 : 4), a.k_page = a.v_page = 2 * per;
      a.positions_axis = stride(a.L), a.positions_batch = stride(times(a.num_axes, a.L));
      const sc_status s = sparseconv_cache_append(&a, nullptr);
      check(s == SC_OK ? message.empty() : !message.empty(), "append message");
    }
    {
      sc_cache_copy a{at<void*>(0), at<const int32_t*>(1), at<const int32_t*>(2)};
      a.page_bytes = rare() ? stride(1 << 20) : (int64_t)(rng() % 5000), a.outer = size(9), a.pages = size(30), a.count = size(40), a.reserved = rare();
      a.page_stride = stride(a.page_bytes), a.outer_stride = stride(times(a.pages, a.page_bytes));
      const sc_status s = sparseconv_cache_copy(&a, nullptr);
      check(s == SC_OK ? message.empty() : !message.empty(), "copy message");
    }
    {
      sc_residual_norm a{at<const void*>(0), at<const void*>(1), rng() % 2 ? at<const void*>(2) : nullptr, at<void*>(3), at<void*>(4),
                         at<const float*>(5), at<const float*>(6), rng() % 2 ? at<const float*>(7) : nullptr, nullptr};
      if (rng() % 6 == 0) a.sum = const_cast<void*>(a.x);
      if (rng() % 6 == 0) a.out = const_cast<void*>(a.y);
      a.dtype = (int32_t)pick({0, 1, 2, 0, 1, 2, 3}), a.B = size(6), a.C = rare() ? size(20000) : size(60), a.L = rng() % 3 ? size(60) : 1;
      a.flags = rng() % 2, a.reserved = rare(), a.scale = 1.0f, a.eps = 1e-6f, a.gate_position = (int64_t)pick({0, 1, 1, rare() ? 2 : 0});
      a.x_channel = stride(a.L), a.x_batch = stride(times(a.C, a.L, pick({1, 2}))), a.y_channel = stride(a.L), a.y_batch = stride(times(a.C, a.L));
      a.sum_channel = a.sum == a.x ? a.x_channel : stride(a.L), a.sum_batch = a.sum == a.x ? a.x_batch : stride(times(a.C, a.L));
      a.out_channel = stride(a.L), a.out_batch = stride(times(a.C, a.L)), a.gate_channel = stride(a.gate_position ? a.L : 1);
      a.gate_batch = stride(times(a.C, a.gate_position ? a.L : 1));
      const sc_status s = sparseconv_residual_norm(&a, nullptr);
      check(s == SC_OK ? message.empty() : !message.empty(), "norm message");
    }
  }
  std::printf("launched %d, failed checks %d\n", launched, failed);
  return failed != 0 || launched < rounds / 4;
}
