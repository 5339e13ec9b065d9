// Drives the sequence operators' entry points (sequence.cpp, its launchers replaced) with seeded random arguments whose
// tensors lie in one small arena, so that they often meet.  The launchers lay every tensor's runs of bytes out and
// see that nothing a call writes shares a byte with itself, with anything it reads or with anything else it
// writes, but for the in-place forms that the header names; and that every plan fits its launch.
#include <algorithm>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>
#include <string>
#include <utility>
#include <vector>

#include "sequence.h"
#include "sequence_plan.h"

namespace {
std::mt19937_64 rng;
int failed = 0, launched[3] = {};
std::string message;

void check(bool ok, const char* what) {
  if (!ok) {
    failed++;
    std::printf("failed: %s\n", what);
  }
}

// The runs of a strided tensor: [first byte, past the last), sorted.
struct Runs {
  std::vector<std::pair<uint64_t, uint64_t>> v;
  Runs(const void* p, int64_t es, int64_t len, std::initializer_list<std::pair<int64_t, int64_t>> dims = {}) {
    if (!p || len <= 0) return;
    std::vector<int64_t> at{0};
    for (auto [n, stride] : dims) {
      std::vector<int64_t> next;
      for (int64_t a : at)
        for (int64_t i = 0; i < n; i++) next.push_back(a + i * stride);
      at.swap(next);
    }
    for (int64_t a : at) v.push_back({(uintptr_t)p + a * es, (uintptr_t)p + (a + len) * es});
    std::sort(v.begin(), v.end());
  }
  bool meets_itself() const {
    for (size_t i = 1; i < v.size(); i++)
      if (v[i].first < v[i - 1].second) return true;
    return false;
  }
};

bool meet(const Runs& a, const Runs& b) {
  size_t i = 0, j = 0;
  uint64_t far_a = 0, far_b = 0;  // inputs may repeat their own bytes: the furthest end so far counts
  while (i < a.v.size() || j < b.v.size()) {
    if (j == b.v.size() || (i < a.v.size() && a.v[i].first <= b.v[j].first)) {
      if (a.v[i].first < far_b) return true;
      far_a = std::max(far_a, a.v[i++].second);
    } else {
      if (b.v[j].first < far_a) return true;
      far_b = std::max(far_b, b.v[j++].second);
    }
  }
  return false;
}

struct Named {
  const char* name;
  Runs runs;
};

void check_call(const char* op, const std::vector<Named>& written, const std::vector<Named>& read) {
  for (size_t i = 0; i < written.size(); i++) {
    const std::string w = std::string(op) + ": " + written[i].name;
    check(!written[i].runs.meets_itself(), (w + " meets itself").c_str());
    for (size_t j = 0; j < i; j++) check(!meet(written[i].runs, written[j].runs), (w + " meets " + written[j].name).c_str());
    for (const Named& r : read) check(!meet(written[i].runs, r.runs), (w + " meets " + r.name).c_str());
  }
}
}  // namespace

namespace sc {
int report(int status, const std::string& msg) {
  message = msg;
  return status;
}

int launch_causal_conv(const sc_causal_conv& a, void*) {
  launched[0]++;
  const int64_t es = a.dtype == SC_F32 ? 4 : 2, per = (int64_t)a.D * (a.K - 1);
  const bool in_place = a.initial_state == a.final_state && a.initial_stride == a.final_stride;
  check_call("conv", {{"out", {a.out, es, a.L, {{a.B, a.out_batch}, {a.D, a.out_channel}}}},
                      {"final", {a.final_state, es, per, {{a.num_slots, a.final_stride}}}}},
             {{"x", {a.x, es, a.L, {{a.B, a.x_batch}, {a.D, a.x_channel}}}},
              {"initial", {in_place ? nullptr : a.initial_state, es, per, {{a.num_slots, a.initial_stride}}}},
              {"weight", {a.weight, 4, (int64_t)a.D * a.K}},
              {"bias", {a.bias, 4, a.D}},
              {"lengths", {a.lengths, 4, a.B}},
              {"slots", {a.slots, 4, a.B}}});
  check(conv_fits(a), "conv fits");
  return 0;
}

int launch_selective_scan(const sc_selective_scan& a, int cus, void*) {
  launched[1]++;
  const int64_t es = a.dtype == SC_F32 ? 4 : 2, per = (int64_t)a.D * a.N;
  const bool in_place = a.initial_state == a.final_state && a.initial_stride == a.final_stride;
  const int64_t need = a.L ? scan_workspace(a, cus) : 0;
  check(!need || a.workspace_bytes >= need, "scan workspace");
  check_call("scan", {{"out", {a.out, es, a.L, {{a.B, a.out_batch}, {a.D, a.out_channel}}}},
                      {"final", {a.final_state, 4, per, {{a.num_slots, a.final_stride}}}},
                      {"workspace", {a.workspace, 1, need}}},
             {{"x", {a.x, es, a.L, {{a.B, a.x_batch}, {a.D, a.x_channel}}}},
              {"dt", {a.dt, es, a.L, {{a.B, a.dt_batch}, {a.D, a.dt_channel}}}},
              {"z", {a.z, es, a.L, {{a.B, a.z_batch}, {a.D, a.z_channel}}}},
              {"b", {a.b, es, a.L, {{a.B, a.b_batch}, {a.G, a.b_group}, {a.N, a.b_state}}}},
              {"c", {a.c, es, a.L, {{a.B, a.c_batch}, {a.G, a.c_group}, {a.N, a.c_state}}}},
              {"initial", {in_place ? nullptr : a.initial_state, 4, per, {{a.num_slots, a.initial_stride}}}},
              {"A", {a.A, 4, per}},
              {"skip", {a.skip, 4, a.D}},
              {"dt_bias", {a.dt_bias, 4, a.D}},
              {"lengths", {a.lengths, 4, a.B}},
              {"slots", {a.slots, 4, a.B}}});
  check(scan_fits(a), "scan fits");
  return 0;
}

int launch_adapter(const sc_adapter& a, int cus, void*) {
  launched[2]++;
  const int64_t es = a.dtype == SC_F32 ? 4 : 2;
  const bool in_place = a.base == a.out && a.base_batch == a.out_batch && a.base_channel == a.out_channel;
  const int64_t need = adapter_workspace(a, cus);
  check(!need || a.workspace_bytes >= need, "adapter workspace");
  check_call("adapter", {{"out", {a.out, es, a.L, {{a.B, a.out_batch}, {a.M, a.out_channel}}}}, {"workspace", {a.workspace, 1, need}}},
             {{"x", {a.x, es, a.L, {{a.B, a.x_batch}, {a.C, a.x_channel}}}},
              {"base", {in_place ? nullptr : a.base, es, a.L, {{a.B, a.base_batch}, {a.M, a.base_channel}}}},
              {"down", {a.down, es, (int64_t)a.adapters * a.R * a.C}},
              {"up", {a.up, es, (int64_t)a.adapters * a.M * a.R}},
              {"scale", {a.scale, 4, a.adapters}},
              {"index", {a.index, 4, a.B}}});
  check(adapter_fits(a), "adapter fits");
  return 0;
}

// (the launchers' own sizes)
int64_t scan_workspace(const sc_selective_scan& a, int cus) {
  if (a.L <= 1) return 0;
  const ScanPlan p = scan_plan(a, cus);
  return p.segments == 1 ? 0 : (int64_t)a.B * p.segments * a.D * (a.N + 1) * 4;
}
int64_t adapter_workspace(const sc_adapter& a, int cus) {
  const AdapterPlan p = adapter_plan(a, cus);
  return p.token ? 0 : (int64_t)p.segments * a.B * a.R * a.L * 4;
}
}  // namespace sc

namespace {
constexpr uintptr_t kArena = 1 << 30;
int64_t below(int64_t n) { return (int64_t)(rng() % (uint64_t)n); }
bool often() { return rng() % 8 != 0; }

// Somewhere in the arena (`room` bytes), at a multiple of `to`; or, as often, well away from it.
template <class P>
P at(int64_t room, int64_t to, int i) {
  if (rng() % 3) return (P)(kArena + ((uintptr_t)(i + 1) << 34));
  return (P)(kArena + (uintptr_t)(below(room / to) * to));
}
int64_t stride(int64_t usual) { return often() ? usual : below(2 * usual + 2); }

// x and out as parts of one tensor, now and then.
void share(const void** x, void* out, int64_t* x_batch, int64_t* x_channel, int64_t* out_batch, int64_t* out_channel, int64_t D, int64_t L,
           int64_t es) {
  if (rng() % 3) return;
  *x_channel = *out_channel = L, *x_batch = *out_batch = 2 * D * L;
  *x = (const void*)((uintptr_t)out + (uintptr_t)(es * (rng() % 2 ? D * L : below(2 * D * L + 1))));
  if (rng() % 4 == 0) *x_channel = *out_channel = 2 * L, *x = (const void*)((uintptr_t)out + (uintptr_t)(es * (rng() % 2 ? L : below(2 * L + 1))));
}
}  // namespace

// Calls that no check may let pass, given to the replaced launchers: each has to be noticed.
int unnoticed() {
  int missed = 0;
  auto noticed = [&](const char* what, auto launch) {
    const int before = failed;
    launch();
    if (failed == before) missed++, std::printf("unnoticed: %s\n", what);
    failed = before;
  };
  char* const m = (char*)kArena;
  auto conv = [&](auto change) {
    sc_causal_conv a{m, m + 4096, (float*)(m + 8192), (float*)(m + 12288), m + 16384, m + 20480, nullptr, nullptr, 80, 10, 80, 10, 24, 24, 0, 2, 8, 10, 4, 2, 1, 0};
    change(a);
    sc::launch_causal_conv(a, nullptr);
  };
  noticed("conv out on x's last byte", [&] { conv([&](sc_causal_conv& a) { a.x = m + 4096 - 640 + 4; }); });
  noticed("conv out meets itself", [&] { conv([&](sc_causal_conv& a) { a.out_channel = 9; }); });
  noticed("conv final on initial", [&] { conv([&](sc_causal_conv& a) { a.final_state = m + 16384 + 4; }); });
  noticed("conv final on out", [&] { conv([&](sc_causal_conv& a) { a.final_state = m + 4096 + 636; }); });
  noticed("conv out on weight", [&] { conv([&](sc_causal_conv& a) { a.weight = (float*)(m + 4096 - 124); }); });
  auto scan = [&](auto change) {
    sc_selective_scan a{};
    a.x = m, a.dt = m + 4096, a.b = m + 8192, a.c = m + 12288, a.out = m + 16384, a.A = (float*)(m + 20480), a.B = 2, a.D = 4, a.L = 8, a.N = 2, a.G = 1;
    a.x_batch = a.dt_batch = a.out_batch = 32, a.x_channel = a.dt_channel = a.out_channel = 8;
    a.b_batch = a.c_batch = 16, a.b_group = a.c_group = 16, a.b_state = a.c_state = 8, a.num_slots = 2, a.initial_stride = a.final_stride = 8;
    change(a);
    sc::launch_selective_scan(a, 256, nullptr);
  };
  noticed("scan out on c's last state", [&] { scan([&](sc_selective_scan& a) { a.c = m + 16384 - 124; }); });
  noticed("scan final on A", [&] { scan([&](sc_selective_scan& a) { a.final_state = (float*)(m + 20480 + 28); }); });
  noticed("scan workspace missing", [&] { scan([&](sc_selective_scan& a) { a.L = 4096; }); });
  auto adapter = [&](auto change) {
    sc_adapter a{m, m + 4096, m + 8192, m + 12288, m + 16384, nullptr, (int32_t*)(m + 20480), m + 24576, 1 << 16, 40, 8, 40, 8, 40, 8, 0, 2, 5, 5, 8, 2, 1, 0};
    change(a);
    sc::launch_adapter(a, 256, nullptr);
  };
  noticed("adapter workspace on out", [&] { adapter([&](sc_adapter& a) { a.workspace = m + 8192 + 304; }); });
  noticed("adapter out on base, other strides", [&] { adapter([&](sc_adapter& a) { a.base = a.out, a.base_channel = 4; }); });
  noticed("adapter out on index", [&] { adapter([&](sc_adapter& a) { a.index = (int32_t*)(m + 8192); }); });
  const int before = failed;
  conv([](sc_causal_conv& a) { a.final_state = (void*)a.initial_state; });
  scan([](sc_selective_scan&) {});
  adapter([](sc_adapter& a) { a.base = a.out; });
  if (failed != before) missed++, std::printf("a good call was taken for a bad one\n");
  return missed;
}

int main(int argc, char** argv) {
  const int rounds = argc > 1 ? std::atoi(argv[1]) : 20000;
  rng.seed(11);
  if (unnoticed()) return 1;
  for (int r = 0; r < rounds; r++) {
    {
      sc_causal_conv a{};
      a.dtype = (int32_t)below(3), a.B = 1 + (int32_t)below(4), a.D = 1 + (int32_t)below(6), a.L = (int32_t)below(12), a.K = 1 + (int32_t)below(4);
      a.num_slots = a.B + (int32_t)below(3);
      const int64_t es = a.dtype == SC_F32 ? 4 : 2, room = 4096, per = (int64_t)a.D * (a.K - 1);
      a.x = at<const void*>(room, es, 0), a.out = at<void*>(room, es, 1), a.weight = at<const float*>(room, 4, 2);
      a.bias = at<const float*>(room, 4, 3), a.lengths = at<const int32_t*>(room, 4, 4), a.slots = at<const int32_t*>(room, 4, 5);
      a.initial_state = at<const void*>(room, es, 6), a.final_state = rng() % 2 ? (void*)a.initial_state : at<void*>(room, es, 7);
      a.x_channel = stride(a.L), a.x_batch = stride(a.D * a.L), a.out_channel = stride(a.L), a.out_batch = stride(a.D * a.L);
      a.initial_stride = stride(per), a.final_stride = rng() % 2 ? a.initial_stride : stride(per);
      share(&a.x, a.out, &a.x_batch, &a.x_channel, &a.out_batch, &a.out_channel, a.D, a.L, es);
      (void)sparseconv_causal_conv(&a, nullptr);
    }
    {
      sc_selective_scan a{};
      a.dtype = (int32_t)below(3), a.B = 1 + (int32_t)below(3), a.G = 1 + (int32_t)below(2), a.D = a.G * (1 + (int32_t)below(3));
      a.L = rng() % 8 ? (int32_t)below(12) : 1000, a.N = 1 + (int32_t)below(4), a.num_slots = a.B + (int32_t)below(3);
      const int64_t es = a.dtype == SC_F32 ? 4 : 2, room = a.L > 12 ? 1 << 18 : 4096, per = (int64_t)a.D * a.N;
      a.x = at<const void*>(room, es, 0), a.dt = at<const void*>(room, es, 1), a.z = at<const void*>(room, es, 2);
      a.b = at<const void*>(room, es, 3), a.c = at<const void*>(room, es, 4), a.out = at<void*>(room, es, 5);
      a.A = at<const float*>(room, 4, 6), a.skip = at<const float*>(room, 4, 7), a.dt_bias = at<const float*>(room, 4, 8);
      a.initial_state = at<const float*>(room, 4, 9), a.final_state = rng() % 2 ? (float*)a.initial_state : at<float*>(room, 4, 10);
      a.lengths = at<const int32_t*>(room, 4, 11), a.slots = at<const int32_t*>(room, 4, 12);
      a.workspace = at<void*>(room, 16, 13), a.workspace_bytes = 1 << 16;
      a.x_channel = stride(a.L), a.dt_channel = stride(a.L), a.z_channel = stride(a.L), a.out_channel = stride(a.L);
      a.x_batch = stride(a.D * a.L), a.dt_batch = stride(a.D * a.L), a.z_batch = stride(a.D * a.L), a.out_batch = stride(a.D * a.L);
      a.b_state = stride(a.L), a.b_group = stride(a.N * a.L), a.b_batch = stride(a.G * a.N * a.L);
      a.c_state = stride(a.L), a.c_group = stride(a.N * a.L), a.c_batch = stride(a.G * a.N * a.L);
      a.initial_stride = stride(per), a.final_stride = rng() % 2 ? a.initial_stride : stride(per);
      const void** in = rng() % 2 ? &a.x : &a.z;
      share(in, a.out, in == &a.x ? &a.x_batch : &a.z_batch, in == &a.x ? &a.x_channel : &a.z_channel, &a.out_batch, &a.out_channel, a.D, a.L, es);
      (void)sparseconv_selective_scan(&a, nullptr);
    }
    {
      sc_adapter a{};
      a.dtype = (int32_t)below(3), a.B = 1 + (int32_t)below(4), a.C = 1 + (int32_t)below(5), a.M = rng() % 2 ? a.C : 1 + (int32_t)below(5);
      a.L = 1 + (int32_t)below(20), a.R = 1 + (int32_t)below(3), a.adapters = 1 + (int32_t)below(3);
      const int64_t es = a.dtype == SC_F32 ? 4 : 2, room = 4096;
      a.x = at<const void*>(room, es, 0), a.out = at<void*>(room, es, 1), a.base = rng() % 2 ? a.out : at<const void*>(room, es, 2);
      a.down = at<const void*>(room, 16, 3), a.up = at<const void*>(room, 16, 4), a.scale = at<const float*>(room, 4, 5);
      a.index = at<const int32_t*>(room, 4, 6), a.workspace = at<void*>(room, 16, 7), a.workspace_bytes = 1 << 16;
      a.x_channel = stride(a.L), a.x_batch = stride(a.C * a.L), a.out_channel = stride(a.L), a.out_batch = stride(a.M * a.L);
      a.base_channel = rng() % 2 ? a.out_channel : stride(a.L), a.base_batch = rng() % 2 ? a.out_batch : stride(a.M * a.L);
      const void** in = rng() % 2 ? &a.x : &a.base;
      share(in, a.out, in == &a.x ? &a.x_batch : &a.base_batch, in == &a.x ? &a.x_channel : &a.base_channel, &a.out_batch, &a.out_channel,
            in == &a.x ? a.C : a.M, a.L, es);
      (void)sparseconv_adapter_apply(&a, nullptr);
    }
  }
  std::printf("launched %d %d %d, failed checks %d\n", launched[0], launched[1], launched[2], failed);
  return failed != 0 || launched[0] < rounds / 8 || launched[1] < rounds / 40 || launched[2] < rounds / 8;
}
