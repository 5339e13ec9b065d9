// The attention operators' launches at the ends of the sizes that they accept (attention_plan.h, for 256 CUs): seeded random sizes over
// the whole of their types, as the entry points' checks leave them.  What fits must be a launch's worth of threads in every kernel that the
// plan asks for, no sum may pass its type (the sanitizer), and "fits" must be what the header says, worked out in 128 bits.
#include <cmath>
#include <cstdint>
#include <cstdio>
#include <cstdlib>
#include <random>

#include "attention_plan.h"

namespace {
std::mt19937_64 rng(5);
int failed = 0, fit = 0;
typedef __int128 Wide;

int32_t upto(int64_t most) {  // 1 .. most, spread over the logarithm
  const double v = std::exp2(std::uniform_real_distribution<double>(0, std::log2((double)most + 1))(rng));
  return (int32_t)(v < 1 ? 1 : v > most ? most : v);
}
void check(bool ok, const char* what, long long a = 0, long long b = 0, long long c = 0, long long d = 0, long long e = 0) {
  if (ok) return;
  if (failed++ < 10) std::printf("failed: %s %lld %lld %lld %lld %lld\n", what, a, b, c, d, e);
}
Wide up(Wide a, Wide b) { return (a + b - 1) / b; }
}  // namespace

int main(int argc, char** argv) {
  const int rounds = argc > 1 ? std::atoi(argv[1]) : 100000;
  for (int r = 0; r < rounds; r++) {
    {
      sc_paged_attention a{};
      a.dtype = rng() % 3, a.G = upto(1 << 16), a.H = a.G * upto((1 << 16) / a.G), a.B = upto(INT32_MAX);
      a.D = 8 * (1 + rng() % 32), a.L = rng() % 3 ? upto(200) : upto((1 << 30) - 1), a.P = 16 << rng() % 5;
      if (rng() % 2) a.B = upto(4 * sc::kMostGroups / a.G + 1);  // near the limit
      a.width = upto((1 << 30) / a.P), a.pages = 1;
      const Wide share = a.H / a.G;
      auto groups = [&](Wide to) { return Wide(a.B) * a.G * up(share * up(a.L, to) * to, 16); };
      bool says = groups(a.L < 128 ? 1 : 128) < sc::kMostGroups;
      // heads that are cut apart at sixteens: fp32 of more than 128 dims with few rows
      if (a.dtype == SC_F32 && a.D > 128 && share * a.L < 96 && a.L >= 16) says = says && groups(16) < sc::kMostGroups;
      const bool fits = sc::attend_fits(a);
      check(fits == says, "attend fits", a.B, a.H, a.G, a.D, a.L);
      if (fits) {
        fit++;
        const sc::AttendPlan p = sc::attend_plan(a, 256);
        const Wide all = Wide(a.B) * a.G * p.tiles * p.splits, rows = Wide(a.B) * a.G * p.tiles * p.rows();
        check(all >= 1 && all * 256 < sc::kGridThreads, "attend grid", a.B, a.H, a.G, a.D, a.L);
        check(rows >= Wide(a.B) * a.H * a.L, "attend rows", a.B, a.H, a.G, a.D, a.L);
        check(p.splits == 1 || rows / (p.splits > 8 && rows < 64 * 256 ? 2 : 16) * 256 < sc::kGridThreads, "attend join grid", a.B, a.H, a.G, a.D, a.L);
        check(Wide(p.tiles) * p.rows() < INT32_MAX, "attend row numbers", a.B, a.H, a.G, a.D, a.L);
        check(sc::attend_workspace(a, 256) == (p.splits == 1 ? 0 : (int64_t)(rows * p.splits * (a.D + 2) * 4)), "attend workspace");
      }
    }
    {
      sc_cache_append a{};
      static const int some = 0;
      a.q = rng() % 4 ? &some : nullptr, a.G = upto(1 << 16), a.H = upto(1 << 16), a.D = 8 * (1 + rng() % 32), a.B = upto(INT32_MAX);
      a.L = rng() % 2 ? upto(15) : upto((1 << 30) - 1), a.pairs = rng() % (a.D / 2 + 1);
      const Wide heads = (a.q ? a.H : 0) + 2 * Wide(a.G), B = a.B, L = a.L;
      const bool says = L < 16 ? B * heads * a.D * L < (Wide(1) << 32) : B * (up(L, 64) + 1) * (up(heads, 8) + 1) < sc::kMostGroups;
      const bool fits = sc::append_fits(a);
      check(fits == says, "append fits", a.B, a.H, a.G, a.D, a.L);
      if (fits) {
        fit++;
        const sc::AppendPlan p = sc::append_plan(a, 256);
        check(p.groups >= 1 && Wide(p.groups) * 256 <= sc::kGridThreads, "append grid", a.B, a.H, a.G, a.D, a.L);
      }
    }
    {
      sc_residual_norm a{};
      static char some[4];
      a.dtype = rng() % 3, a.B = upto(INT32_MAX), a.C = upto((1 << 20) - 1), a.L = rng() % 2 ? 1 : upto((1 << 30) - 1);
      if (rng() % 2) a.B = upto(1 << 23);
      a.x_channel = a.y_channel = a.sum_channel = a.out_channel = rng() % 2 ? 1 : a.L, a.x = a.y = some;
      if (sc::norm_fits(a)) {
        fit++;
        const sc::NormPlan p = sc::norm_plan(a, 256);
        check(Wide(a.B) * (p.form == sc::kNormToken ? 1 : p.tiles) * p.threads < sc::kGridThreads, "norm grid", a.B, a.C, a.L, a.dtype);
      }
    }
  }
  std::printf("fit %d, failed checks %d\n", fit, failed);
  return failed != 0 || fit < rounds / 4;
}
