// Prints the plans that the sequence operators' launches take (sequence_plan.h) on a device of 256 CUs: one line a
// call on standard input, "conv dtype B D L", "scan B D L N G" or "adapter dtype B C M L R".
#include <cstdio>
#include <iostream>
#include <string>

#include "sequence_plan.h"

int main() {
  std::string op;
  while (std::cin >> op) {
    if (op == "conv") {
      sc_causal_conv a{};
      std::cin >> a.dtype >> a.B >> a.D >> a.L;
      std::printf("places=%lld own=%d fits=%d\n", (long long)sc::conv_places(a), sc::conv_own_rows(a), sc::conv_fits(a));
    } else if (op == "scan") {
      sc_selective_scan a{};
      std::cin >> a.B >> a.D >> a.L >> a.N >> a.G;
      const sc::ScanPlan p = sc::scan_plan(a, 256);
      std::printf("ti=%d chunks=%d segments=%d groups=%lld ahead=%d fits=%d\n", p.ti, p.chunks, p.segments, (long long)p.groups, p.ahead,
                  sc::scan_fits(a));
    } else {
      sc_adapter a{};
      std::cin >> a.dtype >> a.B >> a.C >> a.M >> a.L >> a.R;
      const sc::AdapterPlan p = sc::adapter_plan(a, 256);
      std::printf("token=%d ltiles=%d segments=%d rpieces=%d mtiles=%d mrows=%d wide=%d down=%lld up=%lld fits=%d\n", p.token, p.ltiles,
                  p.segments, p.rpieces, p.mtiles, p.mrows, p.wide, (long long)p.down_blocks, (long long)p.up_blocks, sc::adapter_fits(a));
    }
  }
}
