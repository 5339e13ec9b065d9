// Sequence operators (causal_conv.hip, selective_scan.hip, adapter.hip): what their kernels and
// the entry points in sequence.cpp share.
#pragma once
#include <cstdint>
#include <string>

#include "../../include/sparseconv.h"

namespace sc {

// The calling thread's error message (api.cpp); returns status.
int report(int status, const std::string& msg);

// Launchers.  The arguments have been checked; return a hipError_t value as int.
int launch_causal_conv(const sc_causal_conv& a, void* stream);
int launch_selective_scan(const sc_selective_scan& a, int cus, void* stream);
int launch_adapter(const sc_adapter& a, int cus, void* stream);

// Workspace bytes of a launch on a device with that many CUs.
int64_t scan_workspace(const sc_selective_scan& a, int cus);
int64_t adapter_workspace(const sc_adapter& a, int cus);

}  // namespace sc
