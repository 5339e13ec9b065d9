// Attention operators (paged_attention.hip, cache.hip, residual_norm.hip): what their kernels and
// the entry points in attention.cpp share.
#pragma once
#include "sequence.h"

namespace sc {

// Launchers.  The arguments have been checked; return a hipError_t value as int.
int launch_paged_attention(const sc_paged_attention& a, int cus, void* stream);
int launch_cache_append(const sc_cache_append& a, int cus, void* stream);
int launch_cache_copy(const sc_cache_copy& a, void* stream);
int launch_residual_norm(const sc_residual_norm& a, int cus, void* stream);

}  // namespace sc
