// Entry points of the sequence operators (declared in include/sparseconv.h): the argument checks,
// then a launch on the caller's stream.
#include <hip/hip_runtime.h>

#include <algorithm>

#include "checks.h"
#include "sequence_plan.h"

namespace {

// The states' part of the checks: `per` values of `es` bytes a slot.
sc_status check_states(const void* first, int64_t first_stride, const void* last, int64_t last_stride, int64_t per,
                       int64_t es, const int32_t* slots, int num_slots, int B) {
  if (num_slots < 0) return fail(SC_ESHAPE, "num_slots < 0");
  if (misaligned(slots, 4)) return fail(SC_EINVAL, "slots is misaligned");
  if ((!first && !last) || per == 0) return SC_OK;
  if (misaligned(first, es) || misaligned(last, es)) return fail(SC_EINVAL, "a state is misaligned");
  if (!slots && num_slots < B) return fail(SC_ESHAPE, "fewer state slots than sequences");
  for (int64_t stride : {first ? first_stride : per, last ? last_stride : per})
    if (stride < per || stride > kMaxStride || (long double)num_slots * stride >= 1e17L)
      return fail(SC_ESHAPE, "a state's slot stride is smaller than a state, or too large");
  if (first && last && !(first == last && first_stride == last_stride)) {
    const View f{first, 1, num_slots, per, 0, first_stride, es}, l{last, 1, num_slots, per, 0, last_stride, es};
    if (overlap(f, l)) return fail(SC_EINVAL, "initial_state and final_state overlap and are not the same");
  }
  return SC_OK;
}

sc_status check_scan_sizes(const sc_selective_scan* a) {
  if (!a) return fail(SC_EINVAL, "arguments are NULL");
  if (a->dtype < SC_F32 || a->dtype > SC_F16) return fail(SC_EINVAL, "unknown dtype");
  if (a->flags & ~SC_SEQ_SOFTPLUS) return fail(SC_EINVAL, "unknown flag");
  if (a->B < 0 || a->L < 0 || a->D < 1 || a->N < 1 || a->G < 1) return fail(SC_ESHAPE, "B, L >= 0 and D, N, G >= 1");
  if (a->D % a->G) return fail(SC_ESHAPE, "G does not divide D");
  if (a->N > 256) return fail(SC_EUNSUPPORTED, "N > 256");
  if ((int64_t)a->B * a->D >= (1LL << 31) || a->L >= (1 << 30)) return fail(SC_EUNSUPPORTED, "B*D >= 2^31 or L >= 2^30");
  if (!sc::scan_fits(*a)) return fail(SC_EUNSUPPORTED, "more workgroups than a launch holds");
  return SC_OK;
}

sc_status check_adapter_sizes(const sc_adapter* a) {
  if (!a) return fail(SC_EINVAL, "arguments are NULL");
  if (a->dtype < SC_F32 || a->dtype > SC_F16) return fail(SC_EINVAL, "unknown dtype");
  if (a->reserved) return fail(SC_EINVAL, "reserved is not 0");
  if (a->B < 0 || a->L < 0 || a->C < 1 || a->M < 1 || a->R < 1 || a->adapters < 1)
    return fail(SC_ESHAPE, "B, L >= 0 and C, M, R, adapters >= 1");
  if (a->R > 128) return fail(SC_EUNSUPPORTED, "R > 128");
  if ((int64_t)a->B * a->C * a->R >= (1LL << 31) || (int64_t)a->B * a->M * a->R >= (1LL << 31) || a->L >= (1 << 30))
    return fail(SC_EUNSUPPORTED, "B*C*R or B*M*R >= 2^31, or L >= 2^30");
  if (a->C > sc::kAdapterMost || a->M > sc::kAdapterMost) return fail(SC_EUNSUPPORTED, "C or M > 2^31 - 1024");
  if (!sc::adapter_fits(*a)) return fail(SC_EUNSUPPORTED, "more workgroups than a launch holds");
  return SC_OK;
}

}  // namespace

extern "C" {

sc_status sparseconv_causal_conv(const sc_causal_conv* a, void* hip_stream) {
  return guarded([&]() -> sc_status {
    if (!a) return fail(SC_EINVAL, "arguments are NULL");
    if (a->dtype < SC_F32 || a->dtype > SC_F16) return fail(SC_EINVAL, "unknown dtype");
    if ((a->flags & ~SC_SEQ_SILU) || a->reserved) return fail(SC_EINVAL, "unknown flag, or reserved is not 0");
    if (a->B < 0 || a->L < 0 || a->D < 1 || a->K < 1) return fail(SC_ESHAPE, "B, L >= 0 and D, K >= 1");
    if (a->K > 8) return fail(SC_EUNSUPPORTED, "K > 8");
    if (!sc::conv_fits(*a))
      return fail(SC_EUNSUPPORTED, "B*D*ceil(L/8) >= 2^31");
    if (a->B == 0) return SC_OK;
    const int64_t es = size_of(a->dtype), per = (int64_t)a->D * (a->K - 1);
    if (!a->weight || (a->L && (!a->x || !a->out))) return fail(SC_EINVAL, "x, out or weight is NULL");
    if (misaligned(a->x, es) || misaligned(a->out, es) || misaligned(a->weight, 4) || misaligned(a->bias, 4) ||
        misaligned(a->lengths, 4))
      return fail(SC_EINVAL, "a pointer is not aligned to its type");
    const View x{a->x, a->B, a->D, a->L, a->x_batch, a->x_channel, es};
    const View out{a->out, a->B, a->D, a->L, a->out_batch, a->out_channel, es};
    if (!strides_ok(x) || !strides_ok(out)) return fail(SC_ESHAPE, "a stride is negative or too large");
    if (self_overlaps(out)) return fail(SC_EINVAL, "out's strides make it overlap itself");
    if (sc_status s = check_states(a->initial_state, a->initial_stride, a->final_state, a->final_stride, per, es,
                                   a->slots, a->num_slots, a->B))
      return s;
    const View first{per ? a->initial_state : nullptr, 1, a->num_slots, per, 0, a->initial_stride, es};
    const View last{per ? a->final_state : nullptr, 1, a->num_slots, per, 0, a->final_stride, es};
    const View params[] = {{a->weight, 1, 1, (int64_t)a->D * a->K, 0, 0, 4},
                           {a->bias, 1, 1, a->D, 0, 0, 4},
                           {a->lengths, 1, 1, a->B, 0, 0, 4},
                           {a->slots, 1, 1, a->B, 0, 0, 4}};
    if (overlap(x, out) || overlap(x, last) || overlap(out, first) || overlap(out, last))
      return fail(SC_EINVAL, "an output overlaps an input or the other output");
    for (const View& p : params)
      if (overlap(p, out) || overlap(p, last)) return fail(SC_EINVAL, "an output overlaps an input");
    return launched(sc::launch_causal_conv(*a, hip_stream));
  });
}

sc_status sparseconv_selective_scan_workspace(const sc_selective_scan* a, int64_t* bytes) {
  return guarded([&]() -> sc_status {
    if (!bytes) return fail(SC_EINVAL, "bytes is NULL");
    if (sc_status s = check_scan_sizes(a)) return s;
    *bytes = a->B && a->L ? sc::scan_workspace(*a, device_cus()) : 0;
    return SC_OK;
  });
}

sc_status sparseconv_selective_scan(const sc_selective_scan* a, void* hip_stream) {
  return guarded([&]() -> sc_status {
    if (sc_status s = check_scan_sizes(a)) return s;
    if (a->B == 0) return SC_OK;
    const int64_t es = size_of(a->dtype), per = (int64_t)a->D * a->N;
    if (!a->A || (a->L && (!a->x || !a->dt || !a->b || !a->c || !a->out)))
      return fail(SC_EINVAL, "x, dt, b, c, out or A is NULL");
    for (const void* p : {a->x, a->dt, a->z, a->b, a->c, (const void*)a->out})
      if (misaligned(p, es)) return fail(SC_EINVAL, "a pointer is not aligned to its type");
    for (const void* p : {(const void*)a->A, (const void*)a->skip, (const void*)a->dt_bias, (const void*)a->lengths})
      if (misaligned(p, 4)) return fail(SC_EINVAL, "a pointer is not aligned to its type");
    const View out{a->out, a->B, a->D, a->L, a->out_batch, a->out_channel, es};
    for (int64_t s : {a->b_state, a->c_state})
      if (s < 0 || s > kMaxStride) return fail(SC_ESHAPE, "a stride is negative or too large");
    // of b and c the span alone: a (group, state) pair counts as one block of rows
    const View in[] = {{a->x, a->B, a->D, a->L, a->x_batch, a->x_channel, es},
                       {a->dt, a->B, a->D, a->L, a->dt_batch, a->dt_channel, es},
                       {a->z, a->B, a->D, a->L, a->z_batch, a->z_channel, es}};
    const View bc[] = {{a->b, a->B, a->G, (a->N - 1) * a->b_state + a->L, a->b_batch, a->b_group, es},
                       {a->c, a->B, a->G, (a->N - 1) * a->c_state + a->L, a->c_batch, a->c_group, es}};
    for (const View& v : in)
      if (!strides_ok(v)) return fail(SC_ESHAPE, "a stride is negative or too large");
    for (const View& v : bc)
      if (!strides_ok(v)) return fail(SC_ESHAPE, "a stride is negative or too large");
    if (!strides_ok(out)) return fail(SC_ESHAPE, "a stride is negative or too large");
    if (self_overlaps(out)) return fail(SC_EINVAL, "out's strides make it overlap itself");
    if (sc_status s = check_states(a->initial_state, a->initial_stride, a->final_state, a->final_stride, per, 4,
                                   a->slots, a->num_slots, a->B))
      return s;
    const View first{a->initial_state, 1, a->num_slots, per, 0, a->initial_stride, 4};
    const View last{a->final_state, 1, a->num_slots, per, 0, a->final_stride, 4};
    int64_t need = a->L ? sc::scan_workspace(*a, device_cus()) : 0;
    const View ws{need ? a->workspace : nullptr, 1, 1, need, 0, 0, 1};
    if (need && (!a->workspace || a->workspace_bytes < need))
      return fail(SC_EINVAL, "workspace is NULL or smaller than sparseconv_selective_scan_workspace");
    if (need && misaligned(a->workspace, 16)) return fail(SC_EINVAL, "workspace is not 16-byte aligned");
    const View params[] = {{a->A, 1, 1, per, 0, 0, 4},
                           {a->skip, 1, 1, a->D, 0, 0, 4},
                           {a->dt_bias, 1, 1, a->D, 0, 0, 4},
                           {a->lengths, 1, 1, a->B, 0, 0, 4},
                           {a->slots, 1, 1, a->B, 0, 0, 4}};
    if (overlap(out, first) || overlap(out, last) || overlap(ws, out) || overlap(ws, first) || overlap(ws, last))
      return fail(SC_EINVAL, "out, the states and the workspace overlap");
    for (const View* list : {in, bc, params})
      for (int i = 0, n = list == in ? 3 : list == bc ? 2 : 5; i < n; i++)
        if (overlap(list[i], out) || overlap(list[i], last) || overlap(list[i], ws))
          return fail(SC_EINVAL, "an output or the workspace overlaps an input");
    return launched(sc::launch_selective_scan(*a, device_cus(), hip_stream));
  });
}

sc_status sparseconv_adapter_workspace(const sc_adapter* a, int64_t* bytes) {
  return guarded([&]() -> sc_status {
    if (!bytes) return fail(SC_EINVAL, "bytes is NULL");
    if (sc_status s = check_adapter_sizes(a)) return s;
    *bytes = a->B && a->L ? sc::adapter_workspace(*a, device_cus()) : 0;
    return SC_OK;
  });
}

sc_status sparseconv_adapter_apply(const sc_adapter* a, void* hip_stream) {
  return guarded([&]() -> sc_status {
    if (sc_status s = check_adapter_sizes(a)) return s;
    if (a->B == 0 || a->L == 0) return SC_OK;
    const int64_t es = size_of(a->dtype);
    if (!a->x || !a->out || !a->down || !a->up || !a->index) return fail(SC_EINVAL, "x, out, down, up or index is NULL");
    if (misaligned(a->x, es) || misaligned(a->base, es) || misaligned(a->out, es) || misaligned(a->scale, 4) ||
        misaligned(a->index, 4))
      return fail(SC_EINVAL, "a pointer is not aligned to its type");
    if (misaligned(a->down, 16) || misaligned(a->up, 16)) return fail(SC_EINVAL, "down or up is not 16-byte aligned");
    const View x{a->x, a->B, a->C, a->L, a->x_batch, a->x_channel, es};
    const View base{a->base, a->B, a->M, a->L, a->base_batch, a->base_channel, es};
    const View out{a->out, a->B, a->M, a->L, a->out_batch, a->out_channel, es};
    if (!strides_ok(x) || !strides_ok(base) || !strides_ok(out)) return fail(SC_ESHAPE, "a stride is negative or too large");
    if (self_overlaps(out)) return fail(SC_EINVAL, "out's strides make it overlap itself");
    const int64_t need = sc::adapter_workspace(*a, device_cus());
    const View ws{need ? a->workspace : nullptr, 1, 1, need, 0, 0, 1};
    if (need && (!a->workspace || a->workspace_bytes < need))
      return fail(SC_EINVAL, "workspace is NULL or smaller than sparseconv_adapter_workspace");
    if (need && misaligned(a->workspace, 16)) return fail(SC_EINVAL, "workspace is not 16-byte aligned");
    const bool in_place = a->base == a->out && a->base_batch == a->out_batch && a->base_channel == a->out_channel;
    const View in[] = {x,
                       {in_place ? nullptr : a->base, a->B, a->M, a->L, a->base_batch, a->base_channel, es},
                       {a->down, 1, 1, (int64_t)a->adapters * a->R * a->C, 0, 0, es},
                       {a->up, 1, 1, (int64_t)a->adapters * a->M * a->R, 0, 0, es},
                       {a->scale, 1, 1, a->adapters, 0, 0, 4},
                       {a->index, 1, 1, a->B, 0, 0, 4}};
    for (const View& v : in)
      if (overlap(v, out) || overlap(v, ws)) return fail(SC_EINVAL, "an output or the workspace overlaps an input");
    if (overlap(out, ws) || (in_place && overlap(base, ws))) return fail(SC_EINVAL, "out and the workspace overlap");
    return launched(sc::launch_adapter(*a, device_cus(), hip_stream));
  });
}

}  // extern "C"
