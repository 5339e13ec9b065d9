// Entry points of the attention operators (declared in include/sparseconv.h): the argument checks,
// then a launch on the caller's stream.
#include "attention.h"

#include <cmath>

#include "attention_plan.h"
#include "checks.h"

namespace {

bool bad_dtype(int t) { return t < SC_F32 || t > SC_F16; }

// The cache's part of the checks: G heads of D dims, pages of P positions, a table of `width` pages a sequence.
sc_status check_cache_sizes(int G, int D, int P, int width, int pages) {
  if (G < 1 || D < 1 || width < 0 || pages < 1) return fail(SC_ESHAPE, "G, D, pages >= 1 and width >= 0");
  if (G > 65536) return fail(SC_EUNSUPPORTED, "G > 2^16");
  if (D % 8 || D > 256) return fail(SC_EUNSUPPORTED, "D is not a multiple of 8 up to 256");
  if (P < 16 || P > 256 || (P & (P - 1))) return fail(SC_EUNSUPPORTED, "P is not 16, 32, 64, 128 or 256");
  if ((int64_t)width * P > (1 << 30)) return fail(SC_EUNSUPPORTED, "width*P > 2^30");
  return SC_OK;
}

sc_status check_cache(const void* k, const void* v, int64_t k_page, int64_t v_page, int64_t per, int pages, int64_t es,
                      const int32_t* table, int64_t table_batch, int B, int width) {
  if (!k || !v) return fail(SC_EINVAL, "k_pages or v_pages is NULL");
  if (misaligned(k, 16) || misaligned(v, 16)) return fail(SC_EINVAL, "k_pages or v_pages is not 16-byte aligned");
  if (!table && width) return fail(SC_EINVAL, "table is NULL");
  if (misaligned(table, 4)) return fail(SC_EINVAL, "table is misaligned");
  for (int64_t s : {k_page, v_page}) {
    if (s < per || s > kMaxStride || (long double)pages * s >= 1e17L)
      return fail(SC_ESHAPE, "a page stride is smaller than a page, or too large");
    if (s * es % 16) return fail(SC_EINVAL, "a page stride is no multiple of 16 bytes");
  }
  if (table_batch < 0 || table_batch > kMaxStride || (long double)B * table_batch >= 1e17L)
    return fail(SC_ESHAPE, "the table's stride is negative or too large");
  return SC_OK;
}

View table_view(const int32_t* t, int B, int64_t batch, int width) { return {t, 1, B, width, 0, batch, 4}; }

sc_status check_attend_sizes(const sc_paged_attention* a) {
  if (!a) return fail(SC_EINVAL, "arguments are NULL");
  if (bad_dtype(a->dtype)) return fail(SC_EINVAL, "unknown dtype");
  if ((a->flags & ~SC_ATT_OUT_F32) || a->reserved) return fail(SC_EINVAL, "unknown flag, or reserved is not 0");
  if (a->B < 0 || a->L < 0 || a->H < 1 || a->window < 0) return fail(SC_ESHAPE, "B, L, window >= 0 and H >= 1");
  if (sc_status s = check_cache_sizes(a->G, a->D, a->P, a->width, a->pages)) return s;
  if (a->H % a->G) return fail(SC_ESHAPE, "G does not divide H");
  if (a->H > 65536 || a->L >= (1 << 30)) return fail(SC_EUNSUPPORTED, "H > 2^16 or L >= 2^30");
  if (!sc::attend_fits(*a)) return fail(SC_EUNSUPPORTED, "more workgroups than a launch holds");
  return SC_OK;
}

}  // namespace

extern "C" {

sc_status sparseconv_paged_attention_workspace(const sc_paged_attention* a, int64_t* bytes) {
  return guarded([&]() -> sc_status {
    if (!bytes) return fail(SC_EINVAL, "bytes is NULL");
    if (sc_status s = check_attend_sizes(a)) return s;
    *bytes = sc::attend_workspace(*a, device_cus());
    return SC_OK;
  });
}

sc_status sparseconv_paged_attention(const sc_paged_attention* a, void* hip_stream) {
  return guarded([&]() -> sc_status {
    if (sc_status s = check_attend_sizes(a)) return s;
    if (a->B == 0 || a->L == 0) return SC_OK;
    const int64_t es = size_of(a->dtype), os = a->flags & SC_ATT_OUT_F32 ? 4 : es, per = (int64_t)a->G * a->P * a->D;
    if (!a->q || !a->out || !a->past) return fail(SC_EINVAL, "q, out or past is NULL");
    // (the kernels use scale log2(e), scale / cap and cap log2(e))
    if (!std::isfinite(1.5f * a->scale) || !std::isfinite(1.5f * a->cap) || a->cap < 0 || (a->cap > 0 && !std::isfinite(a->scale / a->cap)))
      return fail(SC_EINVAL, "scale, cap or scale / cap is not finite, or cap < 0");
    if (misaligned(a->q, es) || misaligned(a->out, os) || misaligned(a->past, 4) || misaligned(a->lengths, 4) ||
        misaligned(a->prefix, 4) || misaligned(a->slopes, 4))
      return fail(SC_EINVAL, "a pointer is not aligned to its type");
    if (sc_status s = check_cache(a->k_pages, a->v_pages, a->k_page, a->v_page, per, a->pages, es, a->table, a->table_batch, a->B, a->width))
      return s;
    const View q{a->q, a->B, (int64_t)a->H * a->D, a->L, a->q_batch, a->q_channel, es};
    const View out{a->out, a->B, (int64_t)a->H * a->D, a->L, a->out_batch, a->out_channel, os};
    if (!strides_ok(q) || !strides_ok(out)) return fail(SC_ESHAPE, "a stride is negative or too large");
    if (self_overlaps(out)) return fail(SC_EINVAL, "out's strides make it overlap itself");
    const int64_t need = sc::attend_workspace(*a, device_cus());
    const View ws{need ? a->workspace : nullptr, 1, 1, need, 0, 0, 1};
    if (need && (!a->workspace || a->workspace_bytes < need))
      return fail(SC_EINVAL, "workspace is NULL or smaller than sparseconv_paged_attention_workspace");
    if (need && misaligned(a->workspace, 16)) return fail(SC_EINVAL, "workspace is not 16-byte aligned");
    const View in[] = {q,
                       {a->k_pages, 1, a->pages, per, 0, a->k_page, es},
                       {a->v_pages, 1, a->pages, per, 0, a->v_page, es},
                       table_view(a->table, a->B, a->table_batch, a->width),
                       {a->past, 1, 1, a->B, 0, 0, 4},
                       {a->lengths, 1, 1, a->B, 0, 0, 4},
                       {a->prefix, 1, 1, a->B, 0, 0, 4},
                       {a->slopes, 1, 1, a->H, 0, 0, 4}};
    for (const View& v : in)
      if (overlap(v, out) || overlap(v, ws)) return fail(SC_EINVAL, "out or the workspace overlaps an input");
    if (overlap(out, ws)) return fail(SC_EINVAL, "out and the workspace overlap");
    return launched(sc::launch_paged_attention(*a, device_cus(), hip_stream));
  });
}

sc_status sparseconv_cache_append(const sc_cache_append* a, void* hip_stream) {
  return guarded([&]() -> sc_status {
    if (!a) return fail(SC_EINVAL, "arguments are NULL");
    if (bad_dtype(a->dtype) || bad_dtype(a->cache_dtype)) return fail(SC_EINVAL, "unknown dtype");
    if (a->cache_dtype != a->dtype && a->dtype != SC_F32) return fail(SC_EINVAL, "the cache's type is neither dtype nor narrower than fp32");
    if ((a->flags & ~SC_ROT_INTERLEAVED) || a->reserved) return fail(SC_EINVAL, "unknown flag, or reserved is not 0");
    if (a->B < 0 || a->L < 0 || a->H < (a->q ? 1 : 0)) return fail(SC_ESHAPE, "B, L >= 0, and H >= 1 with q");
    if (sc_status s = check_cache_sizes(a->G, a->D, a->P, a->width, a->pages)) return s;
    if (a->pairs < 0 || 2LL * a->pairs > a->D || a->num_axes < 1) return fail(SC_ESHAPE, "0 <= 2*pairs <= D and num_axes >= 1");
    if (a->H > 65536 || a->L >= (1 << 30)) return fail(SC_EUNSUPPORTED, "H > 2^16 or L >= 2^30");
    if (!sc::append_fits(*a)) return fail(SC_EUNSUPPORTED, "more workgroups than a launch holds");
    if (a->B == 0 || a->L == 0) return SC_OK;
    const int64_t es = size_of(a->dtype), cs = size_of(a->cache_dtype), per = (int64_t)a->G * a->P * a->D;
    if (!a->k || !a->v || !a->past || (a->q && !a->q_out) || (a->pairs && !a->freqs)) return fail(SC_EINVAL, "q_out, k, v, past or freqs is NULL");
    if (misaligned(a->q, es) || misaligned(a->q_out, cs) || misaligned(a->k, es) || misaligned(a->v, es) || misaligned(a->freqs, 8) ||
        misaligned(a->axes, 4) || misaligned(a->positions, 4) || misaligned(a->past, 4) || misaligned(a->lengths, 4))
      return fail(SC_EINVAL, "a pointer is not aligned to its type");
    if (sc_status s = check_cache(a->k_pages, a->v_pages, a->k_page, a->v_page, per, a->pages, cs, a->table, a->table_batch, a->B, a->width))
      return s;
    const bool in_place = a->q && a->q == a->q_out && a->dtype == a->cache_dtype && a->q_batch == a->q_out_batch && a->q_channel == a->q_out_channel;
    const View q{a->q, a->B, (int64_t)a->H * a->D, a->L, a->q_batch, a->q_channel, es};
    const View q_out{a->q ? a->q_out : nullptr, a->B, (int64_t)a->H * a->D, a->L, a->q_out_batch, a->q_out_channel, cs};
    const View k{a->k, a->B, (int64_t)a->G * a->D, a->L, a->k_batch, a->k_channel, es};
    const View v{a->v, a->B, (int64_t)a->G * a->D, a->L, a->v_batch, a->v_channel, es};
    const View positions{a->positions, a->B, a->num_axes, a->L, a->positions_batch, a->positions_axis, 4};
    if ((a->q && (!strides_ok(q) || !strides_ok(q_out))) || !strides_ok(k) || !strides_ok(v) || (a->positions && !strides_ok(positions)))
      return fail(SC_ESHAPE, "a stride is negative or too large");
    if (self_overlaps(q_out)) return fail(SC_EINVAL, "q_out's strides make it overlap itself");
    const View kp{a->k_pages, 1, a->pages, per, 0, a->k_page, cs}, vp{a->v_pages, 1, a->pages, per, 0, a->v_page, cs};
    // keys and values of one allocation, page by page
    const View both[2] = {{a->k_pages, a->pages, 1, per, a->k_page, 0, cs}, {a->v_pages, a->pages, 1, per, a->v_page, 0, cs}};
    if (overlap(both[0], both[1])) return fail(SC_EINVAL, "k_pages and v_pages overlap");
    const View in[] = {q, k, v, positions, table_view(a->table, a->B, a->table_batch, a->width),
                       {a->freqs, 1, 1, a->pairs, 0, 0, 8},
                       {a->axes, 1, 1, a->pairs, 0, 0, 4},
                       {a->past, 1, 1, a->B, 0, 0, 4},
                       {a->lengths, 1, 1, a->B, 0, 0, 4}};
    for (const View& i : in)
      if (overlap(i, kp) || overlap(i, vp) || (!(in_place && i.p == q.p && &i == in) && overlap(i, q_out)))
        return fail(SC_EINVAL, "an output overlaps an input");
    if (overlap(q_out, kp) || overlap(q_out, vp)) return fail(SC_EINVAL, "q_out and the cache overlap");
    return launched(sc::launch_cache_append(*a, device_cus(), hip_stream));
  });
}

sc_status sparseconv_cache_copy(const sc_cache_copy* a, void* hip_stream) {
  return guarded([&]() -> sc_status {
    if (!a) return fail(SC_EINVAL, "arguments are NULL");
    if (a->reserved) return fail(SC_EINVAL, "reserved is not 0");
    if (a->outer < 0 || a->pages < 0 || a->count < 0 || a->page_bytes < 0) return fail(SC_ESHAPE, "outer, pages, count, page_bytes >= 0");
    if (a->page_bytes > kMaxStride) return fail(SC_EUNSUPPORTED, "page_bytes is too large");
    if (!sc::copy_fits(*a)) return fail(SC_EUNSUPPORTED, "more workgroups than a launch holds");
    if (!a->outer || !a->pages || !a->count || !a->page_bytes) return SC_OK;
    if (!a->pool || !a->source || !a->target) return fail(SC_EINVAL, "pool, source or target is NULL");
    if (misaligned(a->source, 4) || misaligned(a->target, 4)) return fail(SC_EINVAL, "a pointer is not aligned to its type");
    const View pool{a->pool, a->outer, a->pages, a->page_bytes, a->outer_stride, a->page_stride, 1};
    if (!strides_ok(pool)) return fail(SC_ESHAPE, "a stride is negative or too large");
    if (self_overlaps(pool)) return fail(SC_EINVAL, "pool's strides make it overlap itself");
    if (overlap(pool, View{a->source, 1, 1, a->count, 0, 0, 4}) || overlap(pool, View{a->target, 1, 1, a->count, 0, 0, 4}))
      return fail(SC_EINVAL, "source or target lies in the pool");
    return launched(sc::launch_cache_copy(*a, hip_stream));
  });
}

sc_status sparseconv_residual_norm(const sc_residual_norm* a, void* hip_stream) {
  return guarded([&]() -> sc_status {
    if (!a) return fail(SC_EINVAL, "arguments are NULL");
    if (bad_dtype(a->dtype)) return fail(SC_EINVAL, "unknown dtype");
    if ((a->flags & ~SC_NORM_CENTER) || a->reserved) return fail(SC_EINVAL, "unknown flag, or reserved is not 0");
    if (a->B < 0 || a->L < 0 || a->C < 1) return fail(SC_ESHAPE, "B, L >= 0 and C >= 1");
    if (a->C >= (1 << 20) || a->L >= (1 << 30) || !sc::norm_fits(*a)) return fail(SC_EUNSUPPORTED, "C >= 2^20, L >= 2^30 or B*ceil(L/4) >= 2^22");
    if (a->B == 0 || a->L == 0) return SC_OK;
    const int64_t es = size_of(a->dtype);
    if (!a->x || (!a->sum && !a->out)) return fail(SC_EINVAL, "x, or both of sum and out, is NULL");
    if (!a->y && (a->gate || a->post_weight)) return fail(SC_EINVAL, "gate or post_weight without y");
    if ((!a->post_weight && a->post_bias) || (!a->out && (a->weight || a->bias)))
      return fail(SC_EINVAL, "post_bias without post_weight, or weight or bias without out");
    if (!std::isfinite(a->scale) || !std::isfinite(a->eps) || a->eps < 0) return fail(SC_EINVAL, "scale or eps is not finite, or eps < 0");
    for (const void* p : {a->x, a->y, a->gate, (const void*)a->sum, (const void*)a->out})
      if (misaligned(p, es)) return fail(SC_EINVAL, "a pointer is not aligned to its type");
    for (const float* p : {a->weight, a->bias, a->post_weight, a->post_bias})
      if (misaligned(p, 4)) return fail(SC_EINVAL, "a pointer is not aligned to its type");
    const View x{a->x, a->B, a->C, a->L, a->x_batch, a->x_channel, es}, y{a->y, a->B, a->C, a->L, a->y_batch, a->y_channel, es};
    const View sum{a->sum, a->B, a->C, a->L, a->sum_batch, a->sum_channel, es}, out{a->out, a->B, a->C, a->L, a->out_batch, a->out_channel, es};
    const View gate{a->gate, a->B, a->C, a->gate_position ? a->L : 1, a->gate_batch, a->gate_channel, es};
    if (a->gate_position != 0 && a->gate_position != 1) return fail(SC_ESHAPE, "gate_position is neither 0 nor 1");
    for (const View* v : {&x, &y, &sum, &out, &gate})
      if (v->p && !strides_ok(*v)) return fail(SC_ESHAPE, "a stride is negative or too large");
    if (self_overlaps(sum) || self_overlaps(out)) return fail(SC_EINVAL, "an output's strides make it overlap itself");
    auto same = [](const View& u, const View& v) { return u.p == v.p && u.outer_stride == v.outer_stride && u.row_stride == v.row_stride; };
    if ((overlap(x, sum) && !same(x, sum)) || (overlap(y, out) && !same(y, out)) || overlap(x, out) || overlap(y, sum) ||
        overlap(sum, out) || overlap(gate, sum) || overlap(gate, out))
      return fail(SC_EINVAL, "an output overlaps an input or the other output");
    for (const float* p : {a->weight, a->bias, a->post_weight, a->post_bias}) {
      const View v{p, 1, 1, a->C, 0, 0, 4};
      if (overlap(v, sum) || overlap(v, out)) return fail(SC_EINVAL, "an output overlaps an input");
    }
    return launched(sc::launch_residual_norm(*a, device_cus(), hip_stream));
  });
}

}  // extern "C"
