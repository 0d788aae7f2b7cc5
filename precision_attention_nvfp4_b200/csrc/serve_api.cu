// C ABI of the serving entry points: argument validation, the host-side
// rotary frequencies and tree masks, dispatch to the kernels. See
// include/fpattn.h.
#include <cmath>
#include <cstdint>

#include <cuda_runtime.h>

#include "../../include/fpattn.h"
#include "serve_internal.h"

namespace {

constexpr long double kPi = 3.14159265358979323846264338327950288L;

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

fpattn_status from_cuda(cudaError_t e) {
  if (e == cudaSuccess) return FPATTN_OK;
  if (e == cudaErrorNotSupported) return FPATTN_ERR_UNSUPPORTED;
  return FPATTN_ERR_CUDA;
}

fpattn_status check_rows(const fpattn_rows* r, fpattn::Rows* out) {
  if (!r || !r->data) return FPATTN_ERR_INVALID_ARG;
  if (r->B <= 0 || r->T <= 0 || r->H <= 0) return FPATTN_ERR_INVALID_ARG;
  if (r->d != 64 && r->d != 128) return FPATTN_ERR_UNSUPPORTED;
  // heads are a grid's y index and tokens are counted in 32 bits
  if (r->H > 16384 || static_cast<long long>(r->B) * r->T > (1ll << 31) - 1) return FPATTN_ERR_UNSUPPORTED;
  // the stride of an axis of one is never taken
  const int64_t sb = r->B > 1 ? r->stride_b : 0, st = r->T > 1 ? r->stride_t : 0, sh = r->H > 1 ? r->stride_h : 0;
  if (!aligned(r->data, 16) || ((sb | st | sh) & 7)) return FPATTN_ERR_ALIGNMENT;
  *out = fpattn::Rows{r->data, r->B, r->T, r->H, r->d, sb, st, sh};
  return FPATTN_OK;
}

fpattn_status check_table(const fpattn_rotary_table* t, int d, fpattn::RotaryTable* out) {
  if (!t || !t->turns) return FPATTN_ERR_INVALID_ARG;
  if (t->dim < 16 || t->dim % 16 != 0 || t->dim > d) return FPATTN_ERR_INVALID_ARG;
  if (t->layout != FPATTN_ROTARY_HALF && t->layout != FPATTN_ROTARY_INTERLEAVED) return FPATTN_ERR_INVALID_ARG;
  if (!(std::isfinite(t->magnitude) && t->magnitude > 0.f)) return FPATTN_ERR_INVALID_ARG;
  if (!aligned(t->turns, 8)) return FPATTN_ERR_ALIGNMENT;
  *out = fpattn::RotaryTable{reinterpret_cast<const unsigned long long*>(t->turns), t->dim,
                             t->layout == FPATTN_ROTARY_INTERLEAVED, t->magnitude};
  return FPATTN_OK;
}

fpattn_status check_cache(const fpattn_kv_cache* c, fpattn::KvCache* out) {
  if (!c || !c->k_codes || !c->v_codes || !c->exps) return FPATTN_ERR_INVALID_ARG;
  if (c->num_pages <= 0 || c->H <= 0) return FPATTN_ERR_INVALID_ARG;
  if (c->d != 64 && c->d != 128) return FPATTN_ERR_UNSUPPORTED;
  if (c->page_size != 16 && c->page_size != 32 && c->page_size != 64 && c->page_size != 128)
    return FPATTN_ERR_UNSUPPORTED;
  // (page, head) is one 32-bit coordinate of the kernel's loads
  if (c->H > 4096 || static_cast<long long>(c->num_pages) * c->H > (1ll << 31) - 1) return FPATTN_ERR_UNSUPPORTED;
  if (!aligned(c->k_codes, 16) || !aligned(c->v_codes, 16) || !aligned(c->exps, 16)) return FPATTN_ERR_ALIGNMENT;
  *out = fpattn::KvCache{c->k_codes, c->v_codes, c->exps, c->num_pages, c->H, c->page_size, c->d};
  return FPATTN_OK;
}

fpattn_status check_queries(const fpattn_kv_cache* cache, const fpattn_cache_queries* q, fpattn::CacheAttnArgs* a) {
  fpattn_status s = check_cache(cache, &a->cache);
  if (s != FPATTN_OK) return s;
  if (!q) return FPATTN_ERR_INVALID_ARG;
  fpattn::Rows r;
  if ((s = check_rows(&q->q, &r)) != FPATTN_OK) return s;
  if (r.d != a->cache.d || r.H % a->cache.H != 0) return FPATTN_ERR_INVALID_ARG;
  if (q->B <= 0 || q->max_queries <= 0 || q->max_pages <= 0) return FPATTN_ERR_INVALID_ARG;
  if (q->q_start ? r.B != 1 : (r.B != q->B || r.T != q->max_queries)) return FPATTN_ERR_INVALID_ARG;
  if (!q->page_table || !q->lengths || q->page_table_stride < 0) return FPATTN_ERR_INVALID_ARG;
  if (q->tree_mask && (q->tree_words < (static_cast<long long>(q->max_queries) + 63) / 64 || q->tree_stride_b < 0))
    return FPATTN_ERR_INVALID_ARG;
  if (!(q->softmax_scale >= 0.f && q->softmax_scale <= 1e30f)) return FPATTN_ERR_INVALID_ARG;
  if (!aligned(q->page_table, 4) || !aligned(q->lengths, 4) || !aligned(q->q_start, 4) || !aligned(q->tree_mask, 8))
    return FPATTN_ERR_ALIGNMENT;
  // keys, rows and (below) the work of the whole call are counted in 32 bits
  const long long keys = static_cast<long long>(q->max_pages) * a->cache.page_size;
  const long long rows = static_cast<long long>(q->max_queries) * (r.H / a->cache.H);
  if (keys > (1ll << 30) || rows > (1ll << 28) || q->B > (1 << 24)) return FPATTN_ERR_UNSUPPORTED;
  a->q = r.data;
  a->q_sb = r.sb, a->q_st = r.st, a->q_sh = r.sh;
  a->q_start = q->q_start;
  a->B = q->B;
  a->Tmax = q->max_queries;
  a->rows_total = q->q_start ? r.T : r.B * r.T;
  a->Hq = r.H;
  a->page_table = q->page_table;
  a->max_pages = q->max_pages;
  a->page_table_stride = q->page_table_stride;
  a->lengths = q->lengths;
  a->causal = q->causal != 0;
  a->tree = reinterpret_cast<const long long*>(q->tree_mask);
  a->tree_words = q->tree_words;
  a->tree_sb = q->tree_stride_b;
  if (fpattn::cache_attention_units(*a) > static_cast<double>(1ll << 30)) return FPATTN_ERR_UNSUPPORTED;
  a->scale = q->softmax_scale > 0.f ? q->softmax_scale : 1.0f / std::sqrt(static_cast<float>(a->cache.d));
  return FPATTN_OK;
}

bool same_shape(const fpattn::Rows& a, const fpattn::Rows& b) {
  return a.B == b.B && a.T == b.T && a.H == b.H && a.d == b.d;
}

}  // namespace

extern "C" {

fpattn_status fpattn_rotary_turns(const fpattn_rotary_spec* spec, uint64_t* turns, float* magnitude) {
  if (!spec || !turns || !magnitude) return FPATTN_ERR_INVALID_ARG;
  const fpattn_rotary_spec& s = *spec;
  if (s.dim < 16 || s.dim % 16 != 0 || s.dim > 65536) return FPATTN_ERR_INVALID_ARG;
  if (s.scaling < FPATTN_ROTARY_NONE || s.scaling > FPATTN_ROTARY_WAVELENGTH) return FPATTN_ERR_INVALID_ARG;
  if (!(std::isfinite(s.base) && s.base > 1.0)) return FPATTN_ERR_INVALID_ARG;
  if (s.scaling != FPATTN_ROTARY_NONE && !(std::isfinite(s.factor) && s.factor >= 1.0)) return FPATTN_ERR_INVALID_ARG;
  const bool ramp = s.scaling == FPATTN_ROTARY_YARN || s.scaling == FPATTN_ROTARY_WAVELENGTH;
  if (ramp && !(std::isfinite(s.original_length) && s.original_length > 0.0 && s.slow > 0.0 && s.fast > s.slow &&
                std::isfinite(s.fast)))
    return FPATTN_ERR_INVALID_ARG;
  if (!(std::isfinite(s.magnitude) && s.magnitude >= 0.0)) return FPATTN_ERR_INVALID_ARG;
  // long double has the 64 bits of mantissa that the turns have
  using real = long double;
  const int half = s.dim / 2;
  const real dim = s.dim, factor = s.factor, slow = s.slow, fast = s.fast, length = s.original_length;
  const real base = s.scaling == FPATTN_ROTARY_NTK ? s.base * std::pow(factor, dim / (dim - 2)) : static_cast<real>(s.base);
  real lo = 0, hi = 0;
  if (s.scaling == FPATTN_ROTARY_YARN) {
    auto at = [&](real t) { return dim * std::log(length / (2 * kPi * t)) / (2 * std::log(base)); };
    lo = std::fmax(real(0), std::floor(at(fast)));
    hi = std::fmin(dim - 1, std::ceil(at(slow)));
  }
  for (int i = 0; i < half; ++i) {
    real f = std::pow(base, -2 * i / dim);
    if (s.scaling == FPATTN_ROTARY_LINEAR) {
      f /= factor;
    } else if (s.scaling == FPATTN_ROTARY_YARN) {
      const real r = std::fmin(real(1), std::fmax(real(0), (i - lo) / std::fmax(hi - lo, static_cast<real>(1e-3))));
      f = f * (1 - r) + f / factor * r;
    } else if (s.scaling == FPATTN_ROTARY_WAVELENGTH) {
      const real n = length * f / (2 * kPi);
      const real k = std::fmin(real(1), std::fmax(real(0), (n - slow) / (fast - slow)));
      f = f * k + f / factor * (1 - k);
    }
    turns[i] = static_cast<uint64_t>(std::rint(std::ldexp(f / (2 * kPi), 64)));  // f <= 1: below 2^62
  }
  *magnitude = static_cast<float>(
      s.magnitude > 0.0 ? s.magnitude : (s.scaling == FPATTN_ROTARY_YARN ? 0.1 * std::log(s.factor) + 1.0 : 1.0));
  return FPATTN_OK;
}

fpattn_status fpattn_rotary(const fpattn_rows* x, const fpattn_rotary_table* table, const int64_t* positions,
                            int32_t positions_per_b, int32_t transpose, const fpattn_rows* out,
                            fpattn_stream_t stream) {
  fpattn::Rows xr, o;
  fpattn::RotaryTable tab;
  fpattn_status s;
  if ((s = check_rows(x, &xr)) != FPATTN_OK) return s;
  if ((s = check_rows(out, &o)) != FPATTN_OK) return s;
  if ((s = check_table(table, xr.d, &tab)) != FPATTN_OK) return s;
  if (!positions || !same_shape(xr, o)) return FPATTN_ERR_INVALID_ARG;
  if (xr.data == o.data && (xr.sb != o.sb || xr.st != o.st || xr.sh != o.sh)) return FPATTN_ERR_INVALID_ARG;
  if (!aligned(positions, 8)) return FPATTN_ERR_ALIGNMENT;
  return from_cuda(fpattn::launch_rotary(xr, tab, reinterpret_cast<const long long*>(positions), positions_per_b != 0,
                                         transpose != 0, o, reinterpret_cast<cudaStream_t>(stream)));
}

fpattn_status fpattn_cache_write(const fpattn_kv_cache* cache, const fpattn_rows* k, const fpattn_rows* v,
                                 const int64_t* slots, const fpattn_rotary_table* table, const int64_t* positions,
                                 const fpattn_rows* q, const fpattn_rows* q_out, int32_t* nonfinite_flag,
                                 fpattn_stream_t stream) {
  fpattn::KvCache c;
  fpattn::Rows kr, vr, qr, qo;
  fpattn::RotaryTable tab{};
  fpattn_status s;
  if ((s = check_cache(cache, &c)) != FPATTN_OK) return s;
  if ((s = check_rows(k, &kr)) != FPATTN_OK) return s;
  if ((s = check_rows(v, &vr)) != FPATTN_OK) return s;
  if (!same_shape(kr, vr) || kr.B != 1 || kr.H != c.H || kr.d != c.d || !slots) return FPATTN_ERR_INVALID_ARG;
  if (table) {
    if ((s = check_table(table, c.d, &tab)) != FPATTN_OK) return s;
    if (!positions) return FPATTN_ERR_INVALID_ARG;
  }
  if (!q != !q_out || (q && !table)) return FPATTN_ERR_INVALID_ARG;
  if (q) {
    if ((s = check_rows(q, &qr)) != FPATTN_OK) return s;
    if ((s = check_rows(q_out, &qo)) != FPATTN_OK) return s;
    if (!same_shape(qr, qo) || qr.B != 1 || qr.T != kr.T || qr.d != c.d) return FPATTN_ERR_INVALID_ARG;
    if (qr.data == qo.data && (qr.st != qo.st || qr.sh != qo.sh)) return FPATTN_ERR_INVALID_ARG;
  }
  if (!aligned(slots, 8) || !aligned(positions, 8) || !aligned(nonfinite_flag, 4)) return FPATTN_ERR_ALIGNMENT;
  return from_cuda(fpattn::launch_cache_write(c, kr, vr, reinterpret_cast<const long long*>(slots), tab,
                                              reinterpret_cast<const long long*>(positions), q ? &qr : nullptr,
                                              q ? &qo : nullptr, nonfinite_flag,
                                              reinterpret_cast<cudaStream_t>(stream)));
}

fpattn_status fpattn_cache_read(const fpattn_kv_cache* cache, const int64_t* slots, const fpattn_rows* k_out,
                                const fpattn_rows* v_out, fpattn_stream_t stream) {
  fpattn::KvCache c;
  fpattn::Rows kr, vr;
  fpattn_status s;
  if ((s = check_cache(cache, &c)) != FPATTN_OK) return s;
  if ((s = check_rows(k_out, &kr)) != FPATTN_OK) return s;
  if ((s = check_rows(v_out, &vr)) != FPATTN_OK) return s;
  if (!same_shape(kr, vr) || kr.B != 1 || kr.H != c.H || kr.d != c.d || !slots) return FPATTN_ERR_INVALID_ARG;
  if (!aligned(slots, 8)) return FPATTN_ERR_ALIGNMENT;
  return from_cuda(fpattn::launch_cache_read(c, reinterpret_cast<const long long*>(slots), kr, vr,
                                             reinterpret_cast<cudaStream_t>(stream)));
}

size_t fpattn_cache_attention_workspace(const fpattn_kv_cache* cache, const fpattn_cache_queries* queries) {
  fpattn::CacheAttnArgs a{};
  if (check_queries(cache, queries, &a) != FPATTN_OK) return 0;
  return fpattn::cache_attention_workspace(a);
}

fpattn_status fpattn_cache_attention(const fpattn_kv_cache* cache, const fpattn_cache_queries* queries, void* out,
                                     float* lse, void* workspace, size_t workspace_bytes, fpattn_stream_t stream) {
  fpattn::CacheAttnArgs a{};
  const fpattn_status s = check_queries(cache, queries, &a);
  if (s != FPATTN_OK) return s;
  if (!out) return FPATTN_ERR_INVALID_ARG;
  const size_t need = fpattn::cache_attention_workspace(a);
  if (need > 0 && (!workspace || workspace_bytes < need)) return FPATTN_ERR_INVALID_ARG;
  if (!aligned(out, 16) || !aligned(lse, 4) || (need > 0 && !aligned(workspace, 256))) return FPATTN_ERR_ALIGNMENT;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  return from_cuda(fpattn::launch_cache_attention(a, reinterpret_cast<cudaStream_t>(stream)));
}

fpattn_status fpattn_tree_mask(const int32_t* parents, int32_t n, int32_t words_per_row, int64_t* words,
                               int32_t* depth) {
  if (!parents || !words || n < 1 || words_per_row < (static_cast<int64_t>(n) + 63) / 64) return FPATTN_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i)
    if (parents[i] < -1 || parents[i] >= i) return FPATTN_ERR_INVALID_ARG;
  for (int32_t i = 0; i < n; ++i) {
    uint64_t* row = reinterpret_cast<uint64_t*>(words) + static_cast<size_t>(i) * words_per_row;
    const uint64_t* up = parents[i] < 0 ? nullptr
                                        : reinterpret_cast<uint64_t*>(words) +
                                              static_cast<size_t>(parents[i]) * words_per_row;
    for (int32_t w = 0; w < words_per_row; ++w) row[w] = up ? up[w] : 0u;
    row[i / 64] |= 1ull << (i % 64);
    if (depth) depth[i] = parents[i] < 0 ? 0 : depth[parents[i]] + 1;
  }
  return FPATTN_OK;
}

}  // extern "C"
