// C ABI of the serving operators: argument validation and dispatch (see
// include/ssa.h for the contract).
#include <math.h>
#include <stdint.h>

#include "kernels.h"
#include "ssa.h"

namespace {

using ssa::LaunchCtx;

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
ssa_status from_cuda(cudaError_t e) { return e == cudaSuccess ? SSA_OK : SSA_ERR_CUDA; }

// Elements between tokens of an operand of `heads` heads.
bool bad_stride(int64_t stride, int64_t heads, int d, int es) {
  return stride < heads * d || stride % (16 / es) != 0 || stride > (int64_t{1} << 40);
}

// Rotation and norm fields, shared by the rotation and the append.
ssa_status check_rotation(int d, int rot, int layout, int dtype, int norm, float eps, float mscale) {
  if (d < 1 || rot < 0 || rot > d || (layout != SSA_ROPE_HALF && layout != SSA_ROPE_PAIRS) ||
      (dtype != SSA_F32 && dtype != SSA_BF16) || (norm != 0 && norm != 1) || !isfinite(eps) || eps < 0.f ||
      !isfinite(mscale))
    return SSA_ERR_INVALID_ARG;
  if ((d != 64 && d != 128) || rot % 16 != 0) return SSA_ERR_UNSUPPORTED;
  return SSA_OK;
}

ssa_status check_rope(const ssa_rope_params* p) {
  if (!p || p->n_tokens < 0 || p->h_q < 1 || p->h_kv < 1) return SSA_ERR_INVALID_ARG;
  const ssa_status st = check_rotation(p->d, p->rot, p->layout, p->dtype, p->norm, p->eps, p->mscale);
  if (st != SSA_OK) return st;
  const int es = p->dtype == SSA_BF16 ? 2 : 4;
  if (bad_stride(p->q_stride, p->h_q, p->d, es) || bad_stride(p->k_stride, p->h_kv, p->d, es) ||
      bad_stride(p->q_out_stride, p->h_q, p->d, es) || bad_stride(p->k_out_stride, p->h_kv, p->d, es))
    return SSA_ERR_INVALID_ARG;
  if (p->h_q > 65535 || p->h_kv > 65535) return SSA_ERR_UNSUPPORTED;
  return SSA_OK;
}

// The cache's own shape.
ssa_status check_cache(int n_seq, int max_pages, int n_pages, int page, int h_kv, int d) {
  if (n_seq < 0 || max_pages < 0 || n_pages < 0 || page < 1 || h_kv < 1 || d < 1) return SSA_ERR_INVALID_ARG;
  if ((page != 64 && page != 128) || (d != 64 && d != 128)) return SSA_ERR_UNSUPPORTED;
  // token positions are int32
  if (static_cast<int64_t>(max_pages) * page > INT32_MAX || h_kv > 65535) return SSA_ERR_UNSUPPORTED;
  return SSA_OK;
}

ssa_status check_append(const ssa_append_params* p) {
  if (!p || p->n_tokens < 0 || p->reserved != 0) return SSA_ERR_INVALID_ARG;
  ssa_status st = check_rotation(p->d, p->rot, p->layout, p->dtype, p->norm, p->eps, p->mscale);
  if (st != SSA_OK) return st;
  if ((st = check_cache(p->n_seq, p->max_pages, p->n_pages, p->page, p->h_kv, p->d)) != SSA_OK) return st;
  const int es = p->dtype == SSA_BF16 ? 2 : 4;
  if (bad_stride(p->k_stride, p->h_kv, p->d, es) || bad_stride(p->v_stride, p->h_kv, p->d, es))
    return SSA_ERR_INVALID_ARG;
  if (p->n_seq > (1 << 24)) return SSA_ERR_UNSUPPORTED;
  // pages that the tokens may touch, times kv-heads: the launch counts them in 32 bits
  if ((p->n_tokens / p->page + 2 * static_cast<int64_t>(p->n_seq)) * p->h_kv > INT32_MAX) return SSA_ERR_UNSUPPORTED;
  return SSA_OK;
}

ssa_status check_cache_attn(const ssa_cache_attn_params* p) {
  if (!p || p->n_q < 0 || p->h_q < 1 || p->topk < 0 || p->window < 0 || p->reserved != 0 || !isfinite(p->scale) ||
      !(p->scale > 0.f))
    return SSA_ERR_INVALID_ARG;
  const ssa_status st = check_cache(p->n_seq, p->max_pages, p->n_pages, p->page, p->h_kv, p->d);
  if (st != SSA_OK) return st;
  if (p->h_q % p->h_kv != 0 || (p->topk == 0) != (p->window == 0)) return SSA_ERR_INVALID_ARG;
  if (p->h_q / p->h_kv > 16 || p->topk > 32 || p->window > 4032) return SSA_ERR_UNSUPPORTED;
  // rows and blocks are counted in 32 bits (one product at a time: three would pass 64)
  const int64_t rows = static_cast<int64_t>(p->n_q) * p->h_q;
  if (rows > (INT32_MAX >> 1) || rows * p->n_seq > (INT32_MAX >> 1)) return SSA_ERR_UNSUPPORTED;
  return SSA_OK;
}

ssa_status check_prompt(const ssa_prompt_params* p) {
  if (!p || p->n_seq < 0 || p->n_q < 0 || p->n_kv < 0 || p->h_q < 1 || p->h_kv < 1 || p->d < 1 || p->reserved != 0 ||
      !isfinite(p->scale) || !(p->scale > 0.f) || p->h_q % p->h_kv != 0)
    return SSA_ERR_INVALID_ARG;
  if ((p->d != 64 && p->d != 128) || p->h_q / p->h_kv > 16) return SSA_ERR_UNSUPPORTED;
  if (bad_stride(p->q_stride, p->h_q, p->d, 2) || bad_stride(p->k_stride, p->h_kv, p->d, 2) ||
      bad_stride(p->v_stride, p->h_kv, p->d, 2) || bad_stride(p->o_stride, p->h_q, p->d, 2))
    return SSA_ERR_INVALID_ARG;
  // tensor-map strides are below 2^40 bytes; the grid is counted in 32 bits
  const int64_t most = int64_t{1} << 38;
  if (p->q_stride > most || p->k_stride > most || p->v_stride > most) return SSA_ERR_UNSUPPORTED;
  if (p->n_seq > (1 << 24) || p->h_q > 65535 ||
      (static_cast<int64_t>(p->n_q) + p->n_seq) * p->h_kv > INT32_MAX)
    return SSA_ERR_UNSUPPORTED;
  return SSA_OK;
}

}  // namespace

extern "C" {

ssa_status ssa_rope_frequencies(int32_t schedule, int32_t rot, double base, double factor, double trained_len,
                                double fast, double slow, double* freq, float* mscale) {
  if (!freq || rot < 2 || rot % 2 != 0 || !isfinite(base) || !(base > 1.0) || !isfinite(factor) || !(factor >= 1.0) ||
      schedule < SSA_ROPE_PLAIN || schedule > SSA_ROPE_BLEND)
    return SSA_ERR_INVALID_ARG;
  if (schedule == SSA_ROPE_BASE && rot < 4) return SSA_ERR_INVALID_ARG;
  if (schedule == SSA_ROPE_BLEND &&
      !(isfinite(trained_len) && trained_len >= 1.0 && isfinite(fast) && slow > 0.0 && fast > slow))
    return SSA_ERR_INVALID_ARG;
  if (schedule == SSA_ROPE_BASE) base *= pow(factor, static_cast<double>(rot) / (rot - 2));
  double lo = 0.0, hi = 0.0;
  if (schedule == SSA_ROPE_BLEND) {
    const double two_pi = 6.283185307179586;
    const auto at = [&](double t) { return rot * log(trained_len / (two_pi * t)) / (2.0 * log(base)); };
    lo = fmin(fmax(floor(at(fast)), 0.0), rot - 1.0);
    hi = fmin(fmax(ceil(at(slow)), 0.0), rot - 1.0);
  }
  for (int i = 0; i < rot / 2; ++i) {
    double f = pow(base, -2.0 * i / rot);
    if (schedule == SSA_ROPE_LINEAR) f /= factor;
    if (schedule == SSA_ROPE_BLEND) {
      const double keep = 1.0 - fmin(fmax((i - lo) / fmax(hi - lo, 1e-3), 0.0), 1.0);
      f = f * keep + f / factor * (1.0 - keep);
    }
    freq[i] = f;
  }
  if (mscale) *mscale = schedule == SSA_ROPE_BLEND ? static_cast<float>(0.1 * log(factor) + 1.0) : 1.f;
  return SSA_OK;
}

ssa_status ssa_qk_rope(const ssa_rope_params* pp, const void* Q, const void* K, const float* q_weight,
                       const float* k_weight, const double* freq, const int32_t* positions, void* Q_out, void* K_out,
                       void* stream) {
  ssa_status st = check_rope(pp);
  if (st != SSA_OK) return st;
  const ssa_rope_params& p = *pp;
  if (p.n_tokens == 0) return SSA_OK;
  if (!Q || !K || !Q_out || !K_out || (p.rot > 0 && (!freq || !positions))) return SSA_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(Q_out, 16) || !aligned(K_out, 16) || !aligned(q_weight, 16) ||
      !aligned(k_weight, 16) || !aligned(freq, 16) || !aligned(positions, 4))
    return SSA_ERR_INVALID_ARG;
  // a token in place is read before it is written only at the same place
  if ((Q_out == Q && p.q_out_stride != p.q_stride) || (K_out == K && p.k_out_stride != p.k_stride))
    return SSA_ERR_INVALID_ARG;
  LaunchCtx c;
  if ((st = ssa::make_launch_ctx(stream, c)) != SSA_OK) return st;
  return from_cuda(ssa::launch_qk_rope(p, Q, K, q_weight, k_weight, freq, positions, Q_out, K_out, c));
}

ssa_status ssa_cache_append(const ssa_append_params* pp, const void* K, const void* V, const float* k_weight,
                            const double* freq, const int32_t* new_start, const int32_t* cached,
                            const int32_t* page_table, uint8_t* k_cache, uint8_t* v_cache, float* k_scale,
                            float* v_scale, int32_t* bad_count, void* stream) {
  ssa_status st = check_append(pp);
  if (st != SSA_OK) return st;
  const ssa_append_params& p = *pp;
  if (p.n_tokens == 0 || p.n_seq == 0) return SSA_OK;
  if (!K || !V || (p.rot > 0 && !freq) || !new_start || !cached || (p.max_pages > 0 && !page_table) ||
      (p.n_pages > 0 && (!k_cache || !v_cache || !k_scale || !v_scale)))
    return SSA_ERR_INVALID_ARG;
  if (!aligned(K, 16) || !aligned(V, 16) || !aligned(k_weight, 16) || !aligned(freq, 16) || !aligned(new_start, 4) ||
      !aligned(cached, 4) || !aligned(page_table, 4) || !aligned(k_cache, 16) || !aligned(v_cache, 16) ||
      !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(bad_count, 4))
    return SSA_ERR_INVALID_ARG;
  LaunchCtx c;
  if ((st = ssa::make_launch_ctx(stream, c)) != SSA_OK) return st;
  const ssa::AppendArgs a{K, V, k_weight, freq, new_start, cached, page_table, k_cache, v_cache, k_scale, v_scale, bad_count};
  return from_cuda(ssa::launch_cache_append(p, a, c));
}

size_t ssa_cache_attn_workspace_size(const ssa_cache_attn_params* p) {
  if (check_cache_attn(p) != SSA_OK) return 0;
  return ssa::cache_attn_ws(*p);
}

ssa_status ssa_cache_attn(const ssa_cache_attn_params* pp, const void* Q, const int32_t* page_table,
                          const int32_t* kv_len, const uint8_t* k_cache, const uint8_t* v_cache, const float* k_scale,
                          const float* v_scale, const int32_t* block_idx, void* O, float* lse, int32_t* bad_count,
                          void* ws, size_t ws_bytes, void* stream) {
  ssa_status st = check_cache_attn(pp);
  if (st != SSA_OK) return st;
  const ssa_cache_attn_params& p = *pp;
  if (p.n_seq == 0 || p.n_q == 0) return SSA_OK;
  if (!Q || !kv_len || !O || (p.max_pages > 0 && !page_table) ||
      (p.n_pages > 0 && (!k_cache || !v_cache || !k_scale || !v_scale)) || (p.topk > 0 && !block_idx) ||
      (p.topk == 0 && block_idx))
    return SSA_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(page_table, 4) || !aligned(kv_len, 4) || !aligned(k_cache, 16) ||
      !aligned(v_cache, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(block_idx, 4) ||
      !aligned(O, 16) || !aligned(lse, 4) || !aligned(bad_count, 4))
    return SSA_ERR_INVALID_ARG;
  const size_t need = ssa::cache_attn_ws(p);
  if (need && (!ws || ws_bytes < need || !aligned(ws, 16))) return SSA_ERR_WORKSPACE;
  LaunchCtx c;
  if ((st = ssa::make_launch_ctx(stream, c)) != SSA_OK) return st;
  const ssa::CacheAttnArgs a{Q, page_table, kv_len, k_cache, v_cache, k_scale, v_scale, block_idx, O, lse, bad_count, ws};
  return from_cuda(ssa::launch_cache_attn(p, a, c));
}

ssa_status ssa_prompt_attn(const ssa_prompt_params* pp, const void* Q, const void* K, const void* V,
                           const int32_t* q_start, const int32_t* kv_start, void* O, float* lse, void* stream) {
  ssa_status st = check_prompt(pp);
  if (st != SSA_OK) return st;
  const ssa_prompt_params& p = *pp;
  if (p.n_seq == 0 || p.n_q == 0) return SSA_OK;
  if (!Q || (p.n_kv > 0 && (!K || !V)) || !q_start || !kv_start || !O) return SSA_ERR_INVALID_ARG;
  if (!aligned(Q, 16) || !aligned(K, 16) || !aligned(V, 16) || !aligned(q_start, 4) || !aligned(kv_start, 4) ||
      !aligned(O, 16) || !aligned(lse, 4))
    return SSA_ERR_INVALID_ARG;
  LaunchCtx c;
  if ((st = ssa::make_launch_ctx(stream, c)) != SSA_OK) return st;
  return from_cuda(ssa::launch_prompt_attn(p, Q, K, V, q_start, kv_start, O, lse, c));
}

}  // extern "C"
