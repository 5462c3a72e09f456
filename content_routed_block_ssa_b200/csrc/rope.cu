// Norms of queries and keys per head and their position rotation, one pass
// (rope.cuh has the mathematics).
//
// A warp takes one token and a run of its heads (queries, then keys): 32/LPR
// heads at a time, LPR = d/8 lanes of eight dims each, so a head is read and
// written in 16-byte pieces and its norm is a few shuffles.  The angles of a
// token are computed once per lane and used for all the heads of the run.
// Bytes bound it: each element is read once and written once.
#include <cuda_bf16.h>

#include "kernels.h"
#include "rope.cuh"

namespace ssa {
namespace {

struct RopeArgs {
  const void *Q, *K;
  void *Qo, *Ko;
  const float *qw, *kw;
  const double* freq;
  const int32_t* pos;
  int64_t qs, ks, qos, kos;
  int32_t n_tokens, h_q, h_kv, rot, layout, norm;
  int32_t runs, per_run;   // runs of heads per token, head groups per run
  float eps, mscale;
};

template <typename T, int D>
__global__ void __launch_bounds__(256) rope_kernel(const RopeArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;   // lanes per head, heads per warp
  constexpr int U = 4;                         // head groups in flight
  constexpr bool PRECISE = sizeof(T) == 4;
  const int lane = threadIdx.x & 31, sub = lane % LPR, hr = lane / LPR;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * (blockDim.x / 32) + threadIdx.x / 32;
  const int64_t token = item / a.runs;
  if (token >= a.n_tokens) return;
  const int run = static_cast<int>(item % a.runs);
  const int heads = a.h_q + a.h_kv;
  const int h_end = min(heads, (run + 1) * a.per_run * RPW);

  uint64_t phase[8];
  Turn<PRECISE> turn;
  lane_phases(a.freq, sub, a.rot, a.layout, phase);
  turn.set(phase, sub, a.rot, a.layout, a.rot > 0 ? __ldg(a.pos + token) : 0, a.mscale);
  float qw[8], kw[8];
  lane_weights(a.qw, sub, qw);
  lane_weights(a.kw, sub, kw);
  const T* Q = static_cast<const T*>(a.Q) + token * a.qs + 8 * sub;
  const T* K = static_cast<const T*>(a.K) + token * a.ks + 8 * sub;
  T* Qo = static_cast<T*>(a.Qo) + token * a.qos + 8 * sub;
  T* Ko = static_cast<T*>(a.Ko) + token * a.kos + 8 * sub;

  for (int h0 = run * a.per_run * RPW; h0 < h_end; h0 += U * RPW) {
    Row8<T> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int h = min(h0 + u * RPW + hr, heads - 1);
      r[u].load(h < a.h_q ? Q + static_cast<int64_t>(h) * D : K + static_cast<int64_t>(h - a.h_q) * D);
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (h0 + u * RPW >= h_end) break;   // the same for the whole warp
      const int h = h0 + u * RPW + hr;
      float x[8];
      r[u].get(x);
      if (a.norm) {
        float w[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) w[i] = h < a.h_q ? qw[i] : kw[i];
        norm_row<LPR>(x, w, a.eps);
      }
      turn.apply(x, a.layout, lane, 8 * sub < a.rot);
      if (h < h_end) {
        if (h < a.h_q) Row8<T>::store(Qo + static_cast<int64_t>(h) * D, x);
        else Row8<T>::store(Ko + static_cast<int64_t>(h - a.h_q) * D, x);
      }
    }
  }
}

template <typename T, int D>
cudaError_t run_rope(RopeArgs a, const LaunchCtx& c) {
  constexpr int RPW = 32 / (D / 8);
  const int groups = (a.h_q + a.h_kv + RPW - 1) / RPW;
  // enough warps to fill the GPU (16 per SM) from few tokens, else all the
  // heads of a token in one run; never less than one group per run
  const int64_t want = static_cast<int64_t>(c.sm_count) * 16;
  int64_t runs = (want + a.n_tokens - 1) / a.n_tokens;
  if (runs > groups) runs = groups;
  a.per_run = static_cast<int32_t>((groups + runs - 1) / runs);
  a.runs = (groups + a.per_run - 1) / a.per_run;
  const int64_t items = static_cast<int64_t>(a.n_tokens) * a.runs;
  const int64_t grid = (items + 7) / 8;
  if (grid > 2147483647) return cudaErrorInvalidValue;
  rope_kernel<T, D><<<static_cast<unsigned>(grid), 256, 0, c.stream>>>(a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_qk_rope(const ssa_rope_params& p, const void* Q, const void* K, const float* qw, const float* kw,
                           const double* freq, const int32_t* positions, void* Qo, void* Ko, const LaunchCtx& c) {
  RopeArgs a{};
  a.Q = Q; a.K = K; a.Qo = Qo; a.Ko = Ko;
  a.qw = p.norm ? qw : nullptr;
  a.kw = p.norm ? kw : nullptr;
  a.freq = freq; a.pos = positions;
  a.qs = p.q_stride; a.ks = p.k_stride; a.qos = p.q_out_stride; a.kos = p.k_out_stride;
  a.n_tokens = p.n_tokens; a.h_q = p.h_q; a.h_kv = p.h_kv;
  a.rot = p.rot; a.layout = p.layout; a.norm = p.norm;
  a.eps = p.eps; a.mscale = p.mscale;
  if (p.dtype == SSA_BF16) return p.d == 128 ? run_rope<__nv_bfloat16, 128>(a, c) : run_rope<__nv_bfloat16, 64>(a, c);
  return p.d == 128 ? run_rope<float, 128>(a, c) : run_rope<float, 64>(a, c);
}

}  // namespace ssa
