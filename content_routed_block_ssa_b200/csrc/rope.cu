// Norms of queries and keys per head and their position rotation, one pass
// (rope.cuh has the mathematics).
//
// A warp takes one token and a run of its heads (queries, then keys): 32/LPR
// heads at a time, LPR = d/8 lanes of eight dims each, so that a head is read
// and written whole and its norm is a few shuffles.  The angles of a token are
// computed once per lane, folded with the weights, and used for all the heads
// of the run; with many tokens a warp goes on to the next token and keeps its
// frequencies.  Bytes bound it: each element is read once and written once.
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

// The heads g * RPW + hr, g in [g0, g1), of one of the two operands.
template <typename T, int D>
__device__ __forceinline__ void rope_heads(const T* in, T* out, int heads, int g0, int g1, const float* weight,
                                           const LaneDims& at, const Angles& angles, const RopeArgs& a, int hr) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  constexpr int U = 4;   // head groups in flight
  float w[8];
  lane_weights(weight, at, w);
  Turn turn;
  turn.set(at, angles, w);
  for (int g = g0; g < g1; g += U) {
    Row8<T> r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u].load(in + static_cast<int64_t>(min((g + u) * RPW + hr, heads - 1)) * D, at);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (g + u >= g1) break;   // the same for the whole warp
      const int h = (g + u) * RPW + hr;
      float x[8], y[8];
      r[u].get(x);
      const float f = a.norm ? norm_factor<LPR>(x, a.eps) : 1.f;
      turn.apply(at, x, f, y);
      if (h < heads) Row8<T>::store(out + static_cast<int64_t>(h) * D, at, y);
    }
  }
}

template <typename T, int D>
__global__ void __launch_bounds__(256, sizeof(T) == 2 ? 4 : 3) rope_kernel(const RopeArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;   // lanes per head, heads per warp
  const int lane = threadIdx.x & 31, sub = lane % LPR, hr = lane / LPR;
  const int gq = (a.h_q + RPW - 1) / RPW, gk = (a.h_kv + RPW - 1) / RPW;
  const LaneDims at(sub, a.rot, a.layout);
  uint64_t phase[4];
  at.phases(a.freq, sub, phase);
  const int64_t items = static_cast<int64_t>(a.n_tokens) * a.runs;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; item < items;
       item += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t token = item / a.runs;
    const int g0 = static_cast<int>(item % a.runs) * a.per_run, g1 = min(g0 + a.per_run, gq + gk);
    Angles angles;
    angles.set<sizeof(T) == 4>(at, phase, a.rot > 0 ? __ldg(a.pos + token) : 0, a.mscale);
    if (g0 < gq)
      rope_heads<T, D>(static_cast<const T*>(a.Q) + token * a.qs, static_cast<T*>(a.Qo) + token * a.qos, a.h_q, g0,
                       min(g1, gq), a.qw, at, angles, a, hr);
    if (g1 > gq)
      rope_heads<T, D>(static_cast<const T*>(a.K) + token * a.ks, static_cast<T*>(a.Ko) + token * a.kos, a.h_kv,
                       max(g0 - gq, 0), g1 - gq, a.kw, at, angles, a, hr);
  }
}

template <typename T, int D>
cudaError_t run_rope(RopeArgs a, const LaunchCtx& c) {
  constexpr int RPW = 32 / (D / 8);
  const int groups = (a.h_q + RPW - 1) / RPW + (a.h_kv + RPW - 1) / RPW;
  // enough warps to fill the GPU (16 per SM) from few tokens, else all the
  // heads of a token in one run; never less than one group per run
  const int64_t want = static_cast<int64_t>(c.sm_count) * 16;
  int64_t runs = (want + a.n_tokens - 1) / a.n_tokens;
  if (runs > groups) runs = groups;
  a.per_run = static_cast<int32_t>((groups + runs - 1) / runs);
  a.runs = (groups + a.per_run - 1) / a.per_run;
  const int64_t items = static_cast<int64_t>(a.n_tokens) * a.runs;
  const int64_t most = static_cast<int64_t>(c.sm_count) * (sizeof(T) == 2 ? 4 : 3);   // blocks that run at a time
  const int64_t grid = (items + 7) / 8 < most ? (items + 7) / 8 : most;
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
