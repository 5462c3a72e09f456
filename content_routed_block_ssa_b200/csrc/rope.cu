// Norms of queries and keys per head and their position rotation, one pass
// (rope.cuh has the mathematics).
//
// A warp takes 32/LPR heads at a time, LPR = d/8 lanes of eight dims each, so
// that a head is read and written whole and its norm is a few shuffles.  The
// angles of a token are computed once per lane and used for all its heads.
// Bytes bound it: each element is read once and written once.
//
// Two kernels (see run_rope): with many tokens each warp streams pieces of 2 KB
// of neighbouring heads through shared memory by bulk copies, in and out, two
// loads ahead (128K tokens of 40 heads, d = 128, bf16: 449 to 457 us, 90% of the
// copy rate; straight from registers 508 at best); with few, the heads of a
// token are spread over several warps that load straight to registers, which
// starts sooner (5003 tokens of 16 heads, d = 64, float32: 12.3 us, streamed 16.3).
#include <cuda_bf16.h>

#include "common.cuh"
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
  uint32_t* err;
};

// The heads g * RPW + hr, g in [g0, g1), of one of the two operands.
template <typename T, int D>
__device__ __forceinline__ void rope_heads(const T* in, T* out, int heads, int g0, int g1, const float* weight,
                                           const LaneDims& at, const Angles& angles, const RopeArgs& a, int hr) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  constexpr int U = 2;   // head groups in flight
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

constexpr int kStreamFrom = 4;   // pieces per warp
constexpr int kStreamWarps = 24, kStages = 4, kStageBytes = 2048;
constexpr int kStreamSmem = kStreamWarps * kStages * (kStageBytes + 8);

template <typename T, int D>
__global__ void __launch_bounds__(kStreamWarps * 32, 1) rope_stream_kernel(const RopeArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  constexpr int CH = kStageBytes / (D * static_cast<int>(sizeof(T)));   // heads per piece
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, sub = lane % LPR, hr = lane / LPR;
  uint8_t* ring = smem + warp * (kStages * kStageBytes);
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStreamWarps * kStages * kStageBytes) + warp * kStages;
  if (lane == 0)
#pragma unroll
    for (int s = 0; s < kStages; ++s) mbar_init(&full[s], 1);
  fence_barrier_init();
  __syncwarp();

  const LaneDims at(sub, a.rot, a.layout);
  uint64_t phase[4];
  at.phases(a.freq, sub, phase);
  float qw[8], kw[8];
  lane_weights(a.qw, at, qw);
  lane_weights(a.kw, at, kw);

  // this warp's tokens, `cq` pieces of queries and `ck` of keys each
  const int cq = (a.h_q + CH - 1) / CH, ck = (a.h_kv + CH - 1) / CH, per = cq + ck;
  const int first = blockIdx.x * kStreamWarps + warp, every = gridDim.x * kStreamWarps;
  struct Place {   // a piece: token first + k * every, piece c
    int64_t token;
    int c;
    __device__ __forceinline__ void next(int per, int every) {
      if (++c == per) { c = 0; token += every; }
    }
  };
  const auto heads_of = [&](const Place& w) {
    return w.c < cq ? min(CH, a.h_q - w.c * CH) : min(CH, a.h_kv - (w.c - cq) * CH);
  };
  const auto load = [&](const Place& w, int stage) {
    if (w.token >= a.n_tokens) return;
    if (lane == 0) {
      const T* src = w.c < cq ? static_cast<const T*>(a.Q) + w.token * a.qs + static_cast<int64_t>(w.c) * (CH * D)
                              : static_cast<const T*>(a.K) + w.token * a.ks + static_cast<int64_t>(w.c - cq) * (CH * D);
      const uint32_t bytes = heads_of(w) * (D * sizeof(T));
      mbar_arrive_expect_tx(&full[stage], bytes);
      bulk_load(ring + stage * kStageBytes, src, bytes, &full[stage]);
    }
  };
  Place now{first, 0}, ahead{first, 0};
  load(ahead, 0);
  ahead.next(per, every);
  load(ahead, 1);
  ahead.next(per, every);
  int32_t pos = a.rot > 0 && now.token < a.n_tokens ? __ldg(a.pos + now.token) : 0;
  Angles angles;
  uint32_t parity = 0;   // a bit per stage
  int stage = 0;
  bool ok = true;
  for (; now.token < a.n_tokens; now.next(per, every)) {
    // the load two pieces ahead takes the stage of two pieces ago, whose
    // store has been read out once at most the last one is pending
    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
    load(ahead, (stage + 2) % kStages);
    ahead.next(per, every);
    if (now.c == 0) {
      angles.set<sizeof(T) == 4>(at, phase, pos, a.mscale);
      const int64_t next = now.token + every;
      if (a.rot > 0 && next < a.n_tokens) pos = __ldg(a.pos + next);
    }
    const bool is_q = now.c < cq;
    const int heads = heads_of(now);
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = is_q ? qw[i] : kw[i];
    T* rows = reinterpret_cast<T*>(ring + stage * kStageBytes);
    ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[stage], parity >> stage & 1u, a.err, SITE_ROPE_FULL));
    if (!ok) break;
    parity ^= 1u << stage;
    const auto turn_rows = [&](int n) {   // n known for whole pieces: nothing to test
#pragma unroll
      for (int h0 = 0; h0 < CH; h0 += RPW) {
        if (h0 >= n) break;
        const int h = h0 + hr;
        T* row = rows + min(h, n - 1) * D;
        Row8<T> r;
        r.load(row, at);
        float x[8];
        r.get(x);
        const float f = a.norm ? norm_factor<LPR>(x, a.eps) : 1.f;
        scale_row(x, w);
        angles.turn(at, x);
        scale_row(x, f);
        if (h < n) Row8<T>::store(row, at, x);
      }
    };
    if (heads == CH) turn_rows(CH);
    else turn_rows(heads);
    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    __syncwarp();
    if (lane == 0) {
      T* dst = is_q ? static_cast<T*>(a.Qo) + now.token * a.qos + static_cast<int64_t>(now.c) * (CH * D)
                    : static_cast<T*>(a.Ko) + now.token * a.kos + static_cast<int64_t>(now.c - cq) * (CH * D);
      asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst),
                   "r"(smem_u32(rows)), "r"(static_cast<uint32_t>(heads * (D * sizeof(T))))
                   : "memory");
    }
    asm volatile("cp.async.bulk.commit_group;" ::: "memory");   // empty but in lane 0
    stage = (stage + 1) % kStages;
  }
  if (!ok && lane == 0) {   // a wait gave up: let the copies in flight land (this piece's and two more at most)
    const uint64_t t0 = global_timer_ns();
    for (int k = 0; k < 3; ++k) {
      const int s = (stage + k) % kStages;
      while (!mbar_try_wait(&full[s], parity >> s & 1u) && global_timer_ns() - t0 < kWaitLimitNs) {}
    }
  }
  asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory");
}

template <typename T, int D>
cudaError_t run_rope(RopeArgs a, const LaunchCtx& c) {
  constexpr int RPW = 32 / (D / 8);
  // Bulk copies pay from about four pieces per warp on.
  constexpr int CH = kStageBytes / (D * static_cast<int>(sizeof(T)));
  const int64_t pieces = static_cast<int64_t>(a.n_tokens) * ((a.h_q + CH - 1) / CH + (a.h_kv + CH - 1) / CH);
  if (pieces >= kStreamFrom * static_cast<int64_t>(c.sm_count) * kStreamWarps) {
    const cudaError_t e =
        cudaFuncSetAttribute(rope_stream_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem);
    if (e != cudaSuccess) return e;
    const int64_t blocks = (static_cast<int64_t>(a.n_tokens) + kStreamWarps - 1) / kStreamWarps;
    rope_stream_kernel<T, D><<<static_cast<unsigned>(blocks < c.sm_count ? blocks : c.sm_count), kStreamWarps * 32,
                               kStreamSmem, c.stream>>>(a);
    note_launch();
    return cudaGetLastError();
  }
  const int groups = (a.h_q + RPW - 1) / RPW + (a.h_kv + RPW - 1) / RPW;
  // enough warps to fill the GPU (40 per SM) from few tokens, else all the
  // heads of a token in one run; never less than one group per run
  const int64_t want = static_cast<int64_t>(c.sm_count) * 40;
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
  a.err = c.err;
  if (p.dtype == SSA_BF16) return p.d == 128 ? run_rope<__nv_bfloat16, 128>(a, c) : run_rope<__nv_bfloat16, 64>(a, c);
  return p.d == 128 ? run_rope<float, 128>(a, c) : run_rope<float, 64>(a, c);
}

}  // namespace ssa
