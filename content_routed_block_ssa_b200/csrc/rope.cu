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
// loads ahead (128K tokens of 40 heads, d = 128, bf16: 447 to 450 us, 91% of the
// copy rate; straight from registers 508 at best); with few, the heads of a
// token are spread over several warps that load straight to registers, which
// starts sooner.
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
  int32_t even;            // pieces dealt out evenly to the warps, not tokens
  float eps, mscale;
  uint32_t* err;
};

constexpr int kGroups = 2;   // head groups in flight per warp
constexpr int kDirect = 3;   // blocks per SM

// An item is a run of a token's head groups (RPW heads each, those of the
// queries first).  The first groups' loads start before the angles are computed.
template <typename T, int D>
__global__ void __launch_bounds__(256, kDirect) rope_kernel(const RopeArgs a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, U = kGroups;   // lanes per head, heads per warp
  const int lane = threadIdx.x & 31, sub = lane % LPR, hr = lane / LPR;
  const int gq = (a.h_q + RPW - 1) / RPW, gk = (a.h_kv + RPW - 1) / RPW;
  const LaneDims at(sub, a.rot, a.layout);
  uint64_t phase[4];
  // float64 arithmetic is slow here: once per block or warp, not once per lane
  // (5003 float32 tokens: 12.3 us per lane, 11.1 per block; per warp 12.3, by spills)
  if constexpr (sizeof(T) == 4) {
    __shared__ __align__(16) uint64_t all[64];
    at.block_phases(a.freq, a.rot, all, sub, phase);
  } else {
    at.warp_phases<D>(a.freq, a.rot, sub, phase);
  }
  const int64_t items = static_cast<int64_t>(a.n_tokens) * a.runs;
  for (int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32; item < items;
       item += static_cast<int64_t>(gridDim.x) * 8) {
    const int64_t token = item / a.runs;
    const int g0 = static_cast<int>(item % a.runs) * a.per_run, g1 = min(g0 + a.per_run, gq + gk);
    const T* q = static_cast<const T*>(a.Q) + token * a.qs;
    const T* k = static_cast<const T*>(a.K) + token * a.ks;
    Row8<T> r[U];
    const auto load = [&](int g) {   // U groups from g on, heads past the last repeat it
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int x = min(g + u, g1 - 1);
        r[u].load(x < gq ? q + static_cast<int64_t>(min(x * RPW + hr, a.h_q - 1)) * D
                         : k + static_cast<int64_t>(min((x - gq) * RPW + hr, a.h_kv - 1)) * D,
                  at);
      }
    };
    const int32_t pos = a.rot > 0 ? __ldg(a.pos + token) : 0;
    load(g0);
    Angles angles;
    angles.set<sizeof(T) == 4>(at, phase, pos, a.mscale);
    for (int g = g0; g < g1; g += U) {
      if (g > g0) load(g);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (g + u >= g1) break;   // the same for the whole warp
        const bool is_q = g + u < gq;
        const int h = (is_q ? g + u : g + u - gq) * RPW + hr;
        float x[8], w[8];
        r[u].get(x);
        const float f = a.norm ? norm_factor<LPR>(x, a.eps) : 1.f;
        const float* weight = is_q ? a.qw : a.kw;
        if (weight) {   // from the cache: registers go to the loads
          lane_weights(weight, at, w);
          scale_row(x, w);
        }
        angles.turn(at, x);
        scale_row(x, f);
        if (h < (is_q ? a.h_q : a.h_kv))
          Row8<T>::store((is_q ? static_cast<T*>(a.Qo) + token * a.qos : static_cast<T*>(a.Ko) + token * a.kos) +
                             static_cast<int64_t>(h) * D,
                         at, x);
      }
    }
  }
}

constexpr int kEvenBelow = 4;    // tokens per warp
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
  at.warp_phases<D>(a.freq, a.rot, sub, phase);
  float qw[8], kw[8];
  lane_weights(a.qw, at, qw);
  lane_weights(a.kw, at, kw);

  // A token has `cq` pieces of queries and `ck` of keys.  With several tokens
  // per warp every tokens-th is this warp's, whole; with fewer (a.even) the
  // pieces are dealt out evenly, in runs.
  const int cq = (a.h_q + CH - 1) / CH, ck = (a.h_kv + CH - 1) / CH, per = cq + ck;
  const int first = blockIdx.x * kStreamWarps + warp, every = gridDim.x * kStreamWarps;
  const int step = a.even ? 1 : every;
  struct Place {   // piece c of a token, and how many are left from it on
    int64_t token;
    int c;
    int32_t left;   // (a piece holds at least 128 bytes)
    __device__ __forceinline__ void next(int per, int step) {
      --left;
      if (++c == per) { c = 0; token += step; }
    }
  };
  const auto heads_of = [&](const Place& w) {
    return w.c < cq ? min(CH, a.h_q - w.c * CH) : min(CH, a.h_kv - (w.c - cq) * CH);
  };
  const auto load = [&](const Place& w, int stage) {
    if (w.left <= 0) return;
    if (lane == 0) {
      const T* src = w.c < cq ? static_cast<const T*>(a.Q) + w.token * a.qs + static_cast<int64_t>(w.c) * (CH * D)
                              : static_cast<const T*>(a.K) + w.token * a.ks + static_cast<int64_t>(w.c - cq) * (CH * D);
      const uint32_t bytes = heads_of(w) * (D * sizeof(T));
      mbar_arrive_expect_tx(&full[stage], bytes);
      bulk_load(ring + stage * kStageBytes, src, bytes, &full[stage]);
    }
  };
  Place now{first, 0, first < a.n_tokens ? ((a.n_tokens - 1 - first) / every + 1) * per : 0};
  if (a.even) {
    const int64_t all = static_cast<int64_t>(a.n_tokens) * per, p0 = all * first / every;
    now = Place{p0 / per, static_cast<int>(p0 % per), static_cast<int32_t>(all * (first + 1) / every - p0)};
  }
  Place ahead = now;
  load(ahead, 0);
  ahead.next(per, step);
  load(ahead, 1);
  ahead.next(per, step);
  int32_t pos = a.rot > 0 && now.left > 0 ? __ldg(a.pos + now.token) : 0;
  Angles angles;
  bool turned = false;   // `angles` are the token's
  uint32_t parity = 0;   // a bit per stage
  int stage = 0;
  bool ok = true;
  for (; now.left > 0; now.next(per, step)) {
    // the load two pieces ahead takes the stage of two pieces ago, whose
    // store has been read out once at most the last one is pending
    asm volatile("cp.async.bulk.wait_group.read 1;" ::: "memory");
    __syncwarp();
    load(ahead, (stage + 2) % kStages);
    ahead.next(per, step);
    if (now.c == 0 || !turned) {
      turned = true;
      angles.set<sizeof(T) == 4>(at, phase, pos, a.mscale);
      const int64_t next = now.token + step;
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
  // Bulk copies pay from two pieces per warp on (2000 tokens of 40 heads, d = 128,
  // bf16: 15.7 us straight, 11.5 streamed), from three where a token has only
  // one or two, since each run of a token computes its angles (4000 tokens of 16
  // heads, d = 64, bf16, 2.3 pieces per warp: 7.4 and 8.4 us).
  constexpr int CH = kStageBytes / (D * static_cast<int>(sizeof(T)));
  const int per = (a.h_q + CH - 1) / CH + (a.h_kv + CH - 1) / CH;   // pieces per token
  const int64_t warps = static_cast<int64_t>(c.sm_count) * kStreamWarps;
  if (static_cast<int64_t>(a.n_tokens) * per >= (per > 2 ? 2 : 3) * warps) {
    const cudaError_t e =
        cudaFuncSetAttribute(rope_stream_kernel<T, D>, cudaFuncAttributeMaxDynamicSharedMemorySize, kStreamSmem);
    if (e != cudaSuccess) return e;
    // whole tokens per warp leave a round part empty, even runs of pieces do not
    // (4000 tokens of 40 heads: 26.7 and 18.1 us); but with many the runs are slower
    // (32000: 110 and 126 us)
    a.even = a.n_tokens < kEvenBelow * warps;
    rope_stream_kernel<T, D><<<c.sm_count, kStreamWarps * 32, kStreamSmem, c.stream>>>(a);
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
  const int64_t most = static_cast<int64_t>(c.sm_count) * kDirect;   // blocks that run at a time
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
