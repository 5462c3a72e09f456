// Appending keys and values to the paged 8-bit cache, with the keys' norm and
// rotation on the way (rope.cuh, cache.cuh).
//
// The work is cut by pages: a unit is the new tokens of one sequence that fall
// in one page, and a unit's K or V of one kv-head is quantised as a whole,
// because its scale is the largest exponent among them.  Sequence s owns the
// unit numbers floor(new_start[s] / page) + 2 s and up; it touches at most
// floor(tokens / page) + 2 pages, so the ranges never meet, and a warp finds
// its sequence by a 32-way search without a pass over the lengths.
//
// A block takes one unit's K or V for a run of kv-heads.  With many tokens
// all its threads share a head's rows; with few (decode steps, drafts) each
// warp takes a head of its own, so that nothing waits at a barrier: a unit
// decides for itself, whatever the others hold.  (Chosen by the average, a long
// sequence among short ones was left to single warps: 43 us for 1024 tokens of
// 512 sequences, one of them with half of the tokens, now 28.)  At most one
// token per sequence on average takes a kernel of warps alone, in half the
// registers (512 sequences: 16 us in blocks, 11 so).  Bytes bound long prompts,
// launch and the chain of dependent index loads the rest.
#include <cuda_bf16.h>

#include <type_traits>

#include "cache.cuh"
#include "common.cuh"
#include "kernels.h"
#include "rope.cuh"

namespace ssa {
namespace {

constexpr int kKeep = 4;   // rows of a page per thread
// Heads on their way or in use, in stages of 16 bytes (bf16) per row and thread.
template <typename T>
__host__ __device__ constexpr int page_stages() { return sizeof(T) == 2 ? 4 : 2; }

struct AppendCfg {
  AppendArgs g;
  int64_t k_stride, v_stride;
  int32_t n_tokens, n_seq, max_pages, n_pages, h_kv, rot, layout, norm;
  int32_t n_units;
  int32_t runs, per_run;   // runs of kv-heads per unit, kv-heads per run
  float eps, mscale;
};

struct AppendUnit {
  int32_t t0, n;       // new tokens (rows of K and V)
  int32_t slot0;       // slot of the first
  int32_t pos0;        // its position
  int32_t seq, place;  // its sequence and its page's place there
};

// All lanes of the warp get the unit (n = 0: nothing to do); `count` (one
// caller per unit) adds what is left out to the bad counter.
template <int P>
__device__ __forceinline__ AppendUnit append_unit(const AppendCfg& a, int64_t unit, bool count) {
  const int lane = threadIdx.x & 31;
  AppendUnit u;
  u.n = 0;
  const auto start = [&](int s) { return min(max(__ldg(a.g.new_start + s), 0), a.n_tokens); };
  // the sequence is in [lo, hi): cut by 32 to at most 128, then all at once
  const auto before = [&](int s) { return start(s) / P + 2 * static_cast<int64_t>(s) <= unit; };
  int lo = 0, hi = a.n_seq;
  while (hi - lo > 128) {
    const int step = (hi - lo + 31) / 32;
    const int s = lo + lane * step;
    const int n = __popc(__ballot_sync(0xFFFFFFFFu, s < hi && before(s)));
    if (n == 0) return u;
    lo += (n - 1) * step;
    hi = min(hi, lo + step);
  }
  int n = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const int s = lo + 32 * k + lane;
    n += s < hi && before(s) ? 1 : 0;
  }
  n = static_cast<int>(__reduce_add_sync(0xFFFFFFFFu, static_cast<uint32_t>(n)));
  if (n == 0) return u;
  lo += n - 1;
  const int a0 = start(lo), a1 = max(start(lo + 1), a0);
  const int64_t j = unit - (a0 / P + 2 * static_cast<int64_t>(lo));
  const int have = __ldg(a.g.cached + lo);
  if (j < 0 || a1 == a0) return u;
  if (have < 0) {
    if (count && j == 0 && lane == 0 && a.g.bad) atomicAdd(a.g.bad, a1 - a0);
    return u;
  }
  const int64_t pi = have / P + j;
  const int64_t p0 = max(static_cast<int64_t>(have), pi * P);
  const int64_t p1 = min(static_cast<int64_t>(have) + (a1 - a0), (pi + 1) * P);
  if (p1 <= p0) return u;
  u.n = static_cast<int>(p1 - p0);
  u.t0 = a0 + static_cast<int>(p0 - have);
  u.slot0 = static_cast<int>(p0 - pi * P);
  u.pos0 = static_cast<int>(p0);
  u.seq = lo;
  u.place = pi < a.max_pages ? static_cast<int>(pi) : -1;
  return u;
}

// The unit's page in the pool, -1 when it has none.
__device__ __forceinline__ int unit_page(const AppendCfg& a, const AppendUnit& u, bool count) {
  const int page = u.place >= 0 ? __ldg(a.g.table + static_cast<int64_t>(u.seq) * a.max_pages + u.place) : -1;
  if (page >= 0 && page < a.n_pages) return page;
  if (count && (threadIdx.x & 31) == 0 && a.g.bad) atomicAdd(a.g.bad, u.n);
  return -1;
}

__device__ __forceinline__ float row_amax(const float (&x)[8]) {
  float r = fabsf(x[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) r = fmaxf(r, fabsf(x[i]));
  return r;
}

// The largest finite |x| * f of a row's elements and m (fmaxf leaves NaN out).
__device__ __forceinline__ float finite_amax(const float (&x)[8], float f, float m) {
  float r = row_amax(x) * f;
  if (!(r < INFINITY)) {   // among them an infinity (or all NaN): one by one
    r = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (fabsf(x[i]) * f < INFINITY) r = fmaxf(r, fabsf(x[i]) * f);
  }
  return fmaxf(m, r);
}

__device__ __forceinline__ void store_codes(uint8_t* row, const LaneDims& at, float (&x)[8], float inv) {
  scale_row(x, inv);
  *reinterpret_cast<uint32_t*>(row + at.a) = to_e4m3x2(x[0], x[1]) | to_e4m3x2(x[2], x[3]) << 16;
  *reinterpret_cast<uint32_t*>(row + at.b) = to_e4m3x2(x[4], x[5]) | to_e4m3x2(x[6], x[7]) << 16;
}

// Rounds 16 codes again to a scale 2^-down times coarser.
__device__ __forceinline__ void round_again(uint8_t* p, float down) {
  uint4 v = *reinterpret_cast<uint4*>(p);
  uint32_t* w = reinterpret_cast<uint32_t*>(&v);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    uint32_t out = 0;
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const uint32_t hb = e4m3x2_to_half2(w[i] >> (16 * k) & 0xFFFFu);
      const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&hb));
      out |= to_e4m3x2(f.x * down, f.y * down) << (16 * k);
    }
    w[i] = out;
  }
  *reinterpret_cast<uint4*>(p) = v;
}

// One row's eight dims of this lane in float32: the key weighted and rotated,
// the value as it is.  Returns the norm's factor, which the caller applies
// to the row's maximum and, with the page's scale, to its codes: one product
// per element for both.
template <typename T, int LPR>
__device__ __forceinline__ float append_row(const AppendCfg& a, bool is_k, const Row8<T>& r, const LaneDims& at,
                                            const float (&w)[8], const Angles& g, float (&x)[8]) {
  r.get(x);
  if (!is_k) return 1.f;
  const float f = a.norm ? norm_factor<LPR>(x, a.eps) : 1.f;
  scale_row(x, w);
  g.turn(at, x);
  return f;
}

// The page's exponent, and the rounding of what it held when that grows.
template <int D>
__device__ __forceinline__ int page_exponent(const AppendUnit& u, float amax, float old, uint8_t* codes, int thread,
                                             int threads) {
  const int e_new = scale_exponent(amax);
  if (u.slot0 == 0) return e_new;
  const int e_old = exponent_of(old);
  if (e_new <= e_old) return e_old;
  const float down = pow2(e_old - e_new);
  for (int i = thread; i < u.slot0 * (D / 16); i += threads) round_again(codes + i * 16, down);
  return e_new;
}

// A thread's eight dims of one row, global to its own place in shared memory.
template <typename T>
__device__ __forceinline__ void copy_row8(Run4<T>* a, Run4<T>* b, const T* row, const LaneDims& at) {
  if (sizeof(T) == 2) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(a)), "l"(row + at.a) : "memory");
    asm volatile("cp.async.ca.shared.global [%0], [%1], 8;" ::"r"(smem_u32(b)), "l"(row + at.b) : "memory");
  } else {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(a)), "l"(row + at.a) : "memory");
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(b)), "l"(row + at.b) : "memory");
  }
}

// One head of a unit of few tokens, by a warp: the rows stay in registers
// between the maximum and the rounding.
template <typename T, int D, int P>
__device__ __forceinline__ void append_head(const AppendCfg& a, const AppendUnit& u, bool is_k, int head, int page,
                                            const LaneDims& at, const float (&w)[8], const uint64_t (&phase)[4]) {
  constexpr int LPR = D / 8, RPW = 32 / LPR, F = kKeep;
  const int lane = threadIdx.x & 31, row = lane / LPR;
  const int64_t stride = is_k ? a.k_stride : a.v_stride;
  const T* src = static_cast<const T*>(is_k ? a.g.K : a.g.V) + u.t0 * stride + static_cast<int64_t>(head) * D;
  Row8<T> r[F];
#pragma unroll
  for (int k = 0; k < F; ++k)   // rows past the last repeat it: the same maximum
    if (k * RPW < u.n) r[k].load(src + min(k * RPW + row, u.n - 1) * stride, at);
  const int64_t ph = static_cast<int64_t>(page) * a.h_kv + head;
  uint8_t* codes = (is_k ? a.g.kc : a.g.vc) + ph * (P * D);
  float* scale = (is_k ? a.g.ks : a.g.vs) + ph;
  const float old = u.slot0 > 0 ? *scale : 0.f;
  float x[F][8], f[F], amax = 0.f;
#pragma unroll
  for (int k = 0; k < F; ++k) {
    if (k * RPW >= u.n) continue;   // the same for the warp
    Angles g;
    if (is_k) g.set<sizeof(T) == 4>(at, phase, u.pos0 + min(k * RPW + row, u.n - 1), a.mscale);
    f[k] = append_row<T, LPR>(a, is_k, r[k], at, w, g, x[k]);
    amax = finite_amax(x[k], f[k], amax);
  }
  amax = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax)));   // both orders agree from 0 up
  const int e = page_exponent<D>(u, amax, old, codes, lane, 32);
  const float inv = pow2(-e);
#pragma unroll
  for (int k = 0; k < F; ++k)
    if (k * RPW + row < u.n) store_codes(codes + (u.slot0 + k * RPW + row) * D, at, x[k], f[k] * inv);
  __syncwarp();   // every lane has read the old scale
  if (lane == 0) *scale = pow2(e);
}

// A block per (unit, K or V, run of kv-heads).  With many tokens: the unit is
// looked up and the angles are computed once for all the heads of the run; a
// head's rows stay in registers between the maximum and the rounding, and the
// next heads' are on their way to shared memory, each thread's to its own place
// (no barrier but the one of the maximum).  64K tokens of eight heads: a block per
// kv-head took 205 us, most of it the chain of index loads; the next head
// alone on its way 115 us, bound by the bytes in flight; now 92 us, 66% of the
// copy rate, at half of the issue slots with 16 warps per SM (registers; at d = 64
// four blocks of 128 threads for 16 warps: 67 us with two, 48 with four).
template <typename T, int D, int P>
__global__ void __launch_bounds__(P * D / 8 / kKeep, 512 / (P * D / 8 / kKeep)) append_kernel(const AppendCfg a) {
  constexpr int LPR = D / 8, KEEP = kKeep, THREADS = P * LPR / KEEP, ROWS = THREADS / LPR;
  constexpr int STAGES = page_stages<T>();
  __shared__ float red[2][THREADS / 32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, sub = lane % LPR;
  const int row = threadIdx.x / LPR;
  const bool is_k = (blockIdx.x & 1) == 0;   // keys take longer: the two kinds take turns
  const int item = static_cast<int>(blockIdx.x >> 1);
  const int h0 = item % a.runs * a.per_run, h1 = min(h0 + a.per_run, a.h_kv);
  const bool count = h0 == 0 && is_k && warp == 0;
  const AppendUnit u = append_unit<P>(a, item / a.runs, count);
  if (u.n == 0) return;
  const int64_t stride = is_k ? a.k_stride : a.v_stride;
  const LaneDims at(sub, is_k ? a.rot : 0, a.layout);
  if (u.n <= KEEP * (32 / LPR)) {   // the same for the block
    const int page = unit_page(a, u, count);
    if (page < 0) return;
    float w[8];
    uint64_t phase[4];
    lane_weights(is_k && a.norm ? a.g.k_weight : nullptr, at, w);
    at.warp_phases<D>(a.g.freq, is_k ? a.rot : 0, sub, phase);
    for (int h = h0 + warp; h < h1; h += THREADS / 32) append_head<T, D, P>(a, u, is_k, h, page, at, w, phase);
    return;
  }
  const T* src[KEEP];
#pragma unroll
  for (int k = 0; k < KEEP; ++k)   // rows past the last repeat it: the same maximum
    src[k] = static_cast<const T*>(is_k ? a.g.K : a.g.V) + (u.t0 + min(row + k * ROWS, u.n - 1)) * stride;
  extern __shared__ __align__(16) uint8_t ring_raw[];
  Run4<T>* ring = reinterpret_cast<Run4<T>*>(ring_raw) + threadIdx.x;   // [stages][KEEP][2][THREADS]
  const auto fetch = [&](int h) {   // a group per head, empty past the last
    if (h < h1) {
      Run4<T>* to = ring + (h % STAGES) * (KEEP * 2 * THREADS);
#pragma unroll
      for (int k = 0; k < KEEP; ++k)
        copy_row8(to + 2 * k * THREADS, to + (2 * k + 1) * THREADS, src[k] + static_cast<int64_t>(h) * D, at);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
#pragma unroll
  for (int s = 0; s < STAGES - 1; ++s) fetch(h0 + s);
  const int page = unit_page(a, u, count);   // looked up while the rows are on their way
  if (page < 0) {
    asm volatile("cp.async.wait_all;" ::: "memory");
    return;
  }
  float w[8];
  lane_weights(is_k && a.norm ? a.g.k_weight : nullptr, at, w);
  Angles angles[KEEP];
  if (is_k) {
    uint64_t phase[4];
    at.warp_phases<D>(a.g.freq, is_k ? a.rot : 0, sub, phase);
#pragma unroll
    for (int k = 0; k < KEEP; ++k)
      angles[k].set<sizeof(T) == 4>(at, phase, u.pos0 + min(row + k * ROWS, u.n - 1), a.mscale);
  }
  const int64_t ph = static_cast<int64_t>(page) * a.h_kv + h0;
  uint8_t* codes = (is_k ? a.g.kc : a.g.vc) + ph * (P * D);
  float* scale = (is_k ? a.g.ks : a.g.vs) + ph;
  // key: K, not V; whole: a full page, nothing to test
  const auto heads = [&](auto key, auto whole) {
    for (int h = h0; h < h1; ++h, codes += P * D, ++scale) {
      const float old = !whole && u.slot0 > 0 ? *scale : 0.f;
      fetch(h + STAGES - 1);
      asm volatile("cp.async.wait_group %0;" ::"n"(STAGES - 1) : "memory");
      const Run4<T>* from = ring + (h % STAGES) * (KEEP * 2 * THREADS);
      float x[KEEP][8], f[KEEP];
      float amax = 0.f;
#pragma unroll
      for (int k = 0; k < KEEP; ++k) {
        if (!whole && k * ROWS >= u.n) continue;   // the same for the block
        const Row8<T> r{from[2 * k * THREADS], from[(2 * k + 1) * THREADS]};
        f[k] = append_row<T, LPR>(a, key, r, at, w, angles[k], x[k]);
        amax = fmaxf(amax, row_amax(x[k]) * f[k]);   // fmaxf leaves NaN out
      }
      if (amax == INFINITY) {   // infinities are left out too: one by one
        amax = 0.f;
#pragma unroll
        for (int k = 0; k < KEEP; ++k)
          if (whole || k * ROWS < u.n) amax = finite_amax(x[k], f[k], amax);
      }
      amax = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax)));   // both orders agree from 0 up
      if (lane == 0) red[h & 1][warp] = amax;
      __syncthreads();   // the maxima are there, and every thread has the old scale
      amax = __uint_as_float(
          __reduce_max_sync(0xFFFFFFFFu, __float_as_uint(red[h & 1][lane % (THREADS / 32)])));
      const int e = page_exponent<D>(u, amax, old, codes, threadIdx.x, THREADS);
      const float inv = pow2(-e);
      uint8_t* to = codes + (u.slot0 + row) * D;
#pragma unroll
      for (int k = 0; k < KEEP; ++k)
        if (whole || row + k * ROWS < u.n) store_codes(to + k * ROWS * D, at, x[k], key ? f[k] * inv : inv);
      if (threadIdx.x == 0) *scale = pow2(e);
    }
  };
  if (u.n == P) {
    if (is_k) heads(std::true_type{}, std::true_type{});
    else heads(std::false_type{}, std::true_type{});
  } else {
    if (is_k) heads(std::true_type{}, std::false_type{});
    else heads(std::false_type{}, std::false_type{});
  }
}

// Decode steps, a token per sequence: a warp per (unit, kv-head, K or V), in half
// the registers.  More rows than one pass holds are read twice.
template <typename T, int D, int P>
__global__ void __launch_bounds__(256) append_few_kernel(const AppendCfg a) {
  constexpr int LPR = D / 8, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, sub = lane % LPR, row = lane / LPR;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * 8 + threadIdx.x / 32;
  const int64_t unit = item / (2 * a.h_kv);
  if (unit >= a.n_units) return;
  const int hk = static_cast<int>(item % (2 * a.h_kv));
  const bool is_k = hk < a.h_kv;
  const int head = is_k ? hk : hk - a.h_kv;
  const AppendUnit u = append_unit<P>(a, unit, hk == 0);
  if (u.n == 0) return;
  const int page = unit_page(a, u, hk == 0);
  if (page < 0) return;
  const int64_t stride = is_k ? a.k_stride : a.v_stride;
  const T* src = static_cast<const T*>(is_k ? a.g.K : a.g.V) + static_cast<int64_t>(u.t0) * stride +
                 static_cast<int64_t>(head) * D;
  const LaneDims at(sub, is_k ? a.rot : 0, a.layout);
  float w[8];
  uint64_t phase[4];
  lane_weights(is_k && a.norm ? a.g.k_weight : nullptr, at, w);
  at.warp_phases<D>(a.g.freq, is_k ? a.rot : 0, sub, phase);
  float x[8], f = 1.f;
  const auto value = [&](int i0) {
    const int i = min(i0 + row, u.n - 1);
    Row8<T> r;
    r.load(src + static_cast<int64_t>(i) * stride, at);
    Angles g;
    if (is_k) g.set<sizeof(T) == 4>(at, phase, u.pos0 + i, a.mscale);
    f = append_row<T, LPR>(a, is_k, r, at, w, g, x);
  };
  float amax = 0.f;
  for (int i0 = 0; i0 < u.n; i0 += RPW) {
    value(i0);
    amax = finite_amax(x, f, amax);
  }
  amax = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(amax)));   // both orders agree from 0 up
  const int64_t ph = static_cast<int64_t>(page) * a.h_kv + head;
  uint8_t* codes = (is_k ? a.g.kc : a.g.vc) + ph * (P * D);
  float* scale = (is_k ? a.g.ks : a.g.vs) + ph;
  const int e = page_exponent<D>(u, amax, u.slot0 > 0 ? *scale : 0.f, codes, lane, 32);
  const float inv = pow2(-e);
  for (int i0 = 0; i0 < u.n; i0 += RPW) {
    if (u.n > RPW) value(i0);
    if (i0 + row < u.n) store_codes(codes + (u.slot0 + i0 + row) * D, at, x, f * inv);
  }
  __syncwarp();
  if (lane == 0) *scale = pow2(e);
}

template <typename T, int D, int P>
cudaError_t run_append(AppendCfg a, const LaunchCtx& c) {
  const int64_t units = a.n_tokens / P + 2 * static_cast<int64_t>(a.n_seq);   // below 2^27, times h_kv below 2^31
  a.n_units = static_cast<int32_t>(units);
  if (a.n_tokens <= a.n_seq) {
    append_few_kernel<T, D, P><<<static_cast<unsigned>((units * 2 * a.h_kv + 7) / 8), 256, 0, c.stream>>>(a);
    note_launch();
    return cudaGetLastError();
  }
  // All kv-heads in one run where the units alone give every SM two blocks,
  // else as many runs as that takes (more rounds of shorter blocks: 64
  // sequences of five drafts 11.4 us at four rounds, 10.7 at one).
  constexpr int kThreads = P * D / 8 / kKeep, kSmem = page_stages<T>() * kKeep * kThreads * 8 * sizeof(T);
  int64_t runs = (2 * static_cast<int64_t>(c.sm_count) + 2 * units - 1) / (2 * units);
  if (runs > a.h_kv) runs = a.h_kv;
  a.per_run = static_cast<int32_t>((a.h_kv + runs - 1) / runs);
  a.runs = (a.h_kv + a.per_run - 1) / a.per_run;
  const int64_t grid = units * a.runs * 2;   // several runs only with fewer units than SMs
  const cudaError_t e = cudaFuncSetAttribute(append_kernel<T, D, P>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  if (e != cudaSuccess) return e;
  append_kernel<T, D, P><<<static_cast<unsigned>(grid), kThreads, kSmem, c.stream>>>(a);
  note_launch();
  return cudaGetLastError();
}

template <typename T>
cudaError_t pick_append(const ssa_append_params& p, const AppendCfg& a, const LaunchCtx& c) {
  if (p.d == 128) return p.page == 64 ? run_append<T, 128, 64>(a, c) : run_append<T, 128, 128>(a, c);
  return p.page == 64 ? run_append<T, 64, 64>(a, c) : run_append<T, 64, 128>(a, c);
}

}  // namespace

cudaError_t launch_cache_append(const ssa_append_params& p, const AppendArgs& g, const LaunchCtx& c) {
  AppendCfg a{};
  a.g = g;
  a.k_stride = p.k_stride; a.v_stride = p.v_stride;
  a.n_tokens = p.n_tokens; a.n_seq = p.n_seq; a.max_pages = p.max_pages; a.n_pages = p.n_pages;
  a.h_kv = p.h_kv; a.rot = p.rot; a.layout = p.layout; a.norm = p.norm;
  a.eps = p.eps; a.mscale = p.mscale;
  return p.dtype == SSA_BF16 ? pick_append<__nv_bfloat16>(p, a, c) : pick_append<float>(p, a, c);
}

}  // namespace ssa
