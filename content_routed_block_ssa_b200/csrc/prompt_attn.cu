// Causal attention over packed prompts of different lengths, grouped heads.
//
// A block takes one unit: two tensor-core tiles of 128 rows (or one, where that
// gives more blocks: see launch_prompt_attn), each of QT = 128 / G
// consecutive queries x the G query heads of one kv-head, so the
// keys and values of a kv-head are read once for its whole group.  Per step of
// 128 keys and tile: S = Q K^T (tcgen05, into tensor memory), a softmax of one
// row per thread, P = 2^(s - m) in bf16 over the S columns, O += P V with P
// as the A operand from tensor memory.  The two tiles take turns: while the
// softmax warps of one work, the tensor core runs the other's products.
//
// Per step and tile both products take 2 x 512 tensor-core clocks (d = 128)
// and the 128 x 128 exponentials 1024 clocks of the four special-function
// units: the two bound each other, which is why everything else of the softmax
// is kept short: one thread owns a row (no shuffles), packed float32 pairs,
// and the output is rescaled only when a row's maximum has grown by more
// than 2^8 (any reference gives the same ratios, and 2^8 leaves the sums and
// the bf16 probabilities far from overflow).
//
// A prompt of 16384 (eight heads on one, d = 128) takes 494 to 508 us, 1.1
// PFLOP/s, at the power cap (990 W, 1.77 GHz); without the softmax the loads,
// products and barriers alone take 361 us, and the exponentials 74 us of the
// rest: the chain of one tile (S, softmax, P V) is longer than two tiles hide.
//
// Units are numbered by the packed query rows (floor(q_start / rows) + s and
// up: sequence ranges never meet); the grid starts at the last ones, whose
// causal prefix is the longest.
#include <cuda_bf16.h>
#include <math.h>

#include "common.cuh"
#include "kernels.h"

namespace ssa {
namespace {

// TILES: tensor-core tiles per block.  Two share their keys' loads and take
// turns; one, with half of an SM for its block, gives twice the blocks where
// there are few (see launch_prompt_attn).
template <int D, int TILES>
struct PromptShape {
  static constexpr int ROW = 128;                     // bytes of a 64-dim swizzled row
  static constexpr int HALVES = D / 64;
  static constexpr int TILE = 128 * ROW * HALVES;     // 128 rows (queries x heads, or keys)
  static constexpr int SLOTS = TILES == 2 ? (D == 128 ? 5 : 8) : (D == 128 ? 2 : 5);   // ring of K and V tiles
  static constexpr int BARS = TILES * TILE + SLOTS * TILE;
  static constexpr int NBAR = 1 + 2 * SLOTS + TILES + 2 * TILES + TILES + TILES + 1;
  static constexpr int USED = BARS + NBAR * 8 + 16;
  static constexpr int SMEM = USED + 1024 < 232448 ? USED + 1024 : 232448;
  static constexpr int LOADER = 4 * TILES, ISSUER = LOADER + 1;   // warps: 4 softmax warps per tile, loads, products
  static constexpr int THREADS = (LOADER + 4) * 32;               // and two idle ones that hand over registers
  static constexpr int BLOCKS = TILES == 2 ? 1 : 2;               // per SM
  static constexpr int COLS = 256 * TILES;                        // S of tile t at 128 t, O at 128 (TILES + t)
  // Registers per thread of the softmax warps and of the others, traded at the
  // start: 2 * 208 + 88 = 3 * 168, what a block of 384 threads starts with, and
  // 208 + 48 = 2 * 128 for one of 256 threads at two per SM.
  static constexpr int SOFTMAX_REGS = 208, OTHER_REGS = TILES == 2 ? 88 : 48;
  static_assert(USED <= 232448, "shared memory");
  static_assert(BLOCKS * (SMEM + 1024) <= 233472, "blocks per SM");
};

struct PromptArgs {
  const int32_t *q_start, *kv_start;
  __nv_bfloat16* O;
  float* lse;
  int64_t o_stride;
  int32_t n_seq, n_q, n_kv, h_q, h_kv, G, qt;
  int32_t n_units;
  float scale_log2;
  uint32_t* err;
};

struct PromptUnit {
  int q_row, q0, q_len, k_row, kv_len;   // first packed query row of the unit, its index in the sequence
  bool any;
};

// Warp-collective.
__device__ __forceinline__ PromptUnit prompt_unit(const PromptArgs& a, int rows, int unit) {
  const int lane = threadIdx.x & 31;
  PromptUnit u{};
  const auto start = [&](int s) { return min(max(__ldg(a.q_start + s), 0), a.n_q); };
  // the sequence is in [lo, hi): cut by 32 to at most 128, then all at once
  const auto before = [&](int s) { return start(s) / rows + s <= unit; };
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
  const int64_t q0 = static_cast<int64_t>(unit - (a0 / rows + lo)) * rows;
  if (q0 < 0 || q0 >= a1 - a0) return u;
  u.k_row = min(max(__ldg(a.kv_start + lo), 0), a.n_kv);
  u.kv_len = min(max(__ldg(a.kv_start + lo + 1), u.k_row), a.n_kv) - u.k_row;
  u.q0 = static_cast<int>(q0);
  u.q_row = a0 + u.q0;
  u.q_len = a1 - a0;
  u.any = true;
  return u;
}

__device__ __forceinline__ uint64_t prompt_desc_mn(uint32_t saddr, uint32_t lbo) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>((lbo >> 4) & 0x3FFFu) << 16;   // next 64 dims
  d |= static_cast<uint64_t>(1024 >> 4) << 32;              // next 8 keys
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32"
      " {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_st32(uint32_t taddr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32"
      " [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

// One lane of the warp, the same each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t one;
  asm volatile(
      "{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one != 0;
}

// max of three; NaN if one is.
__device__ __forceinline__ float max3_nan(float a, float b, float c) {
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// 0 * x + acc of bf16 pairs: stays a zero while x is finite.  (By tests of the
// exponents the look over the values took 10 of 230 us of three packed prompts of 8192.)
__device__ __forceinline__ uint32_t times0(uint32_t x, uint32_t acc) {
  asm("fma.rn.bf16x2 %0, %1, %2, %0;" : "+r"(acc) : "r"(x), "r"(0));
  return acc;
}

// A step's P V without the tensor core, a row per thread: where a value that
// some rows of the tile do not attend is not finite (0 * inf is NaN in the
// product).  P in bf16 pairs at p_col, values at sV, keys up to the row's
// `last`; o_col += the product (`first`: =).  Only a tile's last two steps may come
// here, for up to 60 us each (a prompt of 8192, eight heads on one, d = 128, one
// such value near its end: 116 us without, 174 with it).
template <int D>
__device__ __forceinline__ void product_by_hand(uint32_t p_col, uint32_t o_col, const uint8_t* sV, int last, bool first) {
#pragma unroll 1
  for (int d0 = 0; d0 < D; d0 += 16) {
    uint32_t o[16];
    if (first) {   // the same for the tile
#pragma unroll
      for (int k = 0; k < 16; ++k) o[k] = 0;
    } else {
      tmem_ld16(o_col + d0, o);
      tmem_wait_ld();
      tmem_regs_ready(o);
    }
    const uint8_t* half = sV + (d0 >> 6) * (128 * 128);
    const int chunk = (d0 & 63) >> 3;
#pragma unroll 1
    for (int c = 0; c < 128; c += 32) {
      if (__all_sync(0xFFFFFFFFu, c > last)) break;   // (P is not there in a short last step)
      uint32_t p[16];
      tmem_ld16(p_col + c / 2, p);
      tmem_wait_ld();
      tmem_regs_ready(p);
#pragma unroll
      for (int k = 0; k < 32; ++k) {
        const uint8_t* row = half + (c + k) * 128;   // swizzled by the key's place among eight
        const bool in = c + k <= last;
        const float x = in ? __uint_as_float(k & 1 ? p[k / 2] & 0xFFFF0000u : p[k / 2] << 16) : 0.f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const uint4 v = *reinterpret_cast<const uint4*>(row + (((chunk + h) ^ (k & 7)) << 4));
          const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const uint32_t y = in ? w[e] : 0;
            uint32_t* to = o + 8 * h + 2 * e;
            to[0] = __float_as_uint(fmaf(x, __uint_as_float(y << 16), __uint_as_float(to[0])));
            to[1] = __float_as_uint(fmaf(x, __uint_as_float(y & 0xFFFF0000u), __uint_as_float(to[1])));
          }
        }
      }
    }
    tmem_st16(o_col + d0, o);
  }
}

template <int D, int TILES>
__global__ void __launch_bounds__(PromptShape<D, TILES>::THREADS, PromptShape<D, TILES>::BLOCKS)
    prompt_kernel(const __grid_constant__ CUtensorMap tmQ, const __grid_constant__ CUtensorMap tmK,
                  const __grid_constant__ CUtensorMap tmV, const PromptArgs a) {
  using C = PromptShape<D, TILES>;
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x / 32, 0);   // known to be uniform
  const int lane = threadIdx.x & 31;
  const int kvh = blockIdx.x % a.h_kv;
  const PromptUnit u = prompt_unit(a, TILES * a.qt, a.n_units - 1 - static_cast<int>(blockIdx.x / a.h_kv));
  if (!u.any) return;   // the same for every warp

  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  if (static_cast<int>(smem - smem_raw) + C::USED > C::SMEM) {   // never with a 1024-aligned base
    if (threadIdx.x == 0) atomicCAS(a.err, 0u, static_cast<uint32_t>(SITE_PROMPT_SMEM));
    return;
  }
  uint8_t* sQ = smem;                       // [tiles][halves][128 rows][128 B]
  uint8_t* ring = smem + TILES * C::TILE;   // [slots][halves][128 keys][128 B]: K0 V0 K1 V1 ...
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::BARS);
  uint64_t* q_full = bars;
  uint64_t* full = bars + 1;
  uint64_t* empty = full + C::SLOTS;
  uint64_t* s_full = empty + C::SLOTS;     // [tiles]
  uint64_t* p_full = s_full + TILES;       // [tiles][2 halves of the step's keys]
  uint64_t* o_full = p_full + 2 * TILES;   // [tiles] the tile's last product is done
  uint64_t* hand_done = o_full + TILES;    // [tiles] a step's product added by the softmax warps
  uint64_t* mma_done = hand_done + TILES;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int32_t* odd_at = reinterpret_cast<int32_t*>(tmem_slot + 1);   // [tiles] 1 + the step to be added by hand

  // steps of each tile: keys 0 .. position of its last row; a last step that
  // needs no more than half of its 128 keys leaves out the rest
  const int off = u.kv_len - u.q_len;
  int steps[TILES], masked_from[TILES], n = 0;   // masked_from: the first step with keys that some rows do not attend
  bool short_last[TILES];
#pragma unroll
  for (int t = 0; t < TILES; ++t) {
    const int q_first = u.q0 + t * a.qt, last = min(q_first + a.qt, u.q_len) - 1 + off;
    steps[t] = q_first < u.q_len && last >= 0 ? last / 128 + 1 : 0;
    masked_from[t] = max(q_first + off + 1, 0) / 128;
    short_last[t] = steps[t] > 0 && last % 128 < 64;
    n = max(n, steps[t]);
  }

  // the loading lane sets up the barriers and starts the first loads while
  // the others allocate tensor memory
  const int loads = 2 * n;                              // K and V tiles in turn
  const int early = min(loads, C::SLOTS);
  const auto load = [&](int i) {
    const int slot = i % C::SLOTS, row = u.k_row + (i / 2) * 128;
    mbar_arrive_expect_tx(&full[slot], C::TILE);
#pragma unroll
    for (int hf = 0; hf < C::HALVES; ++hf)
      tma_load_3d(ring + slot * C::TILE + hf * 128 * C::ROW, (i & 1) ? &tmV : &tmK, &full[slot], hf * 64, kvh, row);
  };
  if (warp == C::LOADER && lane == 0) {
    mbar_init(q_full, 1);
    for (int s = 0; s < C::SLOTS; ++s) { mbar_init(&full[s], 1); mbar_init(&empty[s], 1); }
    for (int t = 0; t < TILES; ++t) {
      mbar_init(&s_full[t], 1);
      mbar_init(&p_full[2 * t], 4);
      mbar_init(&p_full[2 * t + 1], 4);
      mbar_init(&o_full[t], 1);
      mbar_init(&hand_done[t], 4);
      odd_at[t] = 0;
    }
    mbar_init(mma_done, 1);
    fence_barrier_init();
    if (n > 0) {
      uint32_t bytes = 0;
      for (int t = 0; t < TILES; ++t) bytes += steps[t] > 0 ? static_cast<uint32_t>(a.qt * a.G * C::ROW * C::HALVES) : 0;
      mbar_arrive_expect_tx(q_full, bytes);
      for (int t = 0; t < TILES; ++t)
        if (steps[t] > 0)
#pragma unroll
          for (int hf = 0; hf < C::HALVES; ++hf)
            tma_load_3d(sQ + t * C::TILE + hf * 128 * C::ROW, &tmQ, q_full, hf * 64, kvh * a.G, u.q_row + t * a.qt);
      for (int i = 0; i < early; ++i) load(i);
    }
  }
  if (warp == C::ISSUER) {
    tmem_alloc(tmem_slot, C::COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot, tmem_o = tmem + 128 * TILES;   // S and O of tile t at 128 t of each

  if (warp >= C::LOADER) {
    // this warpgroup hands registers to the softmax warpgroups
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::OTHER_REGS));
    if (warp == C::LOADER) {
      // ------------------------------------------------------------ loads
      if (lane == 0 && n > 0) {
        int i = early;
        for (; i < loads; ++i) {
          if (!mbar_wait(&empty[i % C::SLOTS], (i / C::SLOTS - 1) & 1, a.err, SITE_PROMPT_PRODUCER)) break;
          load(i);
        }
        if (i < loads) {   // a wait gave up: let the copies in flight land
          const uint64_t t0 = global_timer_ns();
          while (!mbar_try_wait(q_full, 0) && global_timer_ns() - t0 < kWaitLimitNs) {}
          for (int k = max(0, i - C::SLOTS); k < i; ++k)
            while (!mbar_try_wait(&full[k % C::SLOTS], (k / C::SLOTS) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {}
        }
      }
    } else if (warp == C::ISSUER) {
      // ------------------------------------------------------------ products
      // The whole warp runs the loop, so that descriptors and counters stay in
      // uniform registers, and one lane issues: with one lane running all of it
      // the issue, not the tensor core, set the pace (about 95 clocks per
      // product of 64).
      const bool leader = elect_one();
      constexpr uint32_t IDESC_S = umma_idesc_bf16(128, 128), IDESC_S64 = umma_idesc_bf16(128, 64);
      constexpr uint32_t IDESC_O = umma_idesc_bf16(128, D) | (1u << 16);   // V is MN-major
      const uint64_t q_desc = umma_desc_sw128(smem_u32(sQ)), k_desc = umma_desc_sw128(smem_u32(ring));
      const uint64_t v_desc = prompt_desc_mn(smem_u32(ring), 128 * C::ROW);
      constexpr uint64_t kTile = C::TILE >> 4;   // in descriptor units of 16 bytes
      const auto scores = [&](int t, int j, int slot) {   // S of tile t, step j, with the keys in `slot`
        const uint32_t idesc = short_last[t] && j + 1 == steps[t] ? IDESC_S64 : IDESC_S;
        if (leader) {
#pragma unroll
          for (int ks = 0; ks < D / 16; ++ks) {
            const uint64_t at = ((ks >> 2) * 128 * C::ROW + (ks & 3) * 32) >> 4;
            umma_bf16(tmem + 128 * t, q_desc + t * kTile + at, k_desc + slot * kTile + at, idesc, ks != 0);
          }
          umma_commit(&s_full[t]);
        }
        __syncwarp();
      };
      const auto wait = [&](uint64_t* bar, int parity) {   // the same answer in every lane
        return __all_sync(0xFFFFFFFFu, mbar_wait(bar, parity, a.err, SITE_PROMPT_MMA)) != 0;
      };
      bool ok = n == 0 || (wait(q_full, 0) && wait(&full[0], 0));
      if (ok && n > 0) {
#pragma unroll
        for (int t = 0; t < TILES; ++t)
          if (steps[t] > 0) scores(t, 0, 0);
        if (leader) umma_commit(&empty[0]);
        __syncwarp();
      }
      int v_slot = 1, v_use = 0;   // slot of load 2 j + 1 and the parity of its use
      int hands[TILES] = {};       // steps added by hand
      for (int j = 0; j < n && ok; ++j) {
        const bool more = j + 1 < n;
        const int k_slot = v_slot + 1 == C::SLOTS ? 0 : v_slot + 1, k_use = k_slot == 0 ? v_use ^ 1 : v_use;   // load 2 j + 2
        ok = wait(&full[v_slot], v_use);
#pragma unroll
        for (int t = 0; t < TILES; ++t) {
          if (!ok) break;
          const bool brief = short_last[t] && j + 1 == steps[t];
          if (j < steps[t]) {
            bool by_hand = false;   // the softmax warps add this step's product themselves
            if (j >= masked_from[t]) {
              ok = ok && wait(&p_full[2 * t], j & 1);
              by_hand = ok && __any_sync(0xFFFFFFFFu, odd_at[t] == j + 1);
            }
            if (by_hand) {
              ok = wait(&hand_done[t], hands[t] & 1);
              ++hands[t];
              tc_fence_after();
              if (ok && leader && j + 1 == steps[t]) umma_commit(&o_full[t]);
              __syncwarp();
            } else {
              // the first half of the keys while the second is exponentiated
#pragma unroll
              for (int h = 0; h < 2; ++h) {
                ok = ok && wait(&p_full[2 * t + h], j & 1);
                tc_fence_after();
                if (ok && leader) {
                  if (h == 0 || !brief)
#pragma unroll
                    for (int ks = 4 * h; ks < 4 * h + 4; ++ks)
                      umma_bf16_tmem_a(tmem_o + 128 * t, tmem + 128 * t + ks * 8,
                                       v_desc + v_slot * kTile + ((ks * 16 * C::ROW) >> 4), IDESC_O, (j | ks) != 0);
                  if (h == 1 && j + 1 == steps[t]) umma_commit(&o_full[t]);
                }
                __syncwarp();
              }
            }
          }
          if (t == TILES - 1 && leader) umma_commit(&empty[v_slot]);
          // S over the P just read: products of one thread run in order
          if (ok && more && j + 1 < steps[t]) {
            ok = wait(&full[k_slot], k_use);
            if (ok) scores(t, j + 1, k_slot);
          }
          if (t == TILES - 1 && more && leader) umma_commit(&empty[k_slot]);
        }
        v_slot = k_slot + 1 == C::SLOTS ? 0 : k_slot + 1;
        v_use = v_slot == 0 ? k_use ^ 1 : k_use;
      }
      if (leader) {
        umma_commit(mma_done);   // all issued products complete before TMEM is freed
        const uint64_t t0 = global_timer_ns();
        while (!mbar_try_wait(mma_done, 0) && global_timer_ns() - t0 < kWaitLimitNs) {}
      }
      __syncwarp();
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::SOFTMAX_REGS));
    // ------------------------------------------------------------ softmax and output, one row per thread
    const int t = TILES == 2 ? warp >> 2 : 0;
    const int my_steps = steps[t];
    const bool my_short = short_last[t];
    const int row = threadIdx.x & 127;
    const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t s_col = tmem + lanes + 128 * t, o_col = tmem_o + lanes + 128 * t;
    const int qi = u.q0 + t * a.qt + row / a.G;             // query of the row within its sequence
    const bool valid = row < a.qt * a.G && qi < u.q_len;
    const int pos = valid ? qi + off : -1;
    const int pos_first = u.q0 + t * a.qt + off;            // of the tile's first row
    float m = -INFINITY;     // reference of the row, in logits before the scale
    uint64_t l2[2] = {0, 0};
    bool ok = true;
    // a barrier of the tile's four warps
    const auto tile_any = [&](bool x) {
      int any;
      asm volatile(
          "{\n\t.reg .pred p, q;\n\tsetp.ne.s32 p, %1, 0;\n\t"
          "barrier.cta.red.or.pred q, %2, 128, p;\n\tselp.s32 %0, 1, 0, q;\n\t}"
          : "=r"(any)
          : "r"(x ? 1 : 0), "r"(1 + t)
          : "memory");
      return any != 0;
    };
    int j = 0;
    for (; j < my_steps; ++j) {
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&s_full[t], j & 1, a.err, SITE_PROMPT_SOFTMAX));
      if (!ok) break;
      tc_fence_after();
      uint32_t r[128];
      const bool brief = my_short && j + 1 == my_steps;     // only the first half of the keys (so masked below)
#pragma unroll
      for (int c = 0; c < 4; ++c)
        if (c < 2 || !brief) tmem_ld32(s_col + 32 * c, r + 32 * c);
      tmem_wait_ld();
      tmem_regs_ready(r);
      const bool masked = j * 128 + 127 > pos_first;        // the same for the tile
      if (masked) {
        const int last = pos - j * 128;
#pragma unroll
        for (int c = 0; c < 128; ++c)
          if (c > last) r[c] = 0xFF800000u;
      }
      float mx[4] = {m, m, m, m};
#pragma unroll
      for (int c = 0; c < 128; c += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k)
          mx[k] = max3_nan(mx[k], __uint_as_float(r[c + 2 * k]), __uint_as_float(r[c + 2 * k + 1]));
      const float mn = max3_nan(max3_nan(mx[0], mx[1], mx[2]), mx[3], mx[3]);
      // a new reference only when the maximum has grown by 2^8 (or from nothing)
      const bool grow = mn > m && (m == -INFINITY || (mn - m) * a.scale_log2 > 8.f);
      if (__any_sync(0xFFFFFFFFu, grow)) {
        const float f = grow ? (m == -INFINITY ? 0.f : fast_exp2((m - mn) * a.scale_log2)) : 1.f;
        if (grow) m = mn;
        const uint64_t f2 = pair(f, f);
#pragma unroll
        for (int k = 0; k < 2; ++k) l2[k] = fma2(l2[k], f2, 0);
        if (j > 0) {   // the tile's earlier products are done: this S came after them
#pragma unroll 1
          for (int c = 0; c < D / 16; ++c) {
            uint32_t o[16];
            tmem_ld16(o_col + 16 * c, o);
            tmem_wait_ld();
            tmem_regs_ready(o);
#pragma unroll
            for (int k = 0; k < 16; ++k) o[k] = __float_as_uint(__uint_as_float(o[k]) * f);
            tmem_st16(o_col + 16 * c, o);
          }
        }
      }
      // a NaN or +inf among the logits: the row is NaN, which the sum carries
      if (!(mn < INFINITY)) l2[0] = pair(__int_as_float(0x7FFFFFFF), 0.f);
      const float mr = m == -INFINITY ? 0.f : m;
      const uint64_t sc2 = pair(a.scale_log2, a.scale_log2), ms2 = pair(-mr * a.scale_log2, -mr * a.scale_log2);
      if (masked) {
        // values of keys that some row of the tile does not attend: those
        // behind the sequence become zero, those inside it are looked over
        const int i = 2 * j + 1;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&full[i % C::SLOTS], (i / C::SLOTS) & 1, a.err, SITE_PROMPT_SOFTMAX));
        if (!ok) break;
        uint8_t* sV = ring + (i % C::SLOTS) * C::TILE;
        const int end = min(u.kv_len - j * 128, 128), from = max(pos_first + 1 - j * 128, 0);
        constexpr int CH = 8 * C::HALVES;   // 16-byte pieces of a key
        const auto piece = [&](int x) {
          return reinterpret_cast<uint4*>(sV + (x % CH >> 3) * 128 * C::ROW + x / CH * C::ROW + (x & 7) * 16);
        };
        for (int x = end * CH + row; x < 128 * CH; x += 128) *piece(x) = make_uint4(0, 0, 0, 0);
        uint32_t odd = 0;
#pragma unroll 4
        for (int x = from * CH + row; x < end * CH; x += 128) {
          const uint4 v = *piece(x);
          odd = times0(v.w, times0(v.z, times0(v.y, times0(v.x, odd))));
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        if (odd & 0x7FFF7FFFu) odd_at[t] = j + 1;   // one is not finite
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        if (h == 0 || !brief) {
          uint32_t p[32];
#pragma unroll
          for (int c = 0; c < 32; ++c) {
            const uint64_t x2 =
                fma2(pair(__uint_as_float(r[64 * h + 2 * c]), __uint_as_float(r[64 * h + 2 * c + 1])), sc2, ms2);
            float x, y;
            unpair(x2, x, y);
            x = fast_exp2(x);
            y = fast_exp2(y);
            l2[c & 1] = add2(l2[c & 1], pair(x, y));
            p[c] = pack_bf16(x, y);
          }
          tmem_st32(s_col + 32 * h, p);
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[2 * t + h]);
      }
      // (after P has left: the tensor core need not wait for this barrier)
      if (masked && tile_any(odd_at[t] == j + 1)) {
        product_by_hand<D>(s_col, o_col, ring + ((2 * j + 1) % C::SLOTS) * C::TILE, pos - j * 128, j == 0);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&hand_done[t]);
      }
    }
    // a warp that gave up before the barrier of step j still meets the others there and after
    for (; j < my_steps; ++j)
      if (j * 128 + 127 > pos_first) tile_any(false);
    float l0, l1, l2_, l3;
    unpair(l2[0], l0, l1);
    unpair(l2[1], l2_, l3);
    const float l = (l0 + l1) + (l2_ + l3);
    const float inv = l == 0.f ? 0.f : 1.f / l;
    const float mr = m == -INFINITY ? 0.f : m * a.scale_log2;
    const int head = kvh * a.G + row % a.G;
    const int64_t q_row = u.q_row + t * a.qt + row / a.G;
    __nv_bfloat16* out = a.O + q_row * a.o_stride + static_cast<int64_t>(head) * D;
    if (ok && my_steps > 0)
      ok = __all_sync(0xFFFFFFFFu, mbar_wait(&o_full[t], 0, a.err, SITE_PROMPT_SOFTMAX));
    if (ok) {
      if (valid && a.lse) a.lse[q_row * a.h_q + head] = l == 0.f ? -INFINITY : (mr + log2f(l)) * 0.6931471805599453f;
      tc_fence_after();
#pragma unroll 1
      for (int c = 0; c < D / 32; ++c) {
        uint32_t o[32];
        if (my_steps > 0) {   // the same for the tile
          tmem_ld32(o_col + 32 * c, o);
          tmem_wait_ld();
          tmem_regs_ready(o);
        } else {
#pragma unroll
          for (int k = 0; k < 32; ++k) o[k] = 0;
        }
        if (valid) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            uint32_t w[4];
#pragma unroll
            for (int e = 0; e < 4; ++e)
              w[e] = pack_bf16(__uint_as_float(o[8 * k + 2 * e]) * inv, __uint_as_float(o[8 * k + 2 * e + 1]) * inv);
            reinterpret_cast<uint4*>(out)[c * 4 + k] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::ISSUER) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, C::COLS);
  }
}

template <int D, int TILES>
cudaError_t run_prompt(const CUtensorMap& tmQ, const CUtensorMap& tmK, const CUtensorMap& tmV, PromptArgs a,
                       const LaunchCtx& c) {
  using C = PromptShape<D, TILES>;
  a.n_units = a.n_q / (TILES * a.qt) + a.n_seq;
  cudaError_t e = cudaFuncSetAttribute(prompt_kernel<D, TILES>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  const int64_t grid = static_cast<int64_t>(a.n_units) * a.h_kv;
  if (grid > INT32_MAX) return cudaErrorInvalidValue;
  prompt_kernel<D, TILES><<<static_cast<unsigned>(grid), C::THREADS, C::SMEM, c.stream>>>(tmQ, tmK, tmV, a);
  note_launch();
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_prompt_attn(const ssa_prompt_params& p, const void* Q, const void* K, const void* V,
                               const int32_t* q_start, const int32_t* kv_start, void* O, float* lse,
                               const LaunchCtx& c) {
  PromptArgs a{};
  a.q_start = q_start; a.kv_start = kv_start;
  a.O = static_cast<__nv_bfloat16*>(O);
  a.lse = lse;
  a.o_stride = p.o_stride;
  a.n_seq = p.n_seq; a.n_q = p.n_q; a.n_kv = p.n_kv; a.h_q = p.h_q; a.h_kv = p.h_kv;
  a.G = p.h_q / p.h_kv;
  a.qt = 128 / a.G;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.err = c.err;
  // without key rows no unit loads any: the maps then describe the queries
  CUtensorMap tmQ, tmK, tmV;
  const bool kv = p.n_kv > 0;
  if (!encode_heads(&tmQ, Q, p.d, p.h_q, p.n_q, p.q_stride, a.G, a.qt) ||
      !encode_heads(&tmK, kv ? K : Q, p.d, kv ? p.h_kv : p.h_q, kv ? p.n_kv : p.n_q, kv ? p.k_stride : p.q_stride, 1,
                    128) ||
      !encode_heads(&tmV, kv ? V : Q, p.d, kv ? p.h_kv : p.h_q, kv ? p.n_kv : p.n_q, kv ? p.v_stride : p.q_stride, 1,
                    128))
    return cudaErrorInvalidValue;
  // One tile per block where a second would mostly be empty (64 prompts of one
  // token, 32 heads on 8: 24 us with two tiles, 15 with one), where blocks of
  // two would leave SMs idle (a prompt of 2000, eight kv-heads, d = 64: 34 us
  // with two, 26 with one), and where they would need a second round that is
  // not long (23 prompts of 48 tokens, eight kv-heads: 10.7 and 7.6 us; but a
  // prompt of 8000, eight heads on one: 113 and 120 us).
  const int64_t two = (static_cast<int64_t>(p.n_q) / (2 * a.qt) + p.n_seq) * p.h_kv;
  if (p.n_q <= static_cast<int64_t>(a.qt) * p.n_seq || two < c.sm_count ||
      (two < 2 * c.sm_count && p.n_kv <= static_cast<int64_t>(4096) * p.n_seq))
    return p.d == 128 ? run_prompt<128, 1>(tmQ, tmK, tmV, a, c) : run_prompt<64, 1>(tmQ, tmK, tmV, a, c);
  return p.d == 128 ? run_prompt<128, 2>(tmQ, tmK, tmV, a, c) : run_prompt<64, 2>(tmQ, tmK, tmV, a, c);
}

}  // namespace ssa
