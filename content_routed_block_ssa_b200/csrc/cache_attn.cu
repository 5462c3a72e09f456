// Attention of new tokens over the paged 8-bit cache, all keys or the
// selected blocks plus the window.
//
// A unit is up to 16 query rows that share a kv-head (new tokens x the G query
// heads of the group; with selected blocks one token's G heads), and a unit's
// keys are cut into `splits` runs, one block each, whose partial results a
// second kernel joins.  Each of a block's three warps walks its own pieces of
// 4 KB of keys and of values (every third of the run) with a ring of bulk
// copies of its own, so no warp waits for another until the end.  The products
// are small against the bytes (2 G flops per byte): the kernel is bound by
// reading codes (64 sequences of up to 16K tokens, 32 heads on 8, d = 128: 224
// to 248 us by the box, 81 to 90% of the copy rate), and the instructions per
// code decide whether it keeps up:
//
//  * the keys and the value dims are the M = 16 rows of the m16n8k16 products
//    (S^T = K Q^T, O^T = V^T P^T) and the query rows their N = 8 columns: a
//    group of up to eight rows wastes nothing, and a lane holds 8 logits and
//    D/4 outputs.  P^T moves from the accumulator's layout to the operand's by
//    one 8x8 transposition per eight keys.
//  * codes become float16 (exact) straight from shared memory to the A
//    operands, without a pass through float32.  The k index of a product may
//    run over the dims (or keys) in any order as long as both operands agree,
//    so a lane takes 16 consecutive bytes of a key (S^T) or of a value row
//    (O^T) and calls them its indexes; for O^T, bytes of two keys are paired
//    by byte permutes before the conversion.
//  * a page's key scale multiplies its logits; its value scale 2^e is added to
//    the base-2 logits: P' = 2^(s + e - M) needs no factor on the output, and
//    the sum of the softmax takes P' 2^-e.  The reference M is the running
//    maximum of s + e less 15 (reference_of): P' is at most 2^15, float16's
//    upper end, so that it keeps its 11 bits down to 2^-29 of the row's largest
//    P' and vanishes below 2^-40.  (Relative to the maximum itself a key 2^-26
//    below it left the output and stayed in the sum: rows that a key with a value of
//    zero dominates by 18 nats came out as 0, whatever their other keys.)
//  * queries become float16 after scaling each row by a power of two to a
//    largest element in [2^14, 2^15): exact down to 2^-29 of the largest.
#include <cuda_bf16.h>
#include <math.h>

#include "cache.cuh"
#include "common.cuh"
#include "kernels.h"
#include "tiles.cuh"

namespace ssa {
namespace {

// Keys per piece: 4 KB of keys (a piece has a fixed cost of some 150 instructions).
constexpr int piece_keys(int d) { return d == 64 ? 64 : 32; }
constexpr int kWarps = 3;
constexpr int kBlocks = 4;     // blocks per SM
constexpr int kMaxEnt = 32 + 4032 / 64 + 2;   // selected blocks and window blocks
constexpr int kSmCount = 148;

struct CacheCfg {
  CacheAttnArgs g;
  int32_t n_seq, n_q, max_pages, n_pages, page, h_q, h_kv, G, topk, window;
  int32_t tiles;     // units per (sequence, kv-head)
  int32_t unit_rows; // rows of a unit without selected blocks: 8 or 16
  int32_t rows;      // partial rows stored per unit
  int32_t splits;
  float scale_log2;
  float* part_o;     // [units][splits][rows][D]
  float2* part_ml;   // [units][splits][rows]: reference, sum
  uint32_t* err;
};

template <int D>
struct CacheShape {
  static constexpr int PIECE = piece_keys(D);
  static constexpr int K_BYTES = PIECE * D;
  static constexpr int STAGE = 2 * K_BYTES;
  static constexpr int STAGES = 16384 / STAGE;
  static constexpr int RING = STAGES * STAGE;
  static constexpr int OROW = D + 4;   // floats per row of the join, skewed over the banks
  static constexpr int BARS = kWarps * RING;
  static constexpr int ENTS = BARS + kWarps * STAGES * 8;
  static constexpr int SMEM = ENTS + (kMaxEnt + 1) * 8;
  static_assert(kWarps * 16 * (OROW + 2) * 4 <= BARS, "the join fits the rings");
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32"
      " {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  const __half2 h = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&h);
}

// 0x80 in every byte that is an e4m3 NaN.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) { return ((w & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u; }

// One query row's A operand halves: 16 dims at 64 c + 16 t of each 64-dim
// part c, scaled by a power of two; returns the logit factor of the row.
template <int D>
__device__ __forceinline__ float load_query(const __nv_bfloat16* q, int t, bool valid, float scale_log2,
                                            uint32_t (&h)[D / 64][8]) {
  float x[D / 64][16];
  float m = 0.f;
#pragma unroll
  for (int c = 0; c < D / 64; ++c) {
    uint4 v[2] = {make_uint4(0, 0, 0, 0), make_uint4(0, 0, 0, 0)};
    if (valid) {
      v[0] = *reinterpret_cast<const uint4*>(q + 64 * c + 16 * t);
      v[1] = *reinterpret_cast<const uint4*>(q + 64 * c + 16 * t + 8);
    }
    const uint32_t* w = reinterpret_cast<const uint32_t*>(v);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      x[c][2 * i] = __uint_as_float(w[i] << 16);
      x[c][2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      m = fmaxf(m, fmaxf(fabsf(x[c][2 * i]), fabsf(x[c][2 * i + 1])));
    }
  }
  m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 1));
  m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 2));
  // largest element to [2^14, 2^15); rows of tiny or infinite elements are
  // clamped so that both factors stay normal floats
  const int e = min(max(static_cast<int>(__float_as_uint(m) >> 23) - 127, -100), 127);
  const float f = pow2(14 - e);
#pragma unroll
  for (int c = 0; c < D / 64; ++c)
#pragma unroll
    for (int i = 0; i < 8; ++i) h[c][i] = half2_bits(x[c][2 * i] * f, x[c][2 * i + 1] * f);
  return scale_log2 * pow2(e - 14);
}

// The reference of the base-2 logits up to m: 15 below it.  Not where float32
// steps are so coarse that m - 15 could round to m - 16 and P' pass float16's
// end; there m itself.  -inf (no keys yet) stays.
__device__ __forceinline__ float reference_of(float m) { return fabsf(m) < 4194304.f ? m - 15.f : m; }

// What a lane keeps of one upcoming piece of its warp.
struct Piece {
  int page;      // -1: outside the pool
  int key0;      // position of its first key
  int lo;        // first position that counts (0, or the window's)
  float ks, vs;
};

// R: query rows of a unit in groups of eight.
template <int D, bool SEL, int R>
__global__ void __launch_bounds__(kWarps * 32, R == 1 ? kBlocks : 3) cache_attn_kernel(const CacheCfg a) {
  using C = CacheShape<D>;
  constexpr int MT = D / 16;    // output tiles of 16 dims
  constexpr int QT = C::PIECE / 16;   // key tiles of a piece
  constexpr int VW = D / 32;    // words of a value row per lane
  extern __shared__ __align__(128) uint8_t smem[];
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, g = lane >> 2, t = lane & 3;
  uint8_t* ring = smem + warp * C::RING;
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + C::BARS) + warp * C::STAGES;
  int2* ents = reinterpret_cast<int2*>(smem + C::ENTS);   // (block | window flag in bit 30, page); then the count

  const int split = blockIdx.x % a.splits;
  const int unit = blockIdx.x / a.splits;
  const int kvh = unit % a.h_kv;
  const int tile = unit / a.h_kv % a.tiles;
  const int seq = unit / a.h_kv / a.tiles;
  const int32_t* table = a.g.table + static_cast<int64_t>(seq) * a.max_pages;
  int entry = -1, entry_page = -1;   // warp 0: this lane's block_idx entry and its page
  if (SEL && warp == 0 && lane < a.topk) {
    entry = __ldg(a.g.idx + ((static_cast<int64_t>(seq) * a.n_q + tile) * a.h_kv + kvh) * a.topk + lane);
    if (entry >= 0 && entry < a.max_pages) entry_page = __ldg(table + entry);
  }
  const int len = min(max(__ldg(a.g.kv_len + seq), 0), a.max_pages * a.page);
  // rows of the unit: row r is token (r0 + r) / G, head (r0 + r) % G
  const int r0 = SEL ? tile * a.G : tile * 8 * R;
  const int n_rows = SEL ? a.G : min(8 * R, a.n_q * a.G - r0);
  const int first = len - a.n_q;                                // position of token 0
  const int pos_lo = first + r0 / a.G, pos_hi = first + (r0 + n_rows - 1) / a.G;
  int pos[R][2];   // of this lane's rows 8 n + 2 t and + 1
#pragma unroll
  for (int n = 0; n < R; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = 8 * n + 2 * t + c;
      pos[n][c] = r < n_rows ? first + (r0 + r) / a.G : -1;
    }
  const int ppb = a.page / C::PIECE;
  const int wlo = SEL ? max(pos_hi - a.window + 1, 0) : 0;

  if (lane == 0)
#pragma unroll
    for (int s = 0; s < C::STAGES; ++s) mbar_init(&full[s], 1);
  fence_barrier_init();
  int n_pieces;
  if (SEL) {
    if (warp == 0) {
      // the used selected blocks, then the window's blocks outside them, with
      // their pages.  The entries' pages are looked up before it is known which
      // entries count: one load less in the chain to the first copy.
      int n = 0;
      if (pos_hi >= 0) {
        const int nvis = (pos_hi + 1) / a.page;
        const bool inrange = entry >= 0 && entry < nvis;
        int run = inrange ? entry : -1;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int y = __shfl_up_sync(0xFFFFFFFFu, run, o);
          if (lane >= o) run = max(run, y);
        }
        int prev = __shfl_up_sync(0xFFFFFFFFu, run, 1);
        if (lane == 0) prev = -1;
        const bool used = inrange && entry > prev;
        const uint32_t um = __ballot_sync(0xFFFFFFFFu, used);
        if (used) ents[__popc(um & ((1u << lane) - 1))] = make_int2(entry, entry_page);
        n = __popc(um);
        const int skipped = __popc(__ballot_sync(0xFFFFFFFFu, lane < a.topk && entry != -1 && !used));
        if (lane == 0 && split == 0 && skipped && a.g.bad) atomicAdd(a.g.bad, skipped);
        __syncwarp();
        const int w1 = pos_hi / a.page;
        for (int b = wlo / a.page; b <= w1; b += 32) {
          const int blk = b + lane;
          bool add = blk <= w1;
          const int pg = add ? __ldg(table + blk) : -1;
          for (int i = 0; i < __popc(um); ++i) add = add && ents[i].x != blk;
          const uint32_t am = __ballot_sync(0xFFFFFFFFu, add);
          if (add) ents[n + __popc(am & ((1u << lane) - 1))] = make_int2(blk | 1 << 30, pg);
          n += __popc(am);
        }
      }
      if (lane == 0) ents[kMaxEnt].x = n;
    }
    __syncthreads();
    n_pieces = ents[kMaxEnt].x * ppb;
  } else {
    __syncwarp();
    n_pieces = pos_hi >= 0 ? pos_hi / C::PIECE + 1 : 0;
  }
  const int c0 = static_cast<int>(static_cast<int64_t>(n_pieces) * split / a.splits);
  const int c1 = static_cast<int>(static_cast<int64_t>(n_pieces) * (split + 1) / a.splits);
  const int n_my = max(0, (c1 - c0 - warp + kWarps - 1) / kWarps);

  const auto fetch = [&](int i) {   // piece i of this warp, one per lane
    Piece p;
    p.page = -1;
    p.key0 = p.lo = 0;
    p.ks = p.vs = 0.f;
    if (i < n_my) {
      const int c = c0 + warp + i * kWarps;
      int blk = c / ppb, page;
      if (SEL) {
        const int2 e = ents[blk];
        blk = e.x & ~(1 << 30);
        p.lo = e.x >> 30 ? wlo : 0;
        page = e.y;
      } else {
        page = __ldg(table + blk);
      }
      p.key0 = blk * a.page + (c % ppb) * C::PIECE;
      if (page >= 0 && page < a.n_pages) {
        p.page = page;
        const int64_t ph = static_cast<int64_t>(page) * a.h_kv + kvh;
        p.ks = __ldg(a.g.ks + ph);
        p.vs = __ldg(a.g.vs + ph);
      } else if (a.g.bad && p.key0 % a.page == 0) {
        atomicAdd(a.g.bad, 1);
      }
    }
    return p;
  };
  const auto issue = [&](int i, const Piece& from) {
    const int page = __shfl_sync(0xFFFFFFFFu, from.page, i & 31);
    const int key0 = __shfl_sync(0xFFFFFFFFu, from.key0, i & 31);
    if (lane == 0) {
      uint64_t* bar = &full[i % C::STAGES];
      if (page < 0) {
        mbar_arrive(bar);
      } else {
        uint8_t* dst = ring + (i % C::STAGES) * C::STAGE;
        const int64_t off = ((static_cast<int64_t>(page) * a.h_kv + kvh) * a.page + key0 % a.page) * D;
        mbar_arrive_expect_tx(bar, C::STAGE);
        bulk_load(dst, a.g.kc + off, C::K_BYTES, bar);
        bulk_load(dst + C::K_BYTES, a.g.vc + off, C::K_BYTES, bar);
      }
    }
  };

  Piece cur = fetch(lane);
#pragma unroll
  for (int i = 0; i < C::STAGES; ++i)
    if (i < n_my) issue(i, cur);
  Piece nxt = fetch(32 + lane);

  // queries while the first copies fly: the B operand of row 8 n + g
  uint32_t Q[R][D / 64][8];
  float qf[R][2];   // logit factors of this lane's rows
#pragma unroll
  for (int n = 0; n < R; ++n) {
    const int r = 8 * n + g;
    const int row = r0 + (r < n_rows ? r : 0), i = row / a.G, h = row % a.G;
    const float f = load_query<D>(static_cast<const __nv_bfloat16*>(a.g.Q) +
                                      ((static_cast<int64_t>(seq) * a.n_q + i) * a.h_q + kvh * a.G + h) * D,
                                  t, r < n_rows, a.scale_log2, Q[n]);
    qf[n][0] = __shfl_sync(0xFFFFFFFFu, f, 8 * t);
    qf[n][1] = __shfl_sync(0xFFFFFFFFu, f, 8 * t + 4);
  }

  // O[n][j]: dims D/8 g + 2 j (c = 0, 1) and + 1 (c = 2, 3), rows 8 n + 2 t (c even) and + 1
  float O[R][MT][4];
  float M[R][2], l[R][2];
#pragma unroll
  for (int n = 0; n < R; ++n) {
#pragma unroll
    for (int j = 0; j < MT; ++j)
#pragma unroll
      for (int c = 0; c < 4; ++c) O[n][j][c] = 0.f;
    M[n][0] = M[n][1] = -INFINITY;
    l[n][0] = l[n][1] = 0.f;
  }

  int done = 0;
  for (; done < n_my; ++done) {
    const int i = done, b = i & 31;
    if (b == 0 && i > 0) {
      cur = nxt;
      nxt = fetch(i + 32 + lane);
    }
    const int page = __shfl_sync(0xFFFFFFFFu, cur.page, b);
    const int key0 = __shfl_sync(0xFFFFFFFFu, cur.key0, b);
    const float ks = __shfl_sync(0xFFFFFFFFu, cur.ks, b);
    const float vs = fmaxf(__shfl_sync(0xFFFFFFFFu, cur.vs, b), 8.077935669463161e-28f);   // 2^-90: sums of its inverse stay finite
    const int lo = SEL ? __shfl_sync(0xFFFFFFFFu, cur.lo, b) : 0;
    const int st = i % C::STAGES;
    if (!__all_sync(0xFFFFFFFFu, mbar_wait(&full[st], (i / C::STAGES) & 1, a.err, SITE_CACHE_FULL))) break;
    if (page >= 0) {
      const uint8_t* sK = ring + st * C::STAGE;
      const uint8_t* sV = sK + C::K_BYTES;
      const float lvs = log2f(vs), ivs = 1.f / vs;
      const bool partial = key0 + C::PIECE - 1 > pos_lo || key0 < lo;
      // S^T = K Q^T: keys 16 q + g (c = 0, 1) and + 8 (c = 2, 3) of this lane
      float S[R][QT][4];
#pragma unroll
      for (int q = 0; q < QT; ++q) {
#pragma unroll
        for (int n = 0; n < R; ++n)
#pragma unroll
          for (int c = 0; c < 4; ++c) S[n][q][c] = 0.f;
#pragma unroll
        for (int c = 0; c < D / 64; ++c) {
          const uint4 x = *reinterpret_cast<const uint4*>(sK + (q * 16 + g) * D + c * 64 + t * 16);
          const uint4 y = *reinterpret_cast<const uint4*>(sK + (q * 16 + 8 + g) * D + c * 64 + t * 16);
          const uint32_t xw[4] = {x.x, x.y, x.z, x.w}, yw[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            uint32_t A[4];
            e4m3x4_to_half2(xw[s], A[0], A[2]);
            e4m3x4_to_half2(yw[s], A[1], A[3]);
#pragma unroll
            for (int n = 0; n < R; ++n) mma_f16(S[n][q], A, Q[n][c][2 * s], Q[n][c][2 * s + 1]);
          }
        }
      }
      float m[R][2];
#pragma unroll
      for (int n = 0; n < R; ++n) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          const float f = qf[n][c] * ks;
#pragma unroll
          for (int q = 0; q < QT; ++q) {
            S[n][q][c] = fmaf(S[n][q][c], f, lvs);
            S[n][q][2 + c] = fmaf(S[n][q][2 + c], f, lvs);
            if (partial) {
              const int kp = key0 + q * 16 + g;
              if (kp > pos[n][c] || kp < lo) S[n][q][c] = -INFINITY;
              if (kp + 8 > pos[n][c] || kp + 8 < lo) S[n][q][2 + c] = -INFINITY;
            }
          }
          m[n][c] = fmaxf(S[n][0][c], S[n][0][2 + c]);
#pragma unroll
          for (int q = 1; q < QT; ++q) m[n][c] = fmaxf(m[n][c], fmaxf(S[n][q][c], S[n][q][2 + c]));
        }
      }
#pragma unroll
      for (int o = 4; o < 32; o <<= 1)
#pragma unroll
        for (int n = 0; n < R; ++n)
#pragma unroll
          for (int c = 0; c < 2; ++c) m[n][c] = fmaxf(m[n][c], __shfl_xor_sync(0xFFFFFFFFu, m[n][c], o));
      bool moved = false;
#pragma unroll
      for (int n = 0; n < R; ++n) {
        m[n][0] = reference_of(m[n][0]);
        m[n][1] = reference_of(m[n][1]);
        moved = moved || m[n][0] > M[n][0] || m[n][1] > M[n][1];
      }
      if (__any_sync(0xFFFFFFFFu, moved)) {   // a reference moved: rescale
#pragma unroll
        for (int n = 0; n < R; ++n) {
          float x[2];
#pragma unroll
          for (int c = 0; c < 2; ++c) {
            const float to = fmaxf(M[n][c], m[n][c]);
            x[c] = to == -INFINITY ? 1.f : fast_exp2(M[n][c] - to);
            M[n][c] = to;
            l[n][c] *= x[c];
          }
#pragma unroll
          for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c) O[n][j][c] *= x[c & 1];
        }
      }
      uint32_t P[R][QT][2];
#pragma unroll
      for (int n = 0; n < R; ++n) {
        const float ra = M[n][0] == -INFINITY ? 0.f : M[n][0], rb = M[n][1] == -INFINITY ? 0.f : M[n][1];
        float sa = 0.f, sb = 0.f;
#pragma unroll
        for (int q = 0; q < QT; ++q)
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            const float x = fast_exp2(S[n][q][2 * k] - ra), y = fast_exp2(S[n][q][2 * k + 1] - rb);
            sa += x;
            sb += y;
            P[n][q][k] = movmatrix_trans(half2_bits(x, y));   // keys 16 q + 8 k + 2 t, + 1 of row 8 n + g
          }
        l[n][0] = fmaf(sa, ivs, l[n][0]);
        l[n][1] = fmaf(sb, ivs, l[n][1]);
      }
      // O^T += V^T P^T: keys 16 q + {2t, 2t+1, 2t+8, 2t+9}
      uint32_t odd = 0;   // NaN among values that not every row attends
#pragma unroll
      for (int q = 0; q < QT; ++q) {
        uint32_t v[4][VW];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int key = 16 * q + 2 * t + (k & 1) + 8 * (k >> 1);
          if (D == 128) {
            const uint4 x = *reinterpret_cast<const uint4*>(sV + key * D + g * 16);
            v[k][0] = x.x; v[k][1] = x.y; v[k][VW - 2] = x.z; v[k][VW - 1] = x.w;
          } else {
            const uint2 x = *reinterpret_cast<const uint2*>(sV + key * D + g * 8);
            v[k][0] = x.x; v[k][1] = x.y;
          }
          if (partial) {
            const int kp = key0 + key;
#pragma unroll
            for (int w = 0; w < VW; ++w) {
              if (kp > pos_hi || kp < lo) {
                v[k][w] = 0;   // no row attends it
              } else {
                const uint32_t nb = nan_bytes(v[k][w]);
                odd |= nb;
                v[k][w] &= ~((nb >> 7) * 0xFFu);
              }
            }
          }
        }
#pragma unroll
        for (int w = 0; w < VW; ++w)
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const uint32_t sel = h ? 0x7362 : 0x5140;
            uint32_t A[4];
            e4m3x4_to_half2(__byte_perm(v[0][w], v[1][w], sel), A[0], A[1]);
            e4m3x4_to_half2(__byte_perm(v[2][w], v[3][w], sel), A[2], A[3]);
#pragma unroll
            for (int n = 0; n < R; ++n) mma_f16(O[n][2 * w + h], A, P[n][q][0], P[n][q][1]);
          }
      }
      if (partial && __any_sync(0xFFFFFFFFu, odd != 0)) {
        // 0 * NaN is NaN: such values stay out of the product and reach the
        // rows that attend them here
        const float bad = __int_as_float(0x7FFFFFFF);
        for (int key = 0; key < C::PIECE; ++key) {
          const int kp = key0 + key;
          if (kp > pos_hi || kp < lo) continue;
#pragma unroll
          for (int j = 0; j < MT; ++j)
#pragma unroll
            for (int c = 0; c < 4; ++c)
              if ((sV[key * D + g * (D / 8) + 2 * j + (c >> 1)] & 0x7F) == 0x7F) {
#pragma unroll
                for (int n = 0; n < R; ++n)
                  if (kp <= pos[n][c & 1]) O[n][j][c] = bad;
              }
        }
      }
    }
    __syncwarp();   // every lane has read the stage
    const int ahead = i + C::STAGES;
    if (ahead < n_my) {
      const bool same = ahead / 32 == i / 32;
      Piece from;
      from.page = same ? cur.page : nxt.page;
      from.key0 = same ? cur.key0 : nxt.key0;
      issue(ahead, from);
    }
  }
  if (done < n_my) {   // a wait gave up: let the copies in flight land
    const uint64_t t0 = global_timer_ns();
    for (int i = done; i < min(done + C::STAGES, n_my); ++i)
      while (!mbar_try_wait(&full[i % C::STAGES], (i / C::STAGES) & 1) && global_timer_ns() - t0 < kWaitLimitNs) {}
  }

  // join the warps: maxima and sums, then outputs, through the rings
#pragma unroll
  for (int o = 4; o < 32; o <<= 1)
#pragma unroll
    for (int n = 0; n < R; ++n)
#pragma unroll
      for (int c = 0; c < 2; ++c) l[n][c] += __shfl_xor_sync(0xFFFFFFFFu, l[n][c], o);
  __syncthreads();
  float* jo = reinterpret_cast<float*>(smem);                                // [warps][8 R][OROW]
  float2* jml = reinterpret_cast<float2*>(jo + kWarps * 8 * R * C::OROW);    // [warps][8 R]
#pragma unroll
  for (int n = 0; n < R; ++n)
#pragma unroll
    for (int c = 0; c < 2; ++c) {
      const int r = 8 * n + 2 * t + c;
      if (g == 0) jml[warp * 8 * R + r] = make_float2(M[n][c], l[n][c]);
      if (r < n_rows) {
        float* to = jo + (warp * 8 * R + r) * C::OROW + g * (D / 8);
#pragma unroll
        for (int j = 0; j < MT; j += 2)
          *reinterpret_cast<float4*>(to + 2 * j) =
              make_float4(O[n][j][c], O[n][j][2 + c], O[n][j + 1][c], O[n][j + 1][2 + c]);
      }
    }
  __syncthreads();
  constexpr int QR = D / 4;   // threads per row
  for (int x = threadIdx.x; x < n_rows * QR; x += kWarps * 32) {
    const int r = x / QR, q = x % QR;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) top = fmaxf(top, jml[w * 8 * R + r].x);
    float sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float2 ml = jml[w * 8 * R + r];
      const float f = top == -INFINITY ? 1.f : exp2f(ml.x - top);
      const float4 y = *reinterpret_cast<const float4*>(jo + (w * 8 * R + r) * C::OROW + 4 * q);
      sum = fmaf(f, ml.y, sum);
      o.x = fmaf(f, y.x, o.x); o.y = fmaf(f, y.y, o.y); o.z = fmaf(f, y.z, o.z); o.w = fmaf(f, y.w, o.w);
    }
    if (a.splits > 1) {
      const int64_t pr = (static_cast<int64_t>(unit) * a.splits + split) * a.rows + r;
      reinterpret_cast<float4*>(a.part_o + pr * D)[q] = o;
      if (q == 0) a.part_ml[pr] = make_float2(top, sum);
    } else {
      const int at = r0 + r;
      const int64_t row = (static_cast<int64_t>(seq) * a.n_q + at / a.G) * a.h_q + kvh * a.G + at % a.G;
      const float inv = sum == 0.f ? 0.f : 1.f / sum;
      uint2 out;
      out.x = pack_bf16(o.x * inv, o.y * inv);
      out.y = pack_bf16(o.z * inv, o.w * inv);
      reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.g.O) + row * D)[q] = out;
      if (q == 0 && a.g.lse) a.g.lse[row] = sum == 0.f ? -INFINITY : (top + log2f(sum)) * 0.6931471805599453f;
    }
  }
}

// Joins the splits of every row: `warps` warps per row (1, 2, 4 or 8, by the
// number of splits), each every warps-th split.
template <int D, bool SEL>
__global__ void __launch_bounds__(256) cache_join_kernel(const CacheCfg a, const int warps) {
  constexpr int E = D / 32;   // dims per lane
  __shared__ float so[8][D];
  __shared__ float2 sml[8];
  // launched while the split kernel still runs: its results are complete after this
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int lane = threadIdx.x & 31, warp = threadIdx.x / 32, w = warp % warps;
  const int64_t item = (static_cast<int64_t>(blockIdx.x) * 8 + warp) / warps;
  const int64_t unit = item / a.rows;
  const int r = static_cast<int>(item % a.rows);
  const int kvh = static_cast<int>(unit % a.h_kv);
  const int tile = static_cast<int>(unit / a.h_kv % a.tiles);
  const int64_t seq = unit / a.h_kv / a.tiles;
  const int at = (SEL ? tile * a.G : tile * a.unit_rows) + r;
  const bool valid = seq < a.n_seq && at < a.n_q * a.G;
  float M = -INFINITY, l = 0.f, acc[E];
#pragma unroll
  for (int e = 0; e < E; ++e) acc[e] = 0.f;
  if (valid) {
    const float2* ml = a.part_ml + unit * a.splits * a.rows + r;
    const float* po = a.part_o + (unit * a.splits * a.rows + r) * D + lane * E;
    for (int s = w + warps * lane; s < a.splits; s += 32 * warps) M = fmaxf(M, ml[static_cast<int64_t>(s) * a.rows].x);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(0xFFFFFFFFu, M, o));
#pragma unroll 4
    for (int s = w; s < a.splits; s += warps) {
      const float2 x = ml[static_cast<int64_t>(s) * a.rows];
      const float f = M == -INFINITY ? 1.f : exp2f(x.x - M);
      const float* y = po + static_cast<int64_t>(s) * a.rows * D;
      l = fmaf(f, x.y, l);
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        const float2 v = *reinterpret_cast<const float2*>(y + e);
        acc[e] = fmaf(f, v.x, acc[e]);
        acc[e + 1] = fmaf(f, v.y, acc[e + 1]);
      }
    }
  }
  if (warps > 1) {
#pragma unroll
    for (int e = 0; e < E; ++e) so[warp][lane * E + e] = acc[e];
    if (lane == 0) sml[warp] = make_float2(M, l);
    __syncthreads();
    if (w != 0) return;
    for (int k = 1; k < warps; ++k) M = fmaxf(M, sml[warp + k].x);
    l = 0.f;
#pragma unroll
    for (int e = 0; e < E; ++e) acc[e] = 0.f;
    for (int k = 0; k < warps; ++k) {
      const float f = M == -INFINITY ? 1.f : exp2f(sml[warp + k].x - M);
      l = fmaf(f, sml[warp + k].y, l);
#pragma unroll
      for (int e = 0; e < E; ++e) acc[e] = fmaf(f, so[warp + k][lane * E + e], acc[e]);
    }
  }
  if (!valid) return;
  const int64_t row = (seq * a.n_q + at / a.G) * a.h_q + kvh * a.G + at % a.G;
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint32_t* out = reinterpret_cast<uint32_t*>(static_cast<__nv_bfloat16*>(a.g.O) + row * D + lane * E);
#pragma unroll
  for (int e = 0; e < E; e += 2) out[e / 2] = pack_bf16(acc[e] * inv, acc[e + 1] * inv);
  if (lane == 0 && a.g.lse) a.g.lse[row] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.6931471805599453f;
}

struct Split {
  int64_t units;
  int tiles, unit_rows, rows, splits;
};

Split split_of(const ssa_cache_attn_params& p) {
  Split s;
  const int G = p.h_q / p.h_kv;
  const bool sel = p.topk > 0;
  // A unit of 24 rows was tried for 17 to 24 (five drafts of four heads): 105 us
  // in place of 114 at d = 128, 133 in place of 128 at d = 64, at 255 registers.
  const int rows = sel ? G : p.n_q * G;
  s.unit_rows = rows <= 8 ? 8 : 16;
  s.tiles = sel ? p.n_q : (rows + s.unit_rows - 1) / s.unit_rows;
  s.rows = rows < s.unit_rows ? rows : s.unit_rows;
  s.units = static_cast<int64_t>(p.n_seq) * p.h_kv * s.tiles;
  int64_t pieces = static_cast<int64_t>(p.max_pages) * p.page / piece_keys(p.d);
  if (sel) {
    const int64_t most = (p.topk + p.window / p.page + 2) * static_cast<int64_t>(p.page / piece_keys(p.d));
    if (pieces > most) pieces = most;
  }
  // One wave of the blocks that run at a time when the units are few, down to
  // one piece per warp (a latency: a sequence of 1000 took 14 us at four pieces
  // per warp, 10 at one); else about four waves, so that ragged lengths even
  // out, with at least eight pieces per warp of the longest axis (16 sequences
  // of up to 4000, five drafts: 68 us at four, 54 at eight), four of selected
  // blocks or where eight would leave SMs idle (8 sequences of five drafts,
  // d = 64: 32 us at eight, 23 at four).
  const int64_t room = kBlocks * kSmCount;
  int64_t n = 1;
  if (s.units * 8 < room) {
    n = room / (s.units < 1 ? 1 : s.units);
    if (n > pieces / kWarps) n = pieces / kWarps;
  } else {
    n = (4 * room + s.units - 1) / s.units;
    if (sel) {
      // units of one size: the split that costs least, a block's set-up and
      // join counted as six pieces of a warp
      int64_t cost = INT64_MAX;
      for (int64_t k = 1; k <= 8; ++k) {
        const int64_t c = (s.units * k + room - 1) / room * (pieces + 6 * kWarps * k) * 840 / k;
        if (c < cost) { cost = c; n = k; }
      }
    }
    int64_t most = pieces / ((sel ? 4 : 8) * kWarps), fill = room / s.units;
    if (fill > pieces / (4 * kWarps)) fill = pieces / (4 * kWarps);
    if (most < fill) most = fill;
    if (n > most) n = most;
  }
  s.splits = static_cast<int>(n < 1 ? 1 : n);
  return s;
}

template <int D, bool SEL, int R>
cudaError_t run_cache_attn(const CacheCfg& a, int64_t units, const LaunchCtx& c) {
  using C = CacheShape<D>;
  cudaError_t e =
      cudaFuncSetAttribute(cache_attn_kernel<D, SEL, R>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  if (e != cudaSuccess) return e;
  if (units * a.splits > INT32_MAX) return cudaErrorInvalidValue;
  cache_attn_kernel<D, SEL, R><<<static_cast<unsigned>(units * a.splits), kWarps * 32, C::SMEM, c.stream>>>(a);
  note_launch();
  if ((e = cudaGetLastError()) != cudaSuccess || a.splits == 1) return e;
  int warps = 1;
  while (warps < 8 && warps * 4 < a.splits) warps *= 2;
  // its launch overlaps the end of the split kernel (it waits for it itself)
  cudaLaunchAttribute early;
  early.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  early.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3(static_cast<unsigned>((units * a.rows * warps + 7) / 8));
  cfg.blockDim = dim3(256);
  cfg.stream = c.stream;
  cfg.attrs = &early;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, cache_join_kernel<D, SEL>, a, warps);
  note_launch();
  return e;
}

template <int D>
cudaError_t pick_cache_attn(const CacheCfg& a, int64_t units, const LaunchCtx& c) {
  if (a.topk)
    return a.unit_rows == 8 ? run_cache_attn<D, true, 1>(a, units, c) : run_cache_attn<D, true, 2>(a, units, c);
  return a.unit_rows == 8 ? run_cache_attn<D, false, 1>(a, units, c) : run_cache_attn<D, false, 2>(a, units, c);
}

}  // namespace

size_t cache_attn_ws(const ssa_cache_attn_params& p) {
  const Split s = split_of(p);
  if (s.splits == 1) return 0;
  return static_cast<size_t>(s.units) * s.splits * s.rows * (p.d * 4 + 8);
}

cudaError_t launch_cache_attn(const ssa_cache_attn_params& p, const CacheAttnArgs& g, const LaunchCtx& c) {
  const Split s = split_of(p);
  CacheCfg a{};
  a.g = g;
  a.n_seq = p.n_seq; a.n_q = p.n_q; a.max_pages = p.max_pages; a.n_pages = p.n_pages; a.page = p.page;
  a.h_q = p.h_q; a.h_kv = p.h_kv; a.G = p.h_q / p.h_kv; a.topk = p.topk; a.window = p.window;
  a.tiles = s.tiles; a.unit_rows = s.unit_rows; a.rows = s.rows; a.splits = s.splits;
  a.scale_log2 = p.scale * 1.4426950408889634f;
  a.part_o = static_cast<float*>(g.ws);
  a.part_ml = reinterpret_cast<float2*>(a.part_o + static_cast<size_t>(s.units) * s.splits * s.rows * p.d);
  a.err = c.err;
  return p.d == 128 ? pick_cache_attn<128>(a, s.units, c) : pick_cache_attn<64>(a, s.units, c);
}

}  // namespace ssa
