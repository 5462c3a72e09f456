// The norm over a head and the rotation of its first dims, for a head held by
// d/8 neighbouring lanes of a warp, eight dims each.
//
//   y = x / sqrt(mean(x^2) + eps) * w,    (a, b) -> (a cos - b sin, b cos + a sin)
//
// with angle = position * freq.  Everything is float32 but the angle: a
// frequency is held as turns per position in 64-bit fixed point (2^64 = one
// turn), so that position * frequency wraps modulo one turn by itself and
// the angle of position 2^31 is as exact as that of position 1 (in float32
// the angle of position 10^6 is off by up to 0.03 rad).
//
// A lane's eight dims are two runs of four.  In the half layout the lanes of
// the rotated part take dims 4 l .. and rot/2 + 4 l .., so that both dims of
// a pair are in one lane: four angles per lane and no exchange (with eight
// consecutive dims per lane it was eight angles and eight shuffles, and the
// rotation of 128K tokens 745 us).  Elsewhere the two runs are neighbours.
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "common.cuh"
#include "ssa.h"

namespace ssa {

// Turns per position, 64-bit fixed point: freq / (2 pi) modulo one to 2^-63 (for
// |freq| below 2^38), from the rounded product and what it leaves: alone, its
// rounding of 2^-53 times the frequency would grow with the position.  Adding
// 3 * 2^51 rounds to a whole number in the sum's low bits, without the slow conversions.
__device__ __forceinline__ uint64_t phase_of(double freq) {
  constexpr double hi = 0.15915494309189535, lo = -9.839338337591243e-18;   // 1 / (2 pi) to 107 bits
  constexpr double whole = 6755399441055744.0, two32 = 4294967296.0;
  const double t = freq * hi, rest = fma(freq, lo, fma(freq, hi, -t));
  const double x = (t - ((t + whole) - whole)) * two32;
  const double u = x + whole;                                                        // the upper 32 bits
  const double v = fma(rest, two32 * two32, (x - (u - whole)) * two32) + whole;      // the lower ones, signed
  return (static_cast<uint64_t>(__double2loint(u)) << 32) +
         static_cast<uint64_t>(__double_as_longlong(v) - __double_as_longlong(whole));
}

// cos and sin of position * frequency.  PRECISE: to float32's rounding;
// else by the fast approximations, whose 2^-21 absolute error in [-pi, pi]
// is far below the rounding of a bf16 or e4m3 result (2^-9, 2^-4).
template <bool PRECISE>
__device__ __forceinline__ void turn_of(uint64_t phase, int32_t pos, float& c, float& s) {
  const uint64_t a = phase * static_cast<uint64_t>(static_cast<int64_t>(pos));
  const int32_t turns = static_cast<int32_t>((a + 0x80000000ull) >> 32);   // turns * 2^32, in [-1/2, 1/2)
  if (PRECISE) {
    sincospif(static_cast<float>(turns) * 4.656612873077393e-10f, &s, &c);   // 2^-31
  } else {
    const float x = static_cast<float>(turns) * 1.4629180792671596e-9f;      // 2 pi 2^-32
    c = __cosf(x);
    s = __sinf(x);
  }
}

// Where a lane's dims lie: runs of four at `a` and `b`.
struct LaneDims {
  int a, b;
  bool rotated;   // this lane's dims turn
  bool half;      // the layout, the same for all lanes
  __device__ __forceinline__ LaneDims(int sub, int rot, int layout) {
    rotated = 8 * sub < rot;
    half = layout == SSA_ROPE_HALF;
    a = rotated && half ? 4 * sub : 8 * sub;
    b = rotated && half ? 4 * sub + rot / 2 : 8 * sub + 4;
  }
  // The lane's four phases: pairs (a + i, b + i), or (a, a + 1), (a + 2, a + 3), (b, b + 1), (b + 2, b + 3);
  // each computed once per block (every thread calls),
  __device__ __forceinline__ void block_phases(const double* freq, int rot, uint64_t (&all)[64], int sub,
                                               uint64_t (&phase)[4]) const {
    if (static_cast<int>(threadIdx.x) < rot / 2) all[threadIdx.x] = phase_of(__ldg(freq + threadIdx.x));
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i) phase[i] = rotated ? all[4 * sub + i] : 0;
  }
  // or, for a head of D dims, once per warp (every lane calls).
  template <int D>
  __device__ __forceinline__ void warp_phases(const double* freq, int rot, int sub, uint64_t (&phase)[4]) const {
    constexpr int N = D / 64;   // phases computed by a lane
    const int lane = threadIdx.x & 31;
    uint64_t own[N];
#pragma unroll
    for (int k = 0; k < N; ++k) own[k] = N * lane + k < rot / 2 ? phase_of(__ldg(freq + N * lane + k)) : 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint64_t p = __shfl_sync(0xFFFFFFFFu, own[i % N], (4 * sub + i) / N & 31);
      phase[i] = rotated ? p : 0;
    }
  }
};

// Four consecutive elements.
template <typename T>
struct Run4;
template <>
struct Run4<__nv_bfloat16> {
  uint2 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint2*>(p); }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = __uint_as_float(v.x << 16);
    x[1] = __uint_as_float(v.x & 0xFFFF0000u);
    x[2] = __uint_as_float(v.y << 16);
    x[3] = __uint_as_float(v.y & 0xFFFF0000u);
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* x) {
    const __nv_bfloat162 l = __floats2bfloat162_rn(x[0], x[1]), h = __floats2bfloat162_rn(x[2], x[3]);
    *reinterpret_cast<uint2*>(p) = make_uint2(*reinterpret_cast<const uint32_t*>(&l), *reinterpret_cast<const uint32_t*>(&h));
  }
};
template <>
struct Run4<float> {
  float4 v;
  __device__ __forceinline__ void load(const float* p) { v = *reinterpret_cast<const float4*>(p); }
  __device__ __forceinline__ void get(float* x) const {
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  }
  static __device__ __forceinline__ void store(float* p, const float* x) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
  }
};

// A lane's eight dims of a head.
template <typename T>
struct Row8 {
  Run4<T> a, b;
  __device__ __forceinline__ void load(const T* row, const LaneDims& at) {
    a.load(row + at.a);
    b.load(row + at.b);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    a.get(x);
    b.get(x + 4);
  }
  static __device__ __forceinline__ void store(T* row, const LaneDims& at, const float (&x)[8]) {
    Run4<T>::store(row + at.a, x);
    Run4<T>::store(row + at.b, x + 4);
  }
};

__device__ __forceinline__ void lane_weights(const float* w, const LaneDims& at, float (&x)[8]) {
  if (w) {
    Row8<float> r;
    r.load(w, at);
    r.get(x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 1.f;
  }
}

// cos and sin of a lane's four pairs at a position, times mscale.
struct Angles {
  float c[4], s[4];
  template <bool PRECISE>
  __device__ __forceinline__ void set(const LaneDims& at, const uint64_t (&phase)[4], int32_t pos, float mscale) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      c[i] = 1.f;
      s[i] = 0.f;
      if (at.rotated) {
        turn_of<PRECISE>(phase[i], pos, c[i], s[i]);
        c[i] *= mscale;
        s[i] *= mscale;
      }
    }
  }
  // Turns a row's dims in place, two pairs at a time; a dim that does not turn
  // takes nothing from its neighbour, infinities neither.
  __device__ __forceinline__ void turn(const LaneDims& at, float (&x)[8]) const {
    const uint64_t minus = pair(-1.f, -1.f);
    if (!at.rotated) return;
    if (at.half) {
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        const uint64_t a = pair(x[i], x[i + 1]), b = pair(x[i + 4], x[i + 5]);
        const uint64_t co = pair(c[i], c[i + 1]), si = pair(s[i], s[i + 1]);
        unpair(fma2(mul2(b, si), minus, mul2(a, co)), x[i], x[i + 1]);
        unpair(fma2(a, si, mul2(b, co)), x[i + 4], x[i + 5]);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = fmaf(-b, s[i], a * c[i]);
        x[2 * i + 1] = fmaf(a, s[i], b * c[i]);
      }
    }
  }
};

// x[i] *= w[i], x[i] *= f.
__device__ __forceinline__ void scale_row(float (&x)[8], const float (&w)[8]) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) unpair(mul2(pair(x[i], x[i + 1]), pair(w[i], w[i + 1])), x[i], x[i + 1]);
}
__device__ __forceinline__ void scale_row(float (&x)[8], float f) {
#pragma unroll
  for (int i = 0; i < 8; i += 2) unpair(mul2(pair(x[i], x[i + 1]), pair(f, f)), x[i], x[i + 1]);
}

// 1 / sqrt(mean(x^2) + eps) over the LPR lanes of a row.
template <int LPR>
__device__ __forceinline__ float norm_factor(const float (&x)[8], float eps) {
  uint64_t q2 = mul2(pair(x[0], x[1]), pair(x[0], x[1]));
#pragma unroll
  for (int i = 2; i < 8; i += 2) q2 = fma2(pair(x[i], x[i + 1]), pair(x[i], x[i + 1]), q2);
  float q, p;
  unpair(q2, q, p);
  q += p;
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
  return rsqrtf(fmaf(q, 1.f / (8 * LPR), eps));
}

}  // namespace ssa
