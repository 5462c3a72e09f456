// The norm over a head and the rotation of its first dims, for a head held by
// d/8 neighbouring lanes of a warp, eight consecutive dims each.
//
//   y = x / sqrt(mean(x^2) + eps) * w,    (a, b) -> (a cos - b sin, b cos + a sin)
//
// with angle = position * freq.  Everything is float32 but the angle: a
// frequency is held as turns per position in 64-bit fixed point (2^64 = one
// turn), so that position * frequency wraps modulo one turn by itself and
// the angle of position 2^31 is as exact as that of position 1 (in float32
// the angle of position 10^6 is off by up to 0.03 rad).
#pragma once

#include <cuda_bf16.h>
#include <stdint.h>

#include "ssa.h"

namespace ssa {

// Turns per position, 64-bit fixed point.
__device__ __forceinline__ uint64_t phase_of(double freq) {
  double t = freq * 0.15915494309189535;   // 1 / (2 pi)
  t -= floor(t);
  return static_cast<uint64_t>(t * 18446744073709551616.0);   // saturates at one turn
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

// Eight consecutive elements of a row.
template <typename T>
struct Row8;
template <>
struct Row8<__nv_bfloat16> {
  uint4 v;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16* p, const float (&x)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Row8<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = *reinterpret_cast<const float4*>(p);
    b = *reinterpret_cast<const float4*>(p + 4);
  }
  __device__ __forceinline__ void get(float (&x)[8]) const {
    x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w;
    x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
  }
  static __device__ __forceinline__ void store(float* p, const float (&x)[8]) {
    *reinterpret_cast<float4*>(p) = make_float4(x[0], x[1], x[2], x[3]);
    *reinterpret_cast<float4*>(p + 4) = make_float4(x[4], x[5], x[6], x[7]);
  }
};

// What one lane needs of a position's rotation, for its eight dims 8*sub ..
// 8*sub + 7 of a head (sub: the lane's place in its row).  Half layout: the
// cos and signed sin of each dim and the lane that holds the partner dims
// (rot is a multiple of 16, so partners lie in one lane); pairs: four cos and
// sin.  Lanes past the rotated dims have cos 1, sin 0.
template <bool PRECISE>
struct Turn {
  float c[8], s[8];
  int partner;   // offset of the partner lane (half layout), 0 when none

  __device__ __forceinline__ void set(const uint64_t (&phase)[8], int sub, int rot, int layout, int32_t pos,
                                      float mscale) {
    partner = 0;
    if (8 * sub >= rot) {
#pragma unroll
      for (int i = 0; i < 8; ++i) { c[i] = 1.f; s[i] = 0.f; }
      return;
    }
    if (layout == SSA_ROPE_HALF) {
      const bool low = 16 * sub < rot;
      partner = low ? rot / 16 : -(rot / 16);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        turn_of<PRECISE>(phase[i], pos, c[i], s[i]);
        c[i] *= mscale;
        s[i] *= low ? -mscale : mscale;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        turn_of<PRECISE>(phase[i], pos, c[i], s[i]);
        c[i] *= mscale;
        s[i] *= mscale;
      }
    }
  }

  // Rotates the row's dims in place; all lanes of the warp take part (those
  // past the rotated dims keep theirs, infinities too).
  __device__ __forceinline__ void apply(float (&x)[8], int layout, int lane, bool rotated) const {
    if (layout == SSA_ROPE_HALF) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float y = __shfl_sync(0xFFFFFFFFu, x[i], lane + partner);
        if (rotated) x[i] = fmaf(y, s[i], x[i] * c[i]);
      }
    } else if (rotated) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float a = x[2 * i], b = x[2 * i + 1];
        x[2 * i] = fmaf(-b, s[i], a * c[i]);
        x[2 * i + 1] = fmaf(a, s[i], b * c[i]);
      }
    }
  }
};

// The phases of a lane's dims.
__device__ __forceinline__ void lane_phases(const double* freq, int sub, int rot, int layout, uint64_t (&phase)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) phase[i] = 0;
  if (8 * sub >= rot) return;
  if (layout == SSA_ROPE_HALF) {
    const int i0 = 8 * sub - (16 * sub < rot ? 0 : rot / 2);
#pragma unroll
    for (int i = 0; i < 8; ++i) phase[i] = phase_of(__ldg(freq + i0 + i));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) phase[i] = phase_of(__ldg(freq + 4 * sub + i));
  }
}

// x / sqrt(mean(x^2) + eps) * w over the LPR lanes of a row.
template <int LPR>
__device__ __forceinline__ void norm_row(float (&x)[8], const float (&w)[8], float eps) {
  float q = 0.f;
#pragma unroll
  for (int i = 0; i < 8; ++i) q = fmaf(x[i], x[i], q);
#pragma unroll
  for (int o = 1; o < LPR; o <<= 1) q += __shfl_xor_sync(0xFFFFFFFFu, q, o);
  const float r = 1.f / sqrtf(q * (1.f / (8 * LPR)) + eps);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = x[i] * r * w[i];
}

__device__ __forceinline__ void lane_weights(const float* w, int sub, float (&x)[8]) {
  Row8<float> r;
  if (w) {
    r.load(w + 8 * sub);
    r.get(x);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 1.f;
  }
}

}  // namespace ssa
