// mx_act.h -- activations of the fused MXFP4 products and their derivatives (gfx950), in
// fp32, and the passage of a tile's sums through LDS to the code that applies them.
//   silu(z)      = z s(z),  s the logistic function; gates swiglu
//   gelu(z)      = z P(z),  P the normal distribution function = erfc(-z / sqrt 2) / 2
//   gelu_tanh(z) = z (1 + tanh u) / 2 = z s(2 u), u = sqrt(2 / pi) (z + 0.044715 z^3); gates geglu
// Written by s and erfc no difference of nearly equal numbers is taken: the error is within
// 2^-20 |z| everywhere.  (Each step rounds by 2^-24 or, v_exp, v_rcp and erfc, up to 2^-20 of
// its value at most; an error d of the exponent moves s by s (1 - s) d, and |x| s (1 - s) < 0.23.)
#pragma once

#include "mx_device.h"
#include "nf4_check.h"

namespace nf4 {
namespace mx {

inline bool known_act(int act) { return act >= NF4_ACT_NONE && act <= NF4_ACT_GEGLU; }
inline bool is_gated(int act) { return act == NF4_ACT_SWIGLU || act == NF4_ACT_GEGLU; }

// s(z): z = -inf gives 0, inf gives 1; v_rcp_f32 is within one unit.
__device__ __forceinline__ float logistic(float z) { return __builtin_amdgcn_rcpf(1.f + __expf(-z)); }

constexpr float kTanhIn = 1.5957691216f;  // 2 sqrt(2 / pi)
constexpr float kTanhCube = 0.044715f;

__device__ __forceinline__ float act_value(int act, float z) {
  switch (act) {
    case NF4_ACT_RELU: return z < 0.f ? 0.f : z;  // NaN stays
    case NF4_ACT_SILU:
    case NF4_ACT_SWIGLU: return z * logistic(z);
    case NF4_ACT_GELU: return 0.5f * z * erfcf(z * -0.70710678119f);
    case NF4_ACT_GELU_TANH:
    case NF4_ACT_GEGLU: return z * logistic(kTanhIn * (z + kTanhCube * z * z * z));
    default: return z;
  }
}

// The derivative, within 2^-20.  s (1 - s) = e / (1 + e)^2 with e = exp(-|x|) loses nothing where
// s nears 1 and overflows nowhere; what it is multiplied with is taken at |z| <= 30, beyond
// which it is 0 and the powers of z would meet it as infinity.
struct Logistic {
  float s, slope;
};
__device__ __forceinline__ Logistic logistic_slope(float x) {
  const float e = __expf(-fabsf(x)), r = __builtin_amdgcn_rcpf(1.f + e);
  return {x < 0.f ? e * r : r, e * r * r};
}
__device__ __forceinline__ float act_slope(int act, float z) {
  const float c = __builtin_amdgcn_fmed3f(z, -30.f, 30.f);
  switch (act) {
    case NF4_ACT_RELU: return z > 0.f ? 1.f : z <= 0.f ? 0.f : z;
    case NF4_ACT_SILU:
    case NF4_ACT_SWIGLU: {
      const Logistic l = logistic_slope(z);
      return l.s + c * l.slope;
    }
    case NF4_ACT_GELU:
      return 0.5f * erfcf(z * -0.70710678119f) + 0.39894228040f * c * __expf(-0.5f * z * z);
    case NF4_ACT_GELU_TANH:
    case NF4_ACT_GEGLU: {
      const Logistic l = logistic_slope(kTanhIn * (z + kTanhCube * z * z * z));
      return l.s + c * l.slope * (kTanhIn * (1.f + 3.f * kTanhCube * c * c));
    }
    default: return 1.f;
  }
}

// Four values under one (uniform) branch.
#define NF4_ACT_CASE(F, A) \
  case A: return f32x4_t{F(A, z[0]), F(A, z[1]), F(A, z[2]), F(A, z[3])};
#define NF4_ACT_CASES(F)                                         \
  switch (act) {                                                 \
    NF4_ACT_CASE(F, NF4_ACT_RELU) NF4_ACT_CASE(F, NF4_ACT_GELU) \
    case NF4_ACT_SWIGLU:                                         \
    NF4_ACT_CASE(F, NF4_ACT_SILU)                                \
    case NF4_ACT_GEGLU:                                          \
    NF4_ACT_CASE(F, NF4_ACT_GELU_TANH)                           \
    default: return f32x4_t{F(NF4_ACT_NONE, z[0]), F(NF4_ACT_NONE, z[1]), F(NF4_ACT_NONE, z[2]), F(NF4_ACT_NONE, z[3])}; \
  }
__device__ __forceinline__ f32x4_t act_values(int act, f32x4_t z) { NF4_ACT_CASES(act_value) }
__device__ __forceinline__ f32x4_t act_slopes(int act, f32x4_t z) { NF4_ACT_CASES(act_slope) }
#undef NF4_ACT_CASES
#undef NF4_ACT_CASE

// The tile's sums, row by row, in LDS: take(z, m0, rows) gets rows m0 .. m0 + rows - 1 of
// 16 NF WV columns (kPitch floats apart, 16 bytes more than the columns so that the 16 rows
// that a wave writes at once fall into different banks) and runs in all threads of the
// workgroup.  Through LDS so that the threads read and write whole lines of what an
// epilogue adds and keeps, and its code is there once, not per register.
template <int MF, int NF, int WV, int KG, int BYTES>
struct TileRows {
  static constexpr int kCols = 16 * NF * WV, kPitch = kCols + 4;
  static constexpr int kPass = 16 * MF * kPitch * 4 <= BYTES ? MF : MF / 2;
  static_assert(16 * kPass * kPitch * 4 <= BYTES && MF % kPass == 0 && MF / kPass <= 2, "half a tile fits");
  template <class TAKE>
  static __device__ __forceinline__ void each(int wave, int kg, const f32x4_t (&acc)[NF][MF], uint8_t *lds,
                                              const TAKE &take) {
    float *const z = reinterpret_cast<float *>(lds);
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
#pragma unroll 1
    for (int h = 0; h < MF / kPass; ++h) {
      __syncthreads();
      if (KG == 1 || kg == 0) {
#pragma unroll
        for (int c = 0; c < NF; ++c)
#pragma unroll
          for (int r = 0; r < kPass; ++r)
            *reinterpret_cast<f32x4_t *>(z + (r * 16 + l16) * kPitch + (wave * NF + c) * 16 + q * 4) =
                kPass == MF || h == 0 ? acc[c][r] : acc[c][kPass == MF ? r : kPass + r];
      }
      __syncthreads();
      take(z, h * kPass * 16, kPass * 16);
    }
  }
};

}  // namespace mx
}  // namespace nf4
