// mx_pack.hip -- MXFP4 quantise+pack and unpack kernels (gfx950).
//
// Format (OCP Microscaling Formats specification 1.0, MXFP4): blocks of 32
// values along K share one power of two 2^(s - 127), each value is an e2m1
// code {0, .5, 1, 1.5, 2, 3, 4, 6} with a sign bit; s = 255 is NaN.  Quantising a
// block: s - 127 = floor(log2(max |w|)) - 2, held to [-127, 127] (2 is the exponent
// of the largest element, 6), code = w / 2^(s - 127) rounded to nearest, ties to
// the even code, beyond 6 to 6.  floor(log2) is the exponent field of the
// largest magnitude, and the rounding is the hardware's conversion, which
// divides by the scale's power of two and rounds so (checked against the rule
// over every tie and the extreme scales).
#include "nf4_check.h"
#include "nf4_device.h"

namespace nf4 {

typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t dpp_max_quad(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xf, 0xf, false);
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xf, 0xf, false);
  return v > o ? v : o;
}

// One thread per 8 consecutive values (one 32-bit word of codes), four threads
// per block, so loads and stores are whole lines.  Bound by memory.  fp32, weights, is read
// past the caches; bf16, an activation that a kernel has just written, is not.  A NaN or
// infinity anywhere in the block is seen as exponent 255 of the largest magnitude's bits,
// which is also the scale byte it then gets.  Measured, 28672 x 4096 fp32: 97 us, 5.5 TB/s;
// 4096 x 4096 bf16: 13 us, 9.5 where it is still in the caches.
template <typename T>
__global__ void __launch_bounds__(256) mx_pack_kernel(const T *__restrict__ W, int64_t nwords,
                                                      uint32_t *__restrict__ codes,
                                                      uint8_t *__restrict__ scales,
                                                      int32_t *__restrict__ status) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= nwords) return;  // whole blocks of four threads leave together
  uint32_t word = 0;
  uint32_t byte;
  if constexpr (sizeof(T) == 4) {
    const f32x4 *p = reinterpret_cast<const f32x4 *>(W) + 2 * i;
    const f32x4 a = __builtin_nontemporal_load(p), b = __builtin_nontemporal_load(p + 1);
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const uint32_t x = __float_as_uint(a[j]) & 0x7fffffffu, y = __float_as_uint(b[j]) & 0x7fffffffu;
      m = max(m, max(x, y));
    }
    const uint32_t ex = dpp_max_quad(m) >> 23;
    byte = ex == 255u ? 255u : ex > 2u ? ex - 2u : 0u;
    const float s = __uint_as_float(byte << 23);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, a[0], a[1], s, 0);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, a[2], a[3], s, 1);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, b[0], b[1], s, 2);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(word, b[2], b[3], s, 3);
  } else {
    const u32x4 v = reinterpret_cast<const u32x4 *>(W)[i];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = max(m, max(v[j] & 0x7fffu, (v[j] >> 16) & 0x7fffu));
    const uint32_t ex = dpp_max_quad(m) >> 7;
    byte = ex == 255u ? 255u : ex > 2u ? ex - 2u : 0u;
    const float s = __uint_as_float(byte << 23);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, __builtin_bit_cast(bf16x2, (uint32_t)v[0]), s, 0);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, __builtin_bit_cast(bf16x2, (uint32_t)v[1]), s, 1);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, __builtin_bit_cast(bf16x2, (uint32_t)v[2]), s, 2);
    word = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(word, __builtin_bit_cast(bf16x2, (uint32_t)v[3]), s, 3);
  }
  const bool bad = byte == 255u;
  codes[i] = bad ? 0u : word;
  if ((threadIdx.x & 3) == 0) {
    scales[i >> 2] = (uint8_t)byte;
    if (bad && status) atomicOr(status, NF4_PACK_NONFINITE);
  }
}

__global__ void mx_clear_status_kernel(int32_t *status) { *status = 0; }

// One thread per word of codes -> 8 values; the conversion multiplies by the block's
// power of two (255: NaN).  Bound by memory: 28672 x 4096 to fp32 95-104 us, 5.1-5.6 TB/s,
// to bf16 55 us, 5.4 TB/s.
template <typename T>
__global__ void __launch_bounds__(256) mx_unpack_kernel(const uint32_t *__restrict__ codes,
                                                        const uint8_t *__restrict__ scales,
                                                        int64_t nwords, T *__restrict__ out) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (i >= nwords) return;
  const uint32_t w = codes[i];
  const float s = __uint_as_float((uint32_t)scales[i >> 2] << 23);
  if constexpr (sizeof(T) == 4) {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, s, 3);
    f32x4 *o = reinterpret_cast<f32x4 *>(out) + 2 * i;
    o[0] = f32x4{a[0], a[1], b[0], b[1]};
    o[1] = f32x4{c[0], c[1], d[0], d[1]};
  } else {
    u32x4 o;
    o[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
    o[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
    o[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
    o[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
    reinterpret_cast<u32x4 *>(out)[i] = o;
  }
}

}  // namespace nf4

extern "C" {

int nf4_mx_pack(const void *W, int dtype, int64_t N, int64_t K, uint8_t *codes, uint8_t *scales,
                int32_t *dev_status, void *stream) {
  if (!W || !codes || !scales || !nf4::known_dtype(dtype)) return NF4_EINVAL;
  if (int r = nf4::check_mx_shape(N, K)) return r;
  if (!nf4::aligned_to(W, 16) || !nf4::aligned_to(codes, 4) ||
      (dev_status && !nf4::aligned_to(dev_status, 4)))
    return NF4_EALIGN;
  if (int r = nf4::device_status()) return r;
  hipStream_t s = (hipStream_t)stream;
  if (dev_status) {
    hipLaunchKernelGGL(nf4::mx_clear_status_kernel, dim3(1), dim3(1), 0, s, dev_status);
    if (hipGetLastError() != hipSuccess) return NF4_ELAUNCH;
  }
  const int64_t nwords = N * (K / 8);
  const dim3 grid((unsigned)((nwords + 255) / 256));
  if (dtype == NF4_F32)
    hipLaunchKernelGGL(nf4::mx_pack_kernel<float>, grid, dim3(256), 0, s, (const float *)W, nwords,
                       (uint32_t *)codes, scales, dev_status);
  else
    hipLaunchKernelGGL(nf4::mx_pack_kernel<uint16_t>, grid, dim3(256), 0, s, (const uint16_t *)W,
                       nwords, (uint32_t *)codes, scales, dev_status);
  return nf4::launch_status(hipGetLastError());
}

int nf4_mx_unpack(const uint8_t *codes, const uint8_t *scales, int64_t N, int64_t K, void *W_out,
                  int dtype, void *stream) {
  if (!codes || !scales || !W_out || !nf4::known_dtype(dtype)) return NF4_EINVAL;
  if (int r = nf4::check_mx_shape(N, K)) return r;
  if (!nf4::aligned_to(codes, 4) || !nf4::aligned_to(W_out, 16)) return NF4_EALIGN;
  if (int r = nf4::device_status()) return r;
  hipStream_t s = (hipStream_t)stream;
  const int64_t nwords = N * (K / 8);
  const dim3 grid((unsigned)((nwords + 255) / 256));
  if (dtype == NF4_F32)
    hipLaunchKernelGGL(nf4::mx_unpack_kernel<float>, grid, dim3(256), 0, s,
                       (const uint32_t *)codes, scales, nwords, (float *)W_out);
  else
    hipLaunchKernelGGL(nf4::mx_unpack_kernel<uint16_t>, grid, dim3(256), 0, s,
                       (const uint32_t *)codes, scales, nwords, (uint16_t *)W_out);
  return nf4::launch_status(hipGetLastError());
}

}  // extern "C"
