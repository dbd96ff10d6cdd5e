// mx_grad.hip -- gradient of the grouped MXFP4 product in its rows (gfx950):
//   dX[i][k] = sum_n dY[i][n] * v(e(i), n, k),  v = element * 2^(scale - 127)
// (the packed matrices are frozen).  The sum runs over the packed rows n, across the
// direction in which codes lie, so fragments are transposed in registers: a
// lane loads one word of codes (8 consecutive k) of 8 consecutive rows n, decodes
// each with its row's block scale into four bf16 pairs along k, and joins the
// pairs of neighbouring rows (v_perm_b32) into pairs along n.  That gives the A
// fragments of 8 MFMAs (16x16x32): MFMA j has the columns k0 + 8 i + j, i = 0 .. 15.
// D: lane l holds row l % 16 and columns k0 + 8 (4 (l / 16) + r) + j, so the eight
// tiles of a lane are 8 consecutive outputs.
#include "mx_device.h"
#include "nf4_check.h"

namespace nf4 {
namespace mx {

struct GradArgs {
  const uint8_t *codes;
  const uint8_t *scales;
  const uint16_t *dY;
  const int32_t *offsets;
  void *dX;
  int64_t R;
  int E, N, K;
  Grid grid;
};

// 16 MF rows x 512 columns a workgroup (128 columns a wave); dY goes through LDS in
// stages of 128 n, laid out as the rows of the forward product.
template <int MF, typename OUT>
__global__ void __launch_bounds__(256, 2) mx_grad_kernel(GradArgs p) {
  constexpr int BM = 16 * MF;
  __shared__ __attribute__((aligned(1024))) uint8_t xs[2][BM * 256];
  int slot, block;
  if (!grid_item(p.grid, &slot, &block)) return;
  const RowTile t = find_tile(p.offsets, p.E, p.R, slot, BM);
  if (t.rows <= 0) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int k0 = block * 512 + wave * 128;
  f32x4_t acc[8][MF];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int r = 0; r < MF; ++r) acc[j][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  if (t.e >= 0) {
    const int kb = p.K >> 5, kc = p.K >> 1;
    const int64_t first = (int64_t)t.e * p.N;
    const __amdgpu_buffer_rsrc_t crs = buffer(p.codes + first * kc, (int64_t)p.N * kc);
    const __amdgpu_buffer_rsrc_t srs = buffer(p.scales + first * kb, (int64_t)p.N * kb);
    const __amdgpu_buffer_rsrc_t yrs =
        buffer(p.dY + (int64_t)t.row0 * p.N, (int64_t)t.rows * p.N * 2);
    const int stages = (p.N + 127) >> 7;
    const int xrow = wave * 4 + q;
    const int xchunk = l16 ^ (xrow & 15);
    const auto load_y = [&](int buf, int s) {
      const int out = s * 128 + xchunk * 8 < p.N ? 0 : kOutside;
#pragma unroll
      for (int i = 0; i < MF; ++i)
        load_lds16(yrs, &xs[buf][(i * 16 + wave * 4) * 256],
                   ((i * 16 + xrow) * p.N * 2 + s * 256 + xchunk * 16) | out);
    };
    // columns past K: another row's codes, their outputs are not stored
    const int kw = (k0 >> 1) + l16 * 4, ks = (k0 >> 5) + (l16 >> 2);
    uint32_t cw[8], sb[8];
    const auto load_w = [&](int n) {  // rows n + 8 q .. + 7; past N: outside the buffer
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int r = n + q * 8 + i;
        const int out = r < p.N ? 0 : kOutside;
        cw[i] = __builtin_amdgcn_raw_buffer_load_b32(crs, (r * kc + kw) | out, 0, 0);
        sb[i] = __builtin_amdgcn_raw_buffer_load_b8(srs, (r * kb + ks) | out, 0, 0);
      }
    };
    load_y(0, 0);
    load_w(0);
    for (int s = 0; s < stages; ++s) {
      lds_loads_done();
      __syncthreads();
      if (s + 1 < stages) load_y((s + 1) & 1, s + 1);
      const uint8_t *x = xs[s & 1] + l16 * 256;
#pragma unroll
      for (int i4 = 0; i4 < 4; ++i4) {
        u32x4_t d[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] = decode8(cw[i], scale_of(sb[i]));
        load_w(s * 128 + (i4 + 1) * 32);
        u32x4_t b[MF];
#pragma unroll
        for (int r = 0; r < MF; ++r)
          b[r] = *reinterpret_cast<const u32x4_t *>(x + r * 4096 + (((i4 * 4 + q) ^ l16) * 16));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          u32x4_t a;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            a[i] = __builtin_amdgcn_perm(d[2 * i + 1][j >> 1], d[2 * i][j >> 1],
                                         (j & 1) ? 0x07060302u : 0x05040100u);
#pragma unroll
          for (int r = 0; r < MF; ++r) acc[j][r] = mfma16(a, b[r], acc[j][r]);
        }
      }
    }
  }
  OUT *X = reinterpret_cast<OUT *>(p.dX);
#pragma unroll
  for (int r = 0; r < MF; ++r) {
    const int m = r * 16 + l16;
    if (m >= t.rows) continue;
    OUT *row = X + (int64_t)(t.row0 + m) * p.K;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + 8 * (4 * q + i);
      if (k >= p.K) continue;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = acc[j][r][i];
      if constexpr (sizeof(OUT) == 4) {
        *reinterpret_cast<f32x4_t *>(row + k) = f32x4_t{v[0], v[1], v[2], v[3]};
        *reinterpret_cast<f32x4_t *>(row + k + 4) = f32x4_t{v[4], v[5], v[6], v[7]};
      } else {
        u32x4_t o;
#pragma unroll
        for (int h = 0; h < 4; ++h) o[h] = bf16_bits(v[2 * h]) | (bf16_bits(v[2 * h + 1]) << 16);
        *reinterpret_cast<u32x4_t *>(row + k) = o;
      }
    }
  }
}

template <int MF>
static hipError_t launch_grad(GradArgs &a, int out_dtype, hipStream_t s) {
  a.grid = make_grid(slots_for(a.R, a.E, true, 16 * MF), (a.K + 511) / 512, 8);
  const int64_t n = grid_size(a.grid);
  if (n * 256 >= (int64_t(1) << 32)) return hipErrorInvalidValue;
  if (out_dtype == NF4_F32)
    hipLaunchKernelGGL((mx_grad_kernel<MF, float>), dim3((unsigned)n), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((mx_grad_kernel<MF, uint16_t>), dim3((unsigned)n), dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace mx
}  // namespace nf4

extern "C" {

int nf4_mx_gemm_grouped_grad(const uint8_t *codes, const uint8_t *scales, int64_t E, int64_t N,
                             int64_t K, const uint16_t *dY, const int32_t *offsets, int64_t R,
                             void *dX, int out_dtype, void *stream) {
  if (E < 1 || R < 0 || !codes || !scales || !offsets || (R > 0 && (!dY || !dX)) ||
      !nf4::known_dtype(out_dtype))
    return NF4_EINVAL;
  if (int r = nf4::check_mx_shape(N, K)) return r;
  if (N % 8 != 0) return NF4_EINVAL;
  if (E > NF4_MOE_MAX_E || R >= (int64_t(1) << 26) || N > (int64_t(1) << 23)) return NF4_ERANGE;
  if (!nf4::aligned_to(codes, 16) || !nf4::aligned_to(dY, 16) || !nf4::aligned_to(dX, 16) ||
      !nf4::aligned_to(offsets, 4))
    return NF4_EALIGN;
  if (int r = nf4::device_status()) return r;
  if (R == 0) return NF4_OK;
  nf4::mx::GradArgs a{codes, scales, dY, offsets, dX, R, (int)E, (int)N, (int)K, {}};
  return nf4::launch_status(nf4::mx::launch_grad<4>(a, out_dtype, (hipStream_t)stream));
}

}  // extern "C"
