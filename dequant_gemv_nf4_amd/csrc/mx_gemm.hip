// mx_gemm.hip -- products of bf16 rows with packed MXFP4 matrices, dense and
// grouped by expert (gfx950):
//   Y[i][n] = sum_k X[i][k] * v(e(i), n, k),  v = element * 2^(scale - 127).
// v is exact in bf16, so the weights are decoded straight into matrix-core
// fragments (two values an instruction) and every product is exact in fp32.
//
// Fragments (v_mfma_f32_16x16x32_bf16, A = weights, B = rows): a step is 128 k.
// Lane l holds weight row n = l % 16 and the 16 bytes of block q = l / 16, i.e.
// k = 32 q .. 32 q + 31 of the step; MFMA j of the four takes k = 32 q + 8 j ..
// + 7 of both operands, so a code word, a block scale and 16 bytes of X line up
// without any shuffle.  D: lane l holds row i = l % 16, columns 4 (l / 16) .. + 3,
// stored as one vector.
#include "mx_device.h"
#include "nf4_check.h"

namespace nf4 {
namespace mx {

struct Args {
  const uint8_t *codes;
  const uint8_t *scales;
  const uint16_t *X;
  const int32_t *offsets;  // null: dense
  void *Y;
  int64_t R;
  int E, N, K;
  Grid grid;
};

// ------------------------------------------------------------ few rows ----
// A workgroup owns 16 CT columns x 16 RT rows; its NW waves take steps w, w + NW,
// ... of K and add their tiles through LDS in wave order.  Weights come from HBM
// once, X from the caches.
template <int RT, int CT, int NW, typename OUT>
__global__ void __launch_bounds__(64 * NW) mx_rows_kernel(Args p) {
  __shared__ f32x4_t part[NW][RT * CT][64];
  int slot, block;
  if (!grid_item(p.grid, &slot, &block)) return;
  const RowTile t = find_tile(p.offsets, p.E, p.R, slot, 16 * RT);
  if (t.rows <= 0) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int n0 = block * 16 * CT;
  const int cols = min(16 * CT, p.N - n0);
  f32x4_t acc[RT][CT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[r][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  if (t.e >= 0) {
    const int kb = p.K >> 5;  // blocks per row
    const int64_t first = (int64_t)t.e * p.N + n0;
    const __amdgpu_buffer_rsrc_t crs = buffer(p.codes + first * (p.K >> 1), (int64_t)cols * (p.K >> 1));
    const __amdgpu_buffer_rsrc_t srs = buffer(p.scales + first * kb, (int64_t)cols * kb);
    const __amdgpu_buffer_rsrc_t xrs =
        buffer(p.X + (int64_t)t.row0 * p.K, (int64_t)t.rows * p.K * 2);
    const int steps = (kb + 3) >> 2;
    constexpr int U = RT * CT >= 4 ? 1 : 2;  // steps whose loads are in flight together
    for (int s0 = wave; s0 < steps; s0 += NW * U) {
      u32x4_t cw[U][CT], xw[U][RT][4];
      uint32_t sb[U][CT];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int b = (s0 + u * NW) * 4 + q;
        const int out = b < kb ? 0 : kOutside;
#pragma unroll
        for (int c = 0; c < CT; ++c) {
          const int n = c * 16 + l16;
          cw[u][c] = __builtin_amdgcn_raw_buffer_load_b128(crs, (n * (p.K >> 1) + b * 16) | out, 0,
                                                           kLoadStream);
          sb[u][c] = __builtin_amdgcn_raw_buffer_load_b8(srs, (n * kb + b) | out, 0, 0);
        }
#pragma unroll
        for (int r = 0; r < RT; ++r)
#pragma unroll
          for (int j = 0; j < 4; ++j)
            xw[u][r][j] = __builtin_amdgcn_raw_buffer_load_b128(
                xrs, ((r * 16 + l16) * p.K * 2 + b * 64 + j * 16) | out, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int j = 0; j < 4; ++j)
#pragma unroll
          for (int c = 0; c < CT; ++c) {
            const u32x4_t a = decode8(cw[u][c][j], scale_of(sb[u][c]));
#pragma unroll
            for (int r = 0; r < RT; ++r) acc[r][c] = mfma16(a, xw[u][r][j], acc[r][c]);
          }
    }
  }
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < CT; ++c) part[wave][r * CT + c][lane] = acc[r][c];
  __syncthreads();
  OUT *Y = reinterpret_cast<OUT *>(p.Y);
  const bool vec = (p.N & 3) == 0;
  for (int i = threadIdx.x; i < RT * CT * 64; i += 64 * NW) {
    const int f = i >> 6, l = i & 63;
    f32x4_t v = part[0][f][l];
#pragma unroll
    for (int w = 1; w < NW; ++w) v += part[w][f][l];
    const int m = f / CT * 16 + (l & 15);
    const int n = n0 + f % CT * 16 + (l >> 4) * 4;
    if (m < t.rows) store4<OUT>(Y + (int64_t)(t.row0 + m) * p.N, n, p.N, v, vec);
  }
}

// ----------------------------------------------------------- many rows ----
// A workgroup of 4 waves owns 16 MF rows x 256 columns; wave w decodes columns
// 64 w .. 64 w + 63 into registers (no weight is decoded twice), the rows'
// 16 MF x 128 tile of X goes through LDS, double-buffered, loaded there directly.  A
// row's 16-byte chunk c sits at chunk c ^ (row % 16), so the 16 rows of a
// fragment read fall into different banks.
constexpr int kTileCols = 256;

template <int MF, typename OUT>
__global__ void __launch_bounds__(256, 2) mx_tile_kernel(Args p) {
  constexpr int BM = 16 * MF;
  __shared__ __attribute__((aligned(1024))) uint8_t xs[2][BM * 256];
  int slot, block;
  if (!grid_item(p.grid, &slot, &block)) return;
  const RowTile t = find_tile(p.offsets, p.E, p.R, slot, BM);
  if (t.rows <= 0) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int n0 = block * kTileCols;
  const int cols = min(kTileCols, p.N - n0);
  f32x4_t acc[4][MF];
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int r = 0; r < MF; ++r) acc[c][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  if (t.e >= 0) {
    const int kb = p.K >> 5;
    const int64_t first = (int64_t)t.e * p.N + n0;
    const __amdgpu_buffer_rsrc_t crs = buffer(p.codes + first * (p.K >> 1), (int64_t)cols * (p.K >> 1));
    const __amdgpu_buffer_rsrc_t srs = buffer(p.scales + first * kb, (int64_t)cols * kb);
    const __amdgpu_buffer_rsrc_t xrs =
        buffer(p.X + (int64_t)t.row0 * p.K, (int64_t)t.rows * p.K * 2);
    const int steps = (kb + 3) >> 2;
    // X loads: wave w, load i covers rows 4 (w + 4 i) .. + 3 of the tile
    const int xrow = wave * 4 + q;
    const int xchunk = l16 ^ (xrow & 15);  // rows 16 i + xrow share row % 16
    const auto load_x = [&](int buf, int s) {
      const int out = s * 16 + xchunk < kb * 4 ? 0 : kOutside;
#pragma unroll
      for (int i = 0; i < MF; ++i)
        load_lds16(xrs, &xs[buf][(i * 16 + wave * 4) * 256],
                   ((i * 16 + xrow) * p.K * 2 + s * 256 + xchunk * 16) | out);
    };
    u32x4_t cw[4];
    uint32_t sb[4];
    const auto load_w = [&](int s) {
      const int b = s * 4 + q;
      const int out = b < kb ? 0 : kOutside;
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        const int n = wave * 64 + c * 16 + l16;
        cw[c] = __builtin_amdgcn_raw_buffer_load_b128(crs, (n * (p.K >> 1) + b * 16) | out, 0, 0);
        sb[c] = __builtin_amdgcn_raw_buffer_load_b8(srs, (n * kb + b) | out, 0, 0);
      }
    };
    load_x(0, 0);
    load_w(0);
    for (int s = 0; s < steps; ++s) {
      lds_loads_done();
      __syncthreads();  // the step's rows are in LDS, the other buffer is free
      u32x4_t c0[4];
      float sc[4];
#pragma unroll
      for (int c = 0; c < 4; ++c) {
        c0[c] = cw[c];
        sc[c] = scale_of(sb[c]);
      }
      if (s + 1 < steps) {
        load_x((s + 1) & 1, s + 1);
        load_w(s + 1);
      }
      const uint8_t *x = xs[s & 1] + l16 * 256;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        u32x4_t b[MF];
#pragma unroll
        for (int r = 0; r < MF; ++r)
          b[r] = *reinterpret_cast<const u32x4_t *>(x + r * 4096 + (((q * 4 + j) ^ l16) * 16));
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const u32x4_t a = decode8(c0[c][j], sc[c]);
#pragma unroll
          for (int r = 0; r < MF; ++r) acc[c][r] = mfma16(a, b[r], acc[c][r]);
        }
      }
    }
  }
  OUT *Y = reinterpret_cast<OUT *>(p.Y);
  const bool vec = (p.N & 3) == 0;
#pragma unroll
  for (int r = 0; r < MF; ++r) {
    const int m = r * 16 + l16;
    if (m >= t.rows) continue;
    OUT *row = Y + (int64_t)(t.row0 + m) * p.N;
#pragma unroll
    for (int c = 0; c < 4; ++c)
      store4<OUT>(row, n0 + wave * 64 + c * 16 + q * 4, p.N, acc[c][r], vec);
  }
}

template <int RT, int CT, int NW>
static hipError_t launch_rows(Args &a, int out_dtype, hipStream_t s) {
  a.grid = make_grid(slots_for(a.R, a.E, a.offsets != nullptr, 16 * RT),
                     (a.N + 16 * CT - 1) / (16 * CT), 8);
  const int64_t n = grid_size(a.grid);
  if (n * 64 * NW >= (int64_t(1) << 32)) return hipErrorInvalidValue;
  if (out_dtype == NF4_F32)
    hipLaunchKernelGGL((mx_rows_kernel<RT, CT, NW, float>), dim3((unsigned)n), dim3(64 * NW), 0, s, a);
  else
    hipLaunchKernelGGL((mx_rows_kernel<RT, CT, NW, uint16_t>), dim3((unsigned)n), dim3(64 * NW), 0,
                       s, a);
  return hipGetLastError();
}

template <int MF>
static hipError_t launch_tile(Args &a, int out_dtype, hipStream_t s) {
  a.grid = make_grid(slots_for(a.R, a.E, a.offsets != nullptr, 16 * MF),
                     (a.N + kTileCols - 1) / kTileCols, 8);
  const int64_t n = grid_size(a.grid);
  if (n * 256 >= (int64_t(1) << 32)) return hipErrorInvalidValue;
  if (out_dtype == NF4_F32)
    hipLaunchKernelGGL((mx_tile_kernel<MF, float>), dim3((unsigned)n), dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((mx_tile_kernel<MF, uint16_t>), dim3((unsigned)n), dim3(256), 0, s, a);
  return hipGetLastError();
}

// Kernel by the rows an expert has on average (dense: all rows).
static hipError_t launch_product(Args &a, int out_dtype, hipStream_t s) {
  const int64_t rows = a.offsets ? (a.R + a.E - 1) / a.E : a.R;
  if (rows <= 16) return launch_rows<1, 1, 8>(a, out_dtype, s);
  if (rows <= 64) return launch_rows<2, 2, 4>(a, out_dtype, s);
  return launch_tile<8>(a, out_dtype, s);
}

}  // namespace mx
}  // namespace nf4

extern "C" {

int nf4_mx_gemm(const uint8_t *codes, const uint8_t *scales, int64_t N, int64_t K,
                const uint16_t *X, int64_t M, void *Y, int out_dtype, void *stream) {
  if (!codes || !scales || !X || !Y || !nf4::known_dtype(out_dtype)) return NF4_EINVAL;
  if (int r = nf4::check_mx_shape(N, K)) return r;
  if (M < 1 || M >= (int64_t(1) << 26)) return NF4_ERANGE;
  if (!nf4::aligned_to(codes, 16) || !nf4::aligned_to(X, 16) || !nf4::aligned_to(Y, 16))
    return NF4_EALIGN;
  if (int r = nf4::device_status()) return r;
  nf4::mx::Args a{codes, scales, X, nullptr, Y, M, 1, (int)N, (int)K, {}};
  return nf4::launch_status(nf4::mx::launch_product(a, out_dtype, (hipStream_t)stream));
}

int nf4_mx_gemm_grouped(const uint8_t *codes, const uint8_t *scales, int64_t E, int64_t N,
                        int64_t K, const uint16_t *X, const int32_t *offsets, int64_t R, void *Y,
                        int out_dtype, void *stream) {
  if (E < 1 || R < 0 || !codes || !scales || !offsets || (R > 0 && (!X || !Y)) ||
      !nf4::known_dtype(out_dtype))
    return NF4_EINVAL;
  if (int r = nf4::check_mx_shape(N, K)) return r;
  if (E > NF4_MOE_MAX_E || R >= (int64_t(1) << 26)) return NF4_ERANGE;
  if (!nf4::aligned_to(codes, 16) || !nf4::aligned_to(X, 16) || !nf4::aligned_to(Y, 16) ||
      !nf4::aligned_to(offsets, 4))
    return NF4_EALIGN;
  if (int r = nf4::device_status()) return r;
  if (R == 0) return NF4_OK;
  nf4::mx::Args a{codes, scales, X, offsets, Y, R, (int)E, (int)N, (int)K, {}};
  return nf4::launch_status(nf4::mx::launch_product(a, out_dtype, (hipStream_t)stream));
}

}  // extern "C"
