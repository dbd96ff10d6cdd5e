// mx_packed.hip -- product of two packed MXFP4 matrices on the block-scaled matrix
// instructions (gfx950):
//   Y[m][n] = sum_k u(m, k) * v(n, k), both of them element * 2^(scale - 127).
//
// v_mfma_scale_f32_16x16x128_f8f6f4 takes the format as it is stored: lane l
// holds row l % 16 and the 16 bytes and the scale byte of block l / 16 of a
// step of 128 k; sums are fp32.  A = weights, B = rows, so a lane ends with four
// consecutive columns of one row.
#include "mx_device.h"
#include "nf4_check.h"

namespace nf4 {
namespace mx {

typedef int i32x8_t __attribute__((ext_vector_type(8)));

struct PackedArgs {
  const uint8_t *codes;
  const uint8_t *scales;
  const uint8_t *xcodes;
  const uint8_t *xscales;
  void *Y;
  int64_t M;
  int N, K;
  Grid grid;
};

__device__ __forceinline__ f32x4_t mfma_scaled(u32x4_t a, uint32_t sa, u32x4_t b, uint32_t sb,
                                               f32x4_t c) {
  const i32x8_t va = {(int)a[0], (int)a[1], (int)a[2], (int)a[3], 0, 0, 0, 0};
  const i32x8_t vb = {(int)b[0], (int)b[1], (int)b[2], (int)b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, c, 4, 4, 0, (int)sa, 0, (int)sb);
}

// ------------------------------------------------------------ few rows ----
// 16 CT columns x 16 RT rows a workgroup, K dealt out to its NW waves by steps;
// tiles meet in LDS and are added in wave order.
template <int RT, int CT, int NW, typename OUT>
__global__ void __launch_bounds__(64 * NW) mx_packed_rows_kernel(PackedArgs p) {
  __shared__ f32x4_t part[NW][RT * CT][64];
  int slot, block;
  if (!grid_item(p.grid, &slot, &block)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int n0 = block * 16 * CT, cols = min(16 * CT, p.N - n0);
  const int64_t m0 = (int64_t)slot * 16 * RT;
  const int rows = (int)min((int64_t)16 * RT, p.M - m0);
  const int kb = p.K >> 5, kc = p.K >> 1;
  const __amdgpu_buffer_rsrc_t crs = buffer(p.codes + (int64_t)n0 * kc, (int64_t)cols * kc);
  const __amdgpu_buffer_rsrc_t srs = buffer(p.scales + (int64_t)n0 * kb, (int64_t)cols * kb);
  const __amdgpu_buffer_rsrc_t xrs = buffer(p.xcodes + m0 * kc, (int64_t)rows * kc);
  const __amdgpu_buffer_rsrc_t ars = buffer(p.xscales + m0 * kb, (int64_t)rows * kb);
  f32x4_t acc[RT][CT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int c = 0; c < CT; ++c) acc[r][c] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int steps = (kb + 3) >> 2;
  constexpr int U = 2;
  for (int s0 = wave; s0 < steps; s0 += NW * U) {
    u32x4_t cw[U][CT], xw[U][RT];
    uint32_t cs[U][CT], xb[U][RT];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = (s0 + u * NW) * 4 + q;
      const int out = b < kb ? 0 : kOutside;
#pragma unroll
      for (int c = 0; c < CT; ++c) {
        const int n = c * 16 + l16;
        cw[u][c] = __builtin_amdgcn_raw_buffer_load_b128(crs, (n * kc + b * 16) | out, 0, kLoadStream);
        cs[u][c] = __builtin_amdgcn_raw_buffer_load_b8(srs, (n * kb + b) | out, 0, 0);
      }
#pragma unroll
      for (int r = 0; r < RT; ++r) {
        const int m = r * 16 + l16;
        xw[u][r] = __builtin_amdgcn_raw_buffer_load_b128(xrs, (m * kc + b * 16) | out, 0, 0);
        xb[u][r] = __builtin_amdgcn_raw_buffer_load_b8(ars, (m * kb + b) | out, 0, 0);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int c = 0; c < CT; ++c)
#pragma unroll
        for (int r = 0; r < RT; ++r)
          acc[r][c] = mfma_scaled(cw[u][c], cs[u][c], xw[u][r], xb[u][r], acc[r][c]);
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
    if (m < rows) store4<OUT>(Y + (m0 + m) * p.N, n, p.N, v, vec);
  }
}

// ----------------------------------------------------------- many rows ----
// A workgroup owns a 256 x 256 tile; WN x WM waves, each 16 NF columns x 16 MF
// rows.  A stage is 256 k: 128 bytes a row of either operand, loaded straight into
// LDS (16-byte chunk c of a row at chunk c ^ (row / 2 % 8), so that the 16
// rows of a fragment fall into different banks), and 8 scale bytes a row;
// double-buffered, one barrier a stage.
template <int WN, int WM, int NF, int MF, bool SVEC, typename OUT>
__global__ void __launch_bounds__(64 * WN * WM, WN *WM / 4) mx_packed_tile_kernel(PackedArgs p) {
  constexpr int BN = 16 * NF * WN, BM = 16 * MF * WM, NT = 64 * WN * WM, ROWS = BN + BM;
  __shared__ __attribute__((aligned(1024))) uint8_t tile[2][ROWS * 128];
  __shared__ u32x2_t sc[2][ROWS];
  int slot, block;
  if (!grid_item(p.grid, &slot, &block)) return;
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int l16 = lane & 15, q = lane >> 4;
  const int wn = wave % WN, wm = wave / WN;
  const int n0 = block * BN, cols = min(BN, p.N - n0);
  const int64_t m0 = (int64_t)slot * BM;
  const int rows = (int)min((int64_t)BM, p.M - m0);
  const int kb = p.K >> 5, kc = p.K >> 1;
  const u32x4_t crs = buffer_words(p.codes + (int64_t)n0 * kc, cols * kc);
  const __amdgpu_buffer_rsrc_t srs = buffer(p.scales + (int64_t)n0 * kb, (int64_t)cols * kb);
  const u32x4_t xrs = buffer_words(p.xcodes + m0 * kc, rows * kc);
  const __amdgpu_buffer_rsrc_t ars = buffer(p.xscales + m0 * kb, (int64_t)rows * kb);
  f32x4_t acc[NF][MF];
#pragma unroll
  for (int c = 0; c < NF; ++c)
#pragma unroll
    for (int r = 0; r < MF; ++r) acc[c][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int stages = (kb + 7) >> 3;
  const uint32_t tiles = lds_address(tile);
  // a wave's load covers 8 rows, the first one 8 (wave + a multiple of 2); lane: row
  // lane / 8, chunk (lane % 8) ^ (row / 2 % 8)
  static_assert(WN * WM % 2 == 0, "row / 2 % 8 of a load depends on the wave alone");
  const int lrow = lane >> 3, lchunk = (lane & 7) ^ ((wave & 1) * 4 + (lrow >> 1));
  const auto load_codes = [&](int buf, int s) {
    const int out = s * 8 + lchunk < kb ? 0 : kOutside;
#pragma unroll
    for (int i = 0; i < BN / 8 / (WN * WM); ++i) {
      const int r = (i * WN * WM + wave) * 8;
      load_lds16(crs, tiles + buf * ROWS * 128 + r * 128, ((r + lrow) * kc + s * 128 + lchunk * 16) | out);
    }
#pragma unroll
    for (int i = 0; i < BM / 8 / (WN * WM); ++i) {
      const int r = (i * WN * WM + wave) * 8;
      load_lds16(xrs, tiles + buf * ROWS * 128 + (BN + r) * 128, ((r + lrow) * kc + s * 128 + lchunk * 16) | out);
    }
  };
  // scales: thread -> rows tid, tid + NT, ... of the BN + BM
  constexpr int SR = (ROWS + NT - 1) / NT;
  u32x2_t sreg[SR];
  const auto load_scales = [&](int s) {
#pragma unroll
    for (int i = 0; i < SR; ++i) {
      const int r = i * NT + tid;
      const bool w = r < BN;
      const int off = (w ? r : r - BN) * kb + s * 8;
      if constexpr (SVEC) {
        // rows are whole words: two words, each inside the row or outside
        const int o0 = r < ROWS && s * 8 < kb ? off : kOutside;
        const int o1 = r < ROWS && s * 8 + 4 < kb ? off + 4 : kOutside;
        const uint32_t a0 = __builtin_amdgcn_raw_buffer_load_b32(srs, w ? o0 : kOutside, 0, 0);
        const uint32_t a1 = __builtin_amdgcn_raw_buffer_load_b32(srs, w ? o1 : kOutside, 0, 0);
        const uint32_t b0 = __builtin_amdgcn_raw_buffer_load_b32(ars, w ? kOutside : o0, 0, 0);
        const uint32_t b1 = __builtin_amdgcn_raw_buffer_load_b32(ars, w ? kOutside : o1, 0, 0);
        sreg[i] = u32x2_t{a0 | b0, a1 | b1};
      } else {
        uint32_t v[2] = {0u, 0u};
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int o = r < ROWS && s * 8 + k < kb ? off + k : kOutside;
          const uint32_t a = __builtin_amdgcn_raw_buffer_load_b8(srs, w ? o : kOutside, 0, 0);
          const uint32_t b = __builtin_amdgcn_raw_buffer_load_b8(ars, w ? kOutside : o, 0, 0);
          v[k >> 2] |= (a | b) << (8 * (k & 3));
        }
        sreg[i] = u32x2_t{v[0], v[1]};
      }
    }
  };
  load_codes(0, 0);
  load_scales(0);
  for (int s = 0; s < stages; ++s) {
    const int buf = s & 1;
#pragma unroll
    for (int i = 0; i < SR; ++i)
      if (i * NT + tid < ROWS) sc[buf][i * NT + tid] = sreg[i];
    lds_loads_but<0>();
    __syncthreads();  // the stage is in LDS, the other buffer is free
    if (s + 1 < stages) {
      load_codes(buf ^ 1, s + 1);
      load_scales(s + 1);
    }
    const uint8_t *wt = &tile[buf][(wn * 16 * NF + l16) * 128];
    const uint8_t *xt = &tile[buf][(BN + wm * 16 * MF + l16) * 128];
    u32x2_t sw[NF], sx[MF];
#pragma unroll
    for (int c = 0; c < NF; ++c) sw[c] = sc[buf][wn * 16 * NF + c * 16 + l16];
#pragma unroll
    for (int r = 0; r < MF; ++r) sx[r] = sc[buf][BN + wm * 16 * MF + r * 16 + l16];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int ch = ((h * 4 + q) ^ (l16 >> 1)) * 16;
      u32x4_t b[MF];
      uint32_t bs[MF];
#pragma unroll
      for (int r = 0; r < MF; ++r) {
        b[r] = *reinterpret_cast<const u32x4_t *>(xt + r * 2048 + ch);
        bs[r] = sx[r][h] >> (8 * q);
      }
#pragma unroll
      for (int c = 0; c < NF; ++c) {
        const u32x4_t a = *reinterpret_cast<const u32x4_t *>(wt + c * 2048 + ch);
        const uint32_t as = sw[c][h] >> (8 * q);
#pragma unroll
        for (int r = 0; r < MF; ++r) acc[c][r] = mfma_scaled(a, as, b[r], bs[r], acc[c][r]);
      }
    }
  }
  OUT *Y = reinterpret_cast<OUT *>(p.Y);
  const bool vec = (p.N & 3) == 0;
#pragma unroll
  for (int r = 0; r < MF; ++r) {
    const int m = (wm * MF + r) * 16 + l16;
    if (m >= rows) continue;
    OUT *row = Y + (m0 + m) * p.N;
#pragma unroll
    for (int c = 0; c < NF; ++c)
      store4<OUT>(row, n0 + (wn * NF + c) * 16 + q * 4, p.N, acc[c][r], vec);
  }
}

template <int RT, int CT, int NW>
static hipError_t launch_packed_rows(PackedArgs &a, int out_dtype, hipStream_t s) {
  a.grid = make_grid((a.M + 16 * RT - 1) / (16 * RT), (a.N + 16 * CT - 1) / (16 * CT), 8);
  const int64_t n = grid_size(a.grid);
  if (n * 64 * NW >= (int64_t(1) << 32)) return hipErrorInvalidValue;
  if (out_dtype == NF4_F32)
    hipLaunchKernelGGL((mx_packed_rows_kernel<RT, CT, NW, float>), dim3((unsigned)n), dim3(64 * NW),
                       0, s, a);
  else
    hipLaunchKernelGGL((mx_packed_rows_kernel<RT, CT, NW, uint16_t>), dim3((unsigned)n),
                       dim3(64 * NW), 0, s, a);
  return hipGetLastError();
}

template <int WN, int WM, int NF, int MF, bool SVEC>
static hipError_t launch_packed_tile(PackedArgs &a, int out_dtype, hipStream_t s) {
  constexpr int BN = 16 * NF * WN, BM = 16 * MF * WM, NT = 64 * WN * WM;
  a.grid = make_grid((a.M + BM - 1) / BM, (a.N + BN - 1) / BN, 8);
  const int64_t n = grid_size(a.grid);
  if (n * NT >= (int64_t(1) << 32)) return hipErrorInvalidValue;
  if (out_dtype == NF4_F32)
    hipLaunchKernelGGL((mx_packed_tile_kernel<WN, WM, NF, MF, SVEC, float>), dim3((unsigned)n),
                       dim3(NT), 0, s, a);
  else
    hipLaunchKernelGGL((mx_packed_tile_kernel<WN, WM, NF, MF, SVEC, uint16_t>), dim3((unsigned)n),
                       dim3(NT), 0, s, a);
  return hipGetLastError();
}

static hipError_t launch_packed(PackedArgs &a, int out_dtype, hipStream_t s) {
  if (a.M <= 16) return launch_packed_rows<1, 1, 8>(a, out_dtype, s);
  if (a.M <= 128) return launch_packed_rows<2, 2, 4>(a, out_dtype, s);
  const bool svec = a.K % 128 == 0 && aligned_to(a.scales, 4) && aligned_to(a.xscales, 4);
  if (svec) return launch_packed_tile<2, 4, 8, 4, true>(a, out_dtype, s);
  return launch_packed_tile<2, 4, 8, 4, false>(a, out_dtype, s);
}

}  // namespace mx
}  // namespace nf4

extern "C" {

int nf4_mx_gemm_packed(const uint8_t *codes, const uint8_t *scales, int64_t N, int64_t K,
                       const uint8_t *xcodes, const uint8_t *xscales, int64_t M, void *Y,
                       int out_dtype, void *stream) {
  if (!codes || !scales || !xcodes || !xscales || !Y || !nf4::known_dtype(out_dtype))
    return NF4_EINVAL;
  if (int r = nf4::check_mx_shape(N, K)) return r;
  if (M < 1 || M >= (int64_t(1) << 26)) return NF4_ERANGE;
  if (!nf4::aligned_to(codes, 16) || !nf4::aligned_to(xcodes, 16) || !nf4::aligned_to(Y, 16))
    return NF4_EALIGN;
  if (int r = nf4::device_status()) return r;
  nf4::mx::PackedArgs a{codes, scales, xcodes, xscales, Y, M, (int)N, (int)K, {}};
  return nf4::launch_status(nf4::mx::launch_packed(a, out_dtype, (hipStream_t)stream));
}

}  // extern "C"
