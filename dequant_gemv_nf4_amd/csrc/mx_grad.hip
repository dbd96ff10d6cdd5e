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
#include "mx_act.h"
#include "mx_grad.h"
#include "mx_plan.h"

namespace nf4 {
namespace mx {

struct GradArgs {
  const uint8_t *codes;
  const uint8_t *scales;
  const uint16_t *dY;
  const int32_t *offsets;  // null: dense
  void *dX;
  int64_t R;
  int E, N, K;
  Grid grid;
  // partial sums (PART): rows of dY are ld values apart, zero from column N up to the next
  // multiple of 8; split i of the n's goes to dX + i R K in fp32, added to what is there times
  // rescale[row] if that is given.
  int64_t ld;
  int splits;
  const float *rescale;
};

// A workgroup owns 16 MF rows x 128 WV columns; its waves form KG groups of WV that
// share out the n.  A stage is 64 n: the rows' tile of dY and the 64 rows of codes (64
// bytes a wave) go straight into LDS, three stages in rotation, one barrier a
// stage; a lane holds the four scale bytes of one n and passes them on through LDS.
// Decoding (two vector instructions a matrix instruction) runs 32 n ahead: a pair of
// columns makes room for the next 32 n's as soon as it is multiplied (before: all of
// it between the matrix instructions of two blocks; 1000 rows of 8 experts 203 -> 191
// us, 2000 387 -> 364, 16382 1758 -> 1745), and the next stage's loads go out after its
// first products (16382 rows 1732 -> 1660 us, each pair on one card).  So a wave waits for stage s + 1 in the
// middle of stage s, when all of s is in its registers, and stage s + 3 goes where s was.
// Bound by the issue of vector instructions beside the matrix instructions, and by the
// card's clock, which such loads hold near 2 GHz: 16382 rows of 8 experts of 14336 x 4096
// 1600-1710 us from one card to the next (1.13-1.20 PFLOP/s).

// dY: chunk of 16 bytes of a 128-byte row, permuted as the rows of the product.
__device__ __forceinline__ int dy_perm(int row) { return (row >> 1) & 7; }
// Codes: row n of a stage lies at row code_row, its 64-byte pieces permuted by
// code_perm, so that the rows n, n + 8, n + 16, n + 24 that the lane quarters of a wave
// read together cover all banks.
template <int WV>
__device__ __forceinline__ int code_row(int n) {
  return WV == 2 ? n ^ ((n >> 4) & 1) : n;
}
template <int WV>
__device__ __forceinline__ int code_perm(int n) {
  return (n >> 3) & (WV - 1);
}

// pair j of the 8 codes of w, as decode8
__device__ __forceinline__ uint32_t decode2(uint32_t w, float scale, int j) {
  switch (j) {
    case 0: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
    case 1: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
    case 2: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
    default: return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  }
}

template <int MF, int WV, int KG, bool SVEC, typename OUT, bool PART>
__global__ void __launch_bounds__(64 * WV *KG, 2) mx_grad_kernel(GradArgs p) {
  constexpr int BM = 16 * MF, NX = 3;
  constexpr int XB = BM * 128, WB = 64 * 64 * WV;
  constexpr int XL = 2 * MF / WV, WL = 4;  // loads a wave
  static_assert(XL * WV == 2 * MF, "whole loads");
  __shared__ __attribute__((aligned(1024))) uint8_t shared[KG][NX * (XB + WB)];
  // the four scale bytes (one per block of 32 of the wave's columns) of each n
  __shared__ __attribute__((aligned(256))) uint32_t sc[KG][WV][NX][64];
  int slot, block;
  if (!grid_item(p.grid, &slot, &block)) return;
  int split = 0;
  if constexpr (PART) {
    split = block % p.splits;
    block /= p.splits;
  }
  const int64_t ld = PART ? p.ld : p.N;
  const RowTile t = find_tile(PART ? nullptr : p.offsets, p.E, p.R, slot, BM);
  if (t.rows <= 0) return;
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wave = wave_all % WV, kg = wave_all / WV;
  const int l16 = lane & 15, q = lane >> 4;
  const int k0 = block * 128 * WV;
  f32x4_t acc[8][MF];
#pragma unroll
  for (int j = 0; j < 8; ++j)
#pragma unroll
    for (int r = 0; r < MF; ++r) acc[j][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  if (t.e >= 0) {
    const int kb = p.K >> 5, kc = p.K >> 1;
    const int64_t first = (int64_t)t.e * p.N;
    const int groups = PART ? KG * p.splits : KG;
    const int stages = (p.N + 63) >> 6, per = (stages + groups - 1) / groups;
    uint8_t *const xlds = shared[kg];
    uint8_t *const wlds = shared[kg] + NX * XB;
    uint32_t *const slds = sc[kg][wave][0];
    const uint32_t xaddr = lds_address(xlds), waddr = lds_address(wlds), saddr = lds_address(slds);
    int xo[XL], wo[WL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int idx = (i * WV + wave) * 64 + lane, row = idx >> 3;
      xo[i] = row * (int)ld * 2 + ((idx & 7) ^ dy_perm(row)) * 16;
    }
#pragma unroll
    for (int i = 0; i < WL; ++i) {
      const int idx = (i * WV + wave) * 64 + lane;
      const int n = code_row<WV>(idx / (4 * WV)), ch = idx % (4 * WV);
      wo[i] = n * kc + (k0 >> 1) + (ch ^ code_perm<WV>(n) * 4) * 16;
    }
    const int xbytes = t.rows * (int)ld * 2;
    const uint8_t *xbase = reinterpret_cast<const uint8_t *>(p.dY + (int64_t)t.row0 * ld);
    const uint8_t *wbase = p.codes + first * kc;
    // Past N the codes are outside their buffer and dY's chunks are masked; columns
    // past K read another row's codes, their outputs are not stored.
    const auto load_stage = [&](int buf, int s) {
      const int adv = s * 128;
      const u32x4_t rs = buffer_words(xbase + adv, max(xbytes - adv, 0));
      const int left = ((PART ? p.N + 7 : p.N) >> 3) - s * 8;
      int o[XL];
#pragma unroll
      for (int i = 0; i < XL; ++i) {
        const int idx = (i * WV + wave) * 64 + lane, row = idx >> 3;
        o[i] = xo[i];
        if (left < 8) o[i] = ((idx & 7) ^ dy_perm(row)) < left ? o[i] : kOutside;
      }
      load_lds16xn<XL, WV * 1024>(rs, xaddr + buf * XB + wave * 1024, o);
      const int rows = max(p.N - s * 64, 0);
      const u32x4_t ws = buffer_words(wbase + (int64_t)s * 64 * kc, rows * kc);
      load_lds16xn<WL, WV * 1024>(ws, waddr + buf * WB + wave * 1024, wo);
    };
    // lane: the four block scales of this wave's columns at n = 64 s + lane; rows that
    // are not whole words go through registers, a stage ahead, from one buffer over the
    // matrix.  Its last word may hold what follows the matrix: a row past N takes zero
    // instead, since a byte of 255 there would be NaN, and so 0 x NaN in every sum.
    const uint8_t *sbase = p.scales + first * kb;
    const int so = lane * kb + (k0 >> 5) + wave * 4;
    const LooseWords loose(sbase, (int64_t)p.N * kb);
    uint32_t snext[2];
    const auto load_scales = [&](int buf, int s) {
      if constexpr (SVEC) {
        const int bytes = max(p.N - s * 64, 0) * kb;
        load_lds4(buffer_words(sbase + (int64_t)s * 64 * kb, bytes), saddr + buf * 256, so);
      } else {
        snext[0] = loose.fetch(so + s * 64 * kb, 0);
        snext[1] = loose.fetch(so + s * 64 * kb, 1);
      }
    };
    // The words of 32 n: row n = 32 h + 8 q + i (code_row and code_perm written out)
    struct Raw {
      uint32_t w[8];
      float s[8];
    };
    const auto read = [&](Raw &w, u32x4_t *b, int buf, int h) __attribute__((always_inline)) {
      const uint8_t *cr = wlds + buf * WB + (h * 32 + q * 8) * 64 * WV + (wave ^ (q & (WV - 1))) * 64 + l16 * 4;
      const int swap = WV == 2 ? q >> 1 : 0;
      const u32x4_t *sr = reinterpret_cast<const u32x4_t *>(slds + buf * 64 + h * 32 + q * 8);
      const u32x4_t s03 = sr[0], s47 = sr[1];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        w.w[i] = *reinterpret_cast<const uint32_t *>(cr + (i ^ swap) * 64 * WV);
        w.s[i] = scale_of(__builtin_amdgcn_ubfe(i < 4 ? s03[i & 3] : s47[i & 3], 8 * (l16 >> 2), 8));
      }
      const uint8_t *xt = xlds + buf * XB + l16 * 128 + ((h * 4 + q) ^ dy_perm(l16)) * 16;
#pragma unroll
      for (int r = 0; r < MF; ++r) b[r] = *reinterpret_cast<const u32x4_t *>(xt + r * 2048);
    };
    uint32_t d[4][8];  // pairs along k: columns 2 j, 2 j + 1 of the lane's 8, of 8 n
    const auto decode = [&](const Raw &w, int j) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < 8; ++i) d[j][i] = decode2(w.w[i], w.s[i], j);
    };
    // multiplies 32 n; a pair of columns that is done makes room for the next 32 n's
    const auto multiply = [&](const u32x4_t *b, const Raw &next, auto more) __attribute__((always_inline)) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u32x4_t a;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          a[i] = __builtin_amdgcn_perm(d[j >> 1][2 * i + 1], d[j >> 1][2 * i],
                                       (j & 1) ? 0x07060302u : 0x05040100u);
#pragma unroll
        for (int r = 0; r < MF; ++r) acc[j][r] = mfma16(a, b[r], acc[j][r]);
        if (j & 1) decode(next, j >> 1);
        more(j);
      }
    };
    const int s0 = (split * KG + kg) * per;
    constexpr int one = XL + WL + (SVEC ? 1 : 0);
    const auto put_scales = [&](int buf, int s) __attribute__((always_inline)) {
      if constexpr (!SVEC) {
        const uint32_t w = loose.word(so + s * 64 * kb, snext[0], snext[1]);
        slds[buf * 64 + lane] = s * 64 + lane < p.N ? w : 0u;
      }
    };
    load_scales(0, s0);
    load_stage(0, s0);
    put_scales(0, s0);
    load_scales(1, s0 + 1);
    load_stage(1, s0 + 1);
    if constexpr (SVEC) load_scales(2, s0 + 2);
    load_stage(2, s0 + 2);
    lds_loads_but<2 * one>();
    __syncthreads();
    Raw w;
    u32x4_t b0[MF], b1[MF];
    read(w, b0, 0, 0);
#pragma unroll
    for (int j = 0; j < 4; ++j) decode(w, j);
    int buf = 0;
    for (int s = s0; s < s0 + per; ++s) {
      const int next = buf == NX - 1 ? 0 : buf + 1;
      read(w, b1, buf, 1);
      multiply(b0, w, [](int) {});
      put_scales(next, s + 1);
      lds_loads_but<one>();
      __syncthreads();  // stage s + 1 is in LDS; all of stage s has been read
      read(w, b0, next, 0);
      multiply(b1, w, [&](int j) __attribute__((always_inline)) {
        if (j != 1) return;  // the loads go out once the matrix cores are fed
        load_scales(buf, SVEC ? s + 3 : s + 2);
        load_stage(buf, s + 3);
      });
      buf = next;
    }
    lds_loads_but<0>();
  }
  if constexpr (KG > 1) {
    static_assert(sizeof(shared) >= (KG - 1) * WV * 64 * 8 * MF * 16, "partial tiles fit the stages");
    f32x4_t *part = reinterpret_cast<f32x4_t *>(&shared[0][0]);  // [kg - 1][wave][f][lane]
    __syncthreads();
    if (kg > 0)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int r = 0; r < MF; ++r)
          part[(((kg - 1) * WV + wave) * 8 * MF + j * MF + r) * 64 + lane] = acc[j][r];
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int g = 0; g < KG - 1; ++g)
#pragma unroll
      for (int j = 0; j < 8; ++j)
#pragma unroll
        for (int r = 0; r < MF; ++r)
          acc[j][r] += part[((g * WV + wave) * 8 * MF + j * MF + r) * 64 + lane];
  }
  OUT *X = reinterpret_cast<OUT *>(p.dX);
  if constexpr (PART) X += (int64_t)split * p.R * p.K;
#pragma unroll
  for (int r = 0; r < MF; ++r) {
    const int m = r * 16 + l16;
    if (m >= t.rows) continue;
    OUT *row = X + (int64_t)(t.row0 + m) * p.K;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int k = k0 + wave * 128 + 8 * (4 * q + i);
      if (k >= p.K) continue;
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = acc[j][r][i];
      if constexpr (PART) {
        f32x4_t lo = {v[0], v[1], v[2], v[3]}, hi = {v[4], v[5], v[6], v[7]};
        f32x4_t *at = reinterpret_cast<f32x4_t *>(row + k);
        if (p.rescale) {
          const float f = p.rescale[t.row0 + m];
          lo += at[0] * f;
          hi += at[1] * f;
        }
        at[0] = lo;
        at[1] = hi;
      } else if constexpr (sizeof(OUT) == 4) {
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

template <int MF, int WV, int KG, bool SVEC, bool PARTS>
static int launch_grad_as(GradArgs &a, int out_dtype, hipStream_t s) {
  const int64_t blocks = (a.K + 128 * WV - 1) / (128 * WV);
  a.grid = make_grid(slots_for(a.R, a.E, a.offsets != nullptr, 16 * MF), blocks * a.splits, 8);
  const int64_t n = grid_size(a.grid);
  if (n * 64 * WV * KG >= (int64_t(1) << 32)) return NF4_ERANGE;
  const dim3 grid((unsigned)n), threads(64 * WV * KG);
  if constexpr (PARTS)
    if (a.ld) {
      hipLaunchKernelGGL((mx_grad_kernel<MF, WV, KG, SVEC, float, true>), grid, threads, 0, s, a);
      return launch_status(hipGetLastError());
    }
  if (out_dtype == NF4_F32)
    hipLaunchKernelGGL((mx_grad_kernel<MF, WV, KG, SVEC, float, false>), grid, threads, 0, s, a);
  else
    hipLaunchKernelGGL((mx_grad_kernel<MF, WV, KG, SVEC, uint16_t, false>), grid, threads, 0, s, a);
  return launch_status(hipGetLastError());
}

// PARTS: also the form whose sums are shared out (a.ld is given)
template <int MF, int WV, int KG, bool PARTS = false>
static int launch_grad(GradArgs &a, int out_dtype, hipStream_t s) {
  if (a.K % 128 == 0 && aligned_to(a.scales, 4))
    return launch_grad_as<MF, WV, KG, true, PARTS>(a, out_dtype, s);
  return launch_grad_as<MF, WV, KG, false, PARTS>(a, out_dtype, s);
}

// The largest tile that is not mostly empty and gives every CU work, with N shared out
// inside the workgroup (K-groups) where tiles are few.  Measured, us, rows of experts of
// matrices N x K, weights from memory:
//   taken                   case                               others
//   64 x 512                16382 of 8 of 14336 x 4096  1700   32 x 512, two K-groups: 2408
//                           2000 of 8 of 14336 x 4096    324   two K-groups: 354
//   64 x 512, two K-groups  1000 of 8 of 14336 x 4096    173   one: 199, 32 x 512, two: 279
//   32 x 512, two           1003 of 32 of 2048 x 2048   27.9   64 x 512, two: 33.6; 32 x 256, two: 32.9
//   32 x 256, two           300 of 8 of 14336 x 4096     101   32 x 512, two: 141; 16 x 256, two: 146
//                           500 of 8 of 14336 x 4096     165   32 x 512, two: 140
//   16 x 256, two           60 of 64 of 4096 x 4096     74.8   four: 79.9
//   16 x 256, four          8 of 8 of 14336 x 4096      79.7   two: 83.3
//                           64 of 1 of 4096 x 4096      25.1   two: 28.0
static int launch_rows_grad(GradArgs &a, int out_dtype, hipStream_t s) {
  const auto tiles = [&](int bm, int bk) {
    return slots_for(a.R, a.E, a.offsets != nullptr, bm) * ((a.K + bk - 1) / bk);
  };
  const int64_t mean = (a.R + a.E - 1) / a.E, rows = mean + mean / 2;
  if (rows > 48) {
    if (tiles(64, 512) >= 256) return launch_grad<4, 4, 1>(a, out_dtype, s);
    if (tiles(64, 512) >= 160) return launch_grad<4, 4, 2>(a, out_dtype, s);
  }
  if (rows > 16) {
    if (tiles(32, 512) >= 224) return launch_grad<2, 4, 2>(a, out_dtype, s);
    if (tiles(32, 256) >= 192) return launch_grad<2, 2, 2>(a, out_dtype, s);
  }
  if (tiles(16, 256) >= 384) return launch_grad<1, 2, 2>(a, out_dtype, s);
  return launch_grad<1, 2, 4>(a, out_dtype, s);
}

// ------------------------------------------------- sums shared out over workgroups ----
// The tile and shares of plan_dense().
static int launch_plan(const DensePlan &d, GradArgs &a, int out_dtype, hipStream_t s) {
  if (d.mf == 1) return launch_grad<1, 2, 2, true>(a, out_dtype, s);
  if (d.mf == 2) return launch_grad<2, 2, 2, true>(a, out_dtype, s);
  return d.kg == 1 ? launch_grad<4, 4, 1, true>(a, out_dtype, s) : launch_grad<4, 4, 2, true>(a, out_dtype, s);
}

int grad_splits(int64_t M, int64_t N, int64_t K) { return plan_dense(M, N, K).splits; }

int launch_grad_parts(const GradParts &g, hipStream_t s) {
  const DensePlan d = plan_dense(g.plan_M, g.plan_N, g.K);
  GradArgs a{g.codes, g.scales, g.dY, nullptr, g.parts, g.M, 1, (int)g.N, (int)g.K, {}, g.ld, d.splits, g.rescale};
  return launch_plan(d, a, NF4_F32, s);
}

// out = the parts' sum, in order.  Bound by memory: two parts of 2048 x 4096 12.5 us (6.7 TB/s,
// from the caches); four of 77 x 5120 4.
template <typename OUT>
__global__ void __launch_bounds__(256)
    mx_parts_kernel(const float *__restrict__ parts, int splits, int64_t size, OUT *__restrict__ out, bool vec) {
  const int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
  if (i >= size) return;
  f32x4_t v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll 8
  for (int k = 0; k < splits; ++k) v += *reinterpret_cast<const f32x4_t *>(parts + k * size + i);
  store4<OUT>(out + i, 0, 4, v, vec);
}

// ------------------------------------------------------- in front of the sums ----
// dZ = dY f'(Z) (gated: dY z_u f'(z_g) and dY f(z_g)) in bf16, and its column sums from the
// unrounded values.  bf16 since that is what the matrix cores take: dZ in two halves of 8 bits
// each would double their work, twice 380 us of 440 at 2048 x 28672 x 4096.  So dX (in bf16) is
// 2.3e-3 of its norm off where one rounding at the end leaves 1.7e-3.  A thread has four columns (of both halves, gated) and every 64th row of
// its workgroup's; the sums are added in one order.
// Bound by memory: 2048 rows of 28672, gated, 62-64 us (4.6-4.7 TB/s); 77 rows of 13824 with the column
// sums 5-6, mostly start and the sums' way through LDS.
template <bool GATED>
__global__ void __launch_bounds__(1024)
    mx_act_grad_kernel(const uint16_t *__restrict__ dY, const uint16_t *__restrict__ Z, int64_t M, int N,
                       int act, int64_t rows_wg, uint16_t *__restrict__ dZ, float *__restrict__ dbias) {
  constexpr int W = GATED ? 8 : 4, LANES = 16;
  __shared__ float part[1024 * W];
  const int cols = GATED ? N >> 1 : N;
  const int c = threadIdx.x % LANES, y = threadIdx.x / LANES, ny = 1024 / LANES;
  const int n = (blockIdx.x * LANES + c) * 4;
  const int64_t m0 = (int64_t)blockIdx.y * rows_wg, m1 = m0 + rows_wg < M ? m0 + rows_wg : M;
  float sum[W];
#pragma unroll
  for (int i = 0; i < W; ++i) sum[i] = 0.f;
  if (n < cols) {
    const auto get = [](const uint16_t *p) __attribute__((always_inline)) {
      const u32x2_t w = *reinterpret_cast<const u32x2_t *>(p);
      return f32x4_t{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
    };
#pragma unroll 2
    for (int64_t m = m0 + y; m < m1; m += ny) {
      const f32x4_t d = get(dY + m * cols + n);
      f32x4_t z = {0.f, 0.f, 0.f, 0.f}, u = z;
      if (Z) z = get(Z + m * N + n);
      if constexpr (GATED) u = get(Z + m * N + cols + n);
      f32x4_t g = act_slopes(act, z) * d;
      if constexpr (GATED) {
        g *= u;
        u = act_values(act, z) * d;
      }
      if (dZ) {
        store4<uint16_t>(dZ + m * N, n, cols, g, true);
        if constexpr (GATED) store4<uint16_t>(dZ + m * N, cols + n, N, u, true);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        sum[i] += g[i];
        if constexpr (GATED) sum[4 + i] += u[i];
      }
    }
  }
  if (!dbias) return;
  dbias += (int64_t)blockIdx.y * N;
#pragma unroll
  for (int i = 0; i < W; ++i) part[(y * LANES + c) * W + i] = sum[i];
  __syncthreads();
  for (int k = threadIdx.x; k < LANES * W; k += 1024) {
    float v = 0.f;
    for (int r = 0; r < ny; ++r) v += part[r * LANES * W + k];
    const int at = ((int)blockIdx.x * LANES + k / W) * 4 + k % 4;
    if (at < cols) dbias[k % W >= 4 ? cols + at : at] = v;
  }
}

// Workgroups that share the rows of a column: without column sums 64 rows each; with them one
// has all, but where columns are few and rows many, whose sums then meet in the workspace.
// Us, one and shared out, the sums' kernel included: 2000 x 8192 gated 50 and 26, 1695 x 15792
// gated 55 and 41, 1000 x 4096 17 and 13; 1024 x 14336 (224 workgroups of columns) is as fast
// as without sums, 38.
static int64_t bias_groups(int64_t M, int64_t N, bool gated) {
  const int64_t blocks = ((gated ? N >> 1 : N) + 63) >> 6;
  if (M < 512 || blocks > 128) return 1;
  const int64_t want = 512 / blocks, most = M >> 6;
  return want < most ? want : most;
}
static int64_t bias_bytes(int64_t groups, int64_t N) { return groups > 1 ? (groups * N * 4 + 255) / 256 * 256 : 0; }

static int launch_parts(const float *parts, int splits, int64_t size, void *out, int out_dtype, hipStream_t s) {
  const dim3 grid((unsigned)((size / 4 + 255) / 256));
  if (out_dtype == NF4_F32)
    hipLaunchKernelGGL((mx_parts_kernel<float>), grid, dim3(256), 0, s, parts, splits, size,
                       static_cast<float *>(out), aligned_to(out, 16));
  else
    hipLaunchKernelGGL((mx_parts_kernel<uint16_t>), grid, dim3(256), 0, s, parts, splits, size,
                       static_cast<uint16_t *>(out), true);
  return launch_status(hipGetLastError());
}

// sums: for bias_groups x N parts of dbias
static int launch_act_grad(const uint16_t *dY, const uint16_t *Z, int64_t M, int64_t N, int act, uint16_t *dZ,
                           float *dbias, float *sums, hipStream_t s) {
  const bool gated = is_gated(act);
  const int64_t cols = gated ? N / 2 : N;
  const int64_t groups = dbias ? bias_groups(M, N, gated) : (M + 63) >> 6;
  const int64_t rows = (M + groups - 1) / groups, used = (M + rows - 1) / rows;
  const dim3 grid((unsigned)((cols + 63) / 64), (unsigned)used);
  float *const to = dbias && used > 1 ? sums : dbias;
  if (gated)
    hipLaunchKernelGGL((mx_act_grad_kernel<true>), grid, dim3(1024), 0, s, dY, Z, M, (int)N, act, rows, dZ, to);
  else
    hipLaunchKernelGGL((mx_act_grad_kernel<false>), grid, dim3(1024), 0, s, dY, Z, M, (int)N, act, rows, dZ, to);
  if (int r = launch_status(hipGetLastError())) return r;
  return dbias && used > 1 ? launch_parts(sums, (int)used, N, dbias, NF4_F32, s) : NF4_OK;
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
  nf4::mx::GradArgs a{codes, scales, dY, offsets, dX, R, (int)E, (int)N, (int)K, {}, 0, 1, nullptr};
  return nf4::mx::launch_rows_grad(a, out_dtype, (hipStream_t)stream);
}

int64_t nf4_mx_linear_grad_workspace_bytes(int64_t N, int64_t K, int64_t M) {
  if (nf4::check_mx_shape(N, K) || N % 8 != 0 || N > (int64_t(1) << 23) || M < 1 || M > (int64_t(1) << 21))
    return -1;
  const int64_t n = nf4::mx::grad_splits(M, N, K);
  return (n > 1 ? n * M * K * 4 : 0) + nf4::mx::bias_bytes(nf4::mx::bias_groups(M, N, true), N);
}

int nf4_mx_linear_grad(const uint8_t *codes, const uint8_t *scales, int64_t N, int64_t K, const uint16_t *dY,
                       const uint16_t *Z, int act, int64_t M, uint16_t *dZ, float *dbias, void *dX,
                       int out_dtype, void *workspace, int64_t workspace_bytes, void *stream) {
  using namespace nf4::mx;
  const bool plain = act == NF4_ACT_NONE;
  if (!codes || !scales || !dY || !dX || !nf4::known_dtype(out_dtype) || !known_act(act) ||
      (!plain && (!Z || !dZ)))
    return NF4_EINVAL;
  if (int r = nf4::check_mx_shape(N, K)) return r;
  if (N % 8 != 0) return NF4_EINVAL;
  // so that every launch below holds its tiles
  if (M < 1 || M > (int64_t(1) << 21) || N > (int64_t(1) << 23)) return NF4_ERANGE;
  if (!nf4::aligned_to(codes, 16) || !nf4::aligned_to(dY, 16) || !nf4::aligned_to(Z, 16) ||
      !nf4::aligned_to(dZ, 16) || !nf4::aligned_to(dX, 16) || !nf4::aligned_to(dbias, 4) ||
      !nf4::aligned_to(workspace, 256))
    return NF4_EALIGN;
  const DensePlan plan = plan_dense(M, N, K);
  const int splits = plan.splits;
  const int64_t sums = dbias ? bias_bytes(bias_groups(M, N, is_gated(act)), N) : 0;
  const int64_t need = sums + (splits > 1 ? splits * M * K * 4 : 0);
  if (need > 0 && (!workspace || workspace_bytes < need)) return NF4_ERANGE;
  if (int r = nf4::device_status()) return r;
  hipStream_t s = (hipStream_t)stream;
  if (!plain || dZ || dbias)
    if (int r = launch_act_grad(dY, plain ? nullptr : Z, M, N, act, dZ, dbias, static_cast<float *>(workspace), s))
      return r;
  const uint16_t *d = plain ? dY : dZ;
  if (splits == 1) {
    GradArgs a{codes, scales, d, nullptr, dX, M, 1, (int)N, (int)K, {}, 0, 1, nullptr};
    return launch_plan(plan, a, out_dtype, s);
  }
  float *parts = reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + sums);
  GradArgs a{codes, scales, d, nullptr, parts, M, 1, (int)N, (int)K, {}, N, splits, nullptr};
  if (int r = launch_plan(plan, a, out_dtype, s)) return r;
  return launch_parts(parts, splits, M * K, dX, out_dtype, s);
}

}  // extern "C"
