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

// A workgroup owns 16 NF WN columns x 16 MF WM rows; its waves form KG groups of WN x WM
// that share out K.  A stage is 128 KS values of k: 64 KS bytes a row of either operand,
// loaded straight into LDS, NB stages in rotation, one barrier a stage (whole 128-byte
// pieces: 64-byte ones and a stage more in flight took 8 % longer).  Scales come
// the same way, 16 bytes (512 k) a row.  Bound by the loads of both operands and, where
// the output is large, by writing it after the last stage.  Measured: 4096 x 28672 x 4096
// 318-335 us (2.9-3.0 PFLOP/s, the matrix cores 34 % busy; 75-85 us are the 470 MB of Y),
// 37 x 6144 x 4096 6.9 us.

// Permutation (XOR) of the 16-byte chunks of a row of 64 KS bytes: the rows that LDS
// serves together in a fragment read (0-3 and 12-15 of one lane quarter with 4-11
// of the next) fall into different banks.
template <int KS>
__device__ __forceinline__ int row_perm(int row) {
  return KS == 2 ? (row >> 1) & 7 : ((row >> 2) & 3) | (row & 3) << 2;
}

template <int WN, int WM, int NF, int MF, int KS, int KG, int NB, bool SVEC, typename OUT>
__global__ void __launch_bounds__(64 * WN *WM *KG, NF *MF > 16 ? 1 : 2) mx_packed_kernel(PackedArgs p) {
  constexpr int WV = WN * WM, BN = 16 * NF * WN, BM = 16 * MF * WM, ROWS = BN + BM;
  constexpr int RB = 64 * KS, RC = 4 * KS, RL = 1024 / RB;  // bytes and chunks a row, rows a load
  constexpr int TB = ROWS * RB, L = TB / 1024 / WV;  // bytes of a stage, loads a wave
  constexpr int SG = 4 / KS;                         // stages per scale load
  constexpr int S = (ROWS + 64 * WV - 1) / (64 * WV), SB = S * WV * 1024, NS = SG == 1 ? 3 : 2;
  static_assert(L * WV * 1024 == TB && BN % 64 == 0, "whole loads");
  __shared__ __attribute__((aligned(1024))) uint8_t shared[KG][NB * TB + NS * SB];
  int slot, block;
  if (!grid_item(p.grid, &slot, &block)) return;
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wave = wave_all % WV, kg = wave_all / WV;
  const int l16 = lane & 15, q = lane >> 4;
  const int wn = wave % WN, wm = wave / WN;
  const int n0 = block * BN, cols = min(BN, p.N - n0);
  const int64_t m0 = (int64_t)slot * BM;
  const int rows = (int)min((int64_t)BM, p.M - m0);
  const int kb = p.K >> 5, kc = p.K >> 1;
  const uint8_t *const wbase = p.codes + (int64_t)n0 * kc, *const xbase = p.xcodes + m0 * kc;
  const uint8_t *const wsbase = p.scales + (int64_t)n0 * kb, *const xsbase = p.xscales + m0 * kb;
  f32x4_t acc[NF][MF];
#pragma unroll
  for (int c = 0; c < NF; ++c)
#pragma unroll
    for (int r = 0; r < MF; ++r) acc[c][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  const int groups = (kb + 15) >> 4, per = (groups + KG - 1) / KG, g0 = kg * per;
  uint8_t *const tiles = shared[kg], *const slds = shared[kg] + NB * TB;
  const uint32_t taddr = lds_address(tiles), saddr = lds_address(slds);
  // load i of a wave: RL rows from row (i * WV + wave) * RL on, of W up to BN, then of X
  int vo[L];
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int row = (i * WV + wave) * RL + lane / RC;
    vo[i] = (row < BN ? row : row - BN) * kc + ((lane % RC) ^ row_perm<KS>(row)) * 16;
  }
  const auto load_stage = [&](int buf, int s) {
    const int adv = s * RB;
    const u32x4_t wrs = buffer_words(wbase + adv, max(cols * kc - adv, 0));
    const u32x4_t xrs = buffer_words(xbase + adv, max(rows * kc - adv, 0));
    const int left = kb - s * RC;
    int o[L];
#pragma unroll
    for (int i = 0; i < L; ++i) {
      o[i] = vo[i];
      if (left < RC)
        o[i] = ((lane % RC) ^ row_perm<KS>((i * WV + wave) * RL + lane / RC)) < left ? o[i] : kOutside;
    }
    const uint32_t at = taddr + buf * TB + wave * 1024;
    const auto rs = [&](int i) { return (i * WV + wave) * RL < BN ? wrs : xrs; };
#pragma unroll
    for (int i = 0; i + 1 < L; i += 2)
      load_lds16x2<WV * 1024>(rs(i), rs(i + 1), at + i * WV * 1024, o[i], o[i + 1]);
    if constexpr (L % 2 == 1) load_lds16(rs(L - 1), at + (L - 1) * WV * 1024, o[L - 1]);
  };
  uint32_t sreg[S][5];
  const auto load_scales = [&](int buf, int g) {
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int row0 = (i * WV + wave) * 64;
      const bool w = row0 < BN;
      const int o = (row0 + lane - (w ? 0 : BN)) * kb;
      if constexpr (SVEC) {  // rows are whole words
        const u32x4_t rs = buffer_words((w ? wsbase : xsbase) + g * 16, max((w ? cols : rows) * kb - g * 16, 0));
        load_lds16(rs, saddr + buf * SB + row0 * 16, o);
      } else {
        const LooseWords loose(w ? wsbase : xsbase, (int64_t)(w ? cols : rows) * kb);
#pragma unroll
        for (int k = 0; k < 5; ++k) sreg[i][k] = loose.fetch(o + g * 16, k);
      }
    }
  };
  const auto put_scales = [&](int buf, int g) {  // !SVEC
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const int row0 = (i * WV + wave) * 64;
      const bool w = row0 < BN;
      const LooseWords loose(w ? wsbase : xsbase, 0);
      const int o = (row0 + lane - (w ? 0 : BN)) * kb + g * 16;
      u32x4_t v;
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = loose.word(o, sreg[i][k], sreg[i][k + 1]);
      *reinterpret_cast<u32x4_t *>(slds + buf * SB + (row0 + lane) * 16) = v;
    }
  };
  // The fragments of 128 k: lane l has row l % 16 and block l / 16 of either operand.
  struct Frags {
    u32x4_t a[NF], b[MF];
    uint32_t as[NF], bs[MF];
  };
  const auto read = [&](Frags &f, int buf, int sbuf, int u, int s, int h) __attribute__((always_inline)) {
    const uint8_t *wt = tiles + buf * TB + (wn * 16 * NF + l16) * RB;
    const uint8_t *xt = tiles + buf * TB + (BN + wm * 16 * MF + l16) * RB;
    const uint8_t *ws = slds + sbuf * SB + (wn * 16 * NF + l16) * 16 + (u * KS + h) * 4;
    const uint8_t *xs = slds + sbuf * SB + (BN + wm * 16 * MF + l16) * 16 + (u * KS + h) * 4;
    // scale bytes past the row's end are the next row's, perhaps NaN
    const int left = kb - (s * KS + h) * 4;
    const uint32_t own = left >= 4 ? ~0u : left <= 0 ? 0u : ~0u >> (32 - 8 * left);
    const int ch = ((h * 4 + q) ^ row_perm<KS>(l16)) * 16;
#pragma unroll
    for (int r = 0; r < MF; ++r) {
      f.b[r] = *reinterpret_cast<const u32x4_t *>(xt + r * 16 * RB + ch);
      f.bs[r] = (*reinterpret_cast<const uint32_t *>(xs + r * 256) & own) >> (8 * q);
    }
#pragma unroll
    for (int c = 0; c < NF; ++c) {
      f.a[c] = *reinterpret_cast<const u32x4_t *>(wt + c * 16 * RB + ch);
      f.as[c] = (*reinterpret_cast<const uint32_t *>(ws + c * 256) & own) >> (8 * q);
    }
  };
  const auto multiply = [&](const Frags &f) __attribute__((always_inline)) {
#pragma unroll
    for (int c = 0; c < NF; ++c)
#pragma unroll
      for (int r = 0; r < MF; ++r) acc[c][r] = mfma_scaled(f.a[c], f.as[c], f.b[r], f.bs[r], acc[c][r]);
  };
  constexpr int ss = SVEC ? S : 0;
  int buf = 0, sbuf = 0;
  load_scales(0, g0);
  load_stage(0, g0 * SG);
  if constexpr (SVEC && SG == 1) load_scales(1, g0 + 1);
#pragma unroll
  for (int i = 1; i < NB - 1; ++i) load_stage(i, g0 * SG + i);
  for (int g = g0; g < g0 + per; ++g) {
#pragma unroll
    for (int u = 0; u < SG; ++u) {
      const int s = g * SG + u;
      if (!SVEC && u == 0) put_scales(sbuf, g);
      // in flight may stay (NB = 3) the next stage and the scales asked for before it
      if (NB == 2)
        lds_loads_but<0>();
      else
        SG == 1 || u == 1 ? lds_loads_but<L + ss>() : lds_loads_but<L>();
      __syncthreads();  // stage s is in LDS; the buffer of the last one is free
      if (u == 0) {
        if constexpr (SVEC && SG == 1)
          load_scales(sbuf == 0 ? 2 : sbuf - 1, g + 2);
        else
          load_scales(sbuf == NS - 1 ? 0 : sbuf + 1, g + 1);
      }
      load_stage(buf == 0 ? NB - 1 : buf - 1, s + NB - 1);
#pragma unroll
      for (int h = 0; h < KS; ++h) {
        Frags f;
        read(f, buf, sbuf, u, s, h);
        multiply(f);
      }
      buf = buf == NB - 1 ? 0 : buf + 1;
    }
    sbuf = sbuf == NS - 1 ? 0 : sbuf + 1;
  }
  lds_loads_but<0>();
  if constexpr (KG > 1) {
    static_assert(sizeof(shared) >= (KG - 1) * WV * 64 * NF * MF * 16, "partial tiles fit the stages");
    f32x4_t *part = reinterpret_cast<f32x4_t *>(&shared[0][0]);  // [kg - 1][wave][f][lane]
    __syncthreads();
    if (kg > 0)
#pragma unroll
      for (int c = 0; c < NF; ++c)
#pragma unroll
        for (int r = 0; r < MF; ++r)
          part[(((kg - 1) * WV + wave) * NF * MF + c * MF + r) * 64 + lane] = acc[c][r];
    __syncthreads();
    if (kg > 0) return;
#pragma unroll
    for (int g = 0; g < KG - 1; ++g)
#pragma unroll
      for (int c = 0; c < NF; ++c)
#pragma unroll
        for (int r = 0; r < MF; ++r)
          acc[c][r] += part[((g * WV + wave) * NF * MF + c * MF + r) * 64 + lane];
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

template <int WN, int WM, int NF, int MF, int KS, int KG, int NB, bool SVEC>
static int launch_packed_as(PackedArgs &a, int out_dtype, hipStream_t s) {
  constexpr int BN = 16 * NF * WN, BM = 16 * MF * WM, NT = 64 * WN * WM * KG;
  a.grid = make_grid((a.M + BM - 1) / BM, (a.N + BN - 1) / BN, 8);
  const int64_t n = grid_size(a.grid);
  if (n * NT >= (int64_t(1) << 32)) return NF4_ERANGE;
  if (out_dtype == NF4_F32)
    hipLaunchKernelGGL((mx_packed_kernel<WN, WM, NF, MF, KS, KG, NB, SVEC, float>), dim3((unsigned)n),
                       dim3(NT), 0, s, a);
  else
    hipLaunchKernelGGL((mx_packed_kernel<WN, WM, NF, MF, KS, KG, NB, SVEC, uint16_t>), dim3((unsigned)n),
                       dim3(NT), 0, s, a);
  return launch_status(hipGetLastError());
}

template <int WN, int WM, int NF, int MF, int KS, int KG, int NB>
static int launch_tile(PackedArgs &a, int out_dtype, hipStream_t s) {
  if (a.K % 128 == 0 && aligned_to(a.scales, 4) && aligned_to(a.xscales, 4))
    return launch_packed_as<WN, WM, NF, MF, KS, KG, NB, true>(a, out_dtype, s);
  return launch_packed_as<WN, WM, NF, MF, KS, KG, NB, false>(a, out_dtype, s);
}

// The largest tile that is not mostly empty and leaves few CUs without one, else a
// small one with K shared out inside the workgroup (K-groups).  Measured, us, M x N x K,
// weights from memory (in brackets: tiles of the kind taken):
//   taken                    case                               others
//   256 x 256                4096 x 28672 x 4096 (1792)  335    128 x 128: 371
//                            4096 x 4096 x 4096 (256)     52    128 x 128: 60
//   128 x 128                2048 x 4096 x 14336 (512)    87    256 x 256 (128): 119, 64 x 128: 116
//   64 x 128                 512 x 4096 x 4096 (256)    14.3    128 x 128: 18.7
//                            64 x 28672 x 4096 (224)    18.7    64 x 64, two K-groups: 22.0
//   64 x 64, two K-groups    256 x 4096 x 4096 (256)     9.8    64 x 128: 13.1, 32 x 64, two: 13.2
//   32 x 64, two             37 x 6144 x 4096 (192)      7.6    64 x 64, two: 8.6; 16 x 64: 8.5
//   16 x 64                  1 x 28672 x 4096 (448)     14.0    two K-groups: 16.7
//   16 x 64, two             16 x 4096 x 14336 (64)     13.4    one: 19.3; 32 x 64, two: 15.3
static int launch_packed(PackedArgs &a, int out_dtype, hipStream_t s) {
  const auto tiles = [&](int bm, int bn) {
    return ((a.M + bm - 1) / bm) * ((a.N + bn - 1) / bn);
  };
  constexpr int kFill = 192;
  if (a.M > 128 && tiles(256, 256) >= kFill)
    return launch_tile<2, 4, 8, 4, 2, 1, 2>(a, out_dtype, s);
  if (a.M > 64 && tiles(128, 128) >= kFill) return launch_tile<2, 2, 4, 4, 2, 1, 2>(a, out_dtype, s);
  if (a.M > 32) {
    if (tiles(64, 128) >= kFill) return launch_tile<2, 2, 4, 2, 2, 1, 3>(a, out_dtype, s);
    if (tiles(64, 64) >= kFill) return launch_tile<2, 2, 2, 2, 2, 2, 3>(a, out_dtype, s);
  }
  if (a.M > 16 && tiles(32, 64) >= 64) return launch_tile<4, 1, 1, 2, 2, 2, 3>(a, out_dtype, s);
  if (tiles(16, 64) >= 384) return launch_tile<4, 1, 1, 1, 4, 1, 2>(a, out_dtype, s);
  return launch_tile<4, 1, 1, 1, 4, 2, 3>(a, out_dtype, s);
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
  return nf4::mx::launch_packed(a, out_dtype, (hipStream_t)stream);
}

}  // extern "C"
