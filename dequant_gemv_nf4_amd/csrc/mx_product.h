// mx_product.h -- kernels of bf16 rows times packed MXFP4 matrices (gfx950), from which
// the plain, fused and expert products are compiled:
//   sum_k X[i][k] * v(e(i), n, k),  v = element * 2^(scale - 127).
// v is exact in bf16, so the weights are decoded straight into matrix-core
// fragments (two values an instruction) and every product is exact in fp32.
//
// Fragments (v_mfma_f32_16x16x32_bf16, A = weights, B = rows): a step is 128 k.
// Lane l holds weight row n = l % 16 and the 16 bytes of block q = l / 16, i.e.
// k = 32 q .. 32 q + 31 of the step; MFMA j of the four takes k = 32 q + 8 j ..
// + 7 of both operands, so a code word, a block scale and 16 bytes of X line up
// without any shuffle.  D: lane l holds row i = l % 16, columns 4 (l / 16) .. + 3,
// stored as one vector.
#pragma once

#include "mx_device.h"
#include "mx_plan.h"
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

// What a kernel takes its rows from and does with its sums is compiled in:
//   ROWS  which rows a workgroup has (find; uniform over the workgroup, with LDS that is free
//         until it returns) and where row m
//         of them lies in X (place, a row of `base`), `whole` rows of which there are;
//   EPI   kPairs: weight rows of the two halves of the matrix alternate (0, N/2, 1, N/2 +
//         1, ..), so that a gate and what it gates meet in one lane; kPlain: the sums are
//         the outputs.  Else rows_out (row kernel) and tile_out (tiles) take them.
struct SortedRows {
  __device__ __forceinline__ RowTile find(const Args &p, int slot, int bm, void *) const {
    return find_tile(p.offsets, p.E, p.R, slot, bm);
  }
  __device__ __forceinline__ int64_t base(const RowTile &t) const { return t.row0; }
  __device__ __forceinline__ int whole(const Args &, const RowTile &t) const { return t.rows; }
  __device__ __forceinline__ int place(const RowTile &, int m) const { return m; }
};
struct PlainOut {
  static constexpr bool kPairs = false, kPlain = true;
};

// Row r of a workgroup's columns within the weights from its first on.
template <bool PAIRS>
__device__ __forceinline__ int weight_row(int r, int N) {
  return PAIRS ? (r >> 1) + (r & 1 ? N >> 1 : 0) : r;
}

// ------------------------------------------------------- one to four rows ----
// A wave's load of codes is 1 KiB of one weight row (2048 k, one block a lane), so
// every line is read whole; the lane's 32 values of each row of X stay in
// registers while the wave walks weight rows.  Waves (c, g) of a workgroup:
// chunk c of K, weight rows g, g + G, ... of the workgroup's; chunks' sums meet in
// LDS and are added in order.  A tile is up to TR rows; the walk is compiled for
// one, two and TR of them and chosen by how many there are, so an expert with
// several rows reads its weights once and one with a single row pays for one.
// Bound by memory where the matrix is large, else by starting and filling the pipeline.
// Measured, M = 1, us with weights from memory (TB/s of codes and scales): 57344 x 8192 42.4
// (5.9), 28672 x 4096 13.3 (4.7), 4096 x 14336 8.5 (3.7), 4096 x 4096 4.8 (1.9).  60 rows of
// 64 experts of 4096 x 4096: 53 (5.1).

constexpr int kAhead = 4;  // weight rows a wave has in flight
// Row tiles of one column block that go to one XCD (a group of the grid): a weight row
// that several of them need comes from memory once.
constexpr int kRowTiles = 8;

// The sums over the wave of four values a lane, in 10 instructions (44 one at a
// time): halves, then rows of 16 lanes change places, so each step adds two values'
// parts at once.  The lanes of row r of 16 end with value 2 (r % 2) + r / 2.
__device__ __forceinline__ float sum4(const float (&v)[4]) {
  const auto add = [](auto s) { return __uint_as_float(s[0]) + __uint_as_float(s[1]); };
  const float a = add(__builtin_amdgcn_permlane32_swap(__float_as_uint(v[0]), __float_as_uint(v[1]), false, false));
  const float b = add(__builtin_amdgcn_permlane32_swap(__float_as_uint(v[2]), __float_as_uint(v[3]), false, false));
  float s = add(__builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false));
  s += dpp_f32<0xB1>(s);   // quad_perm [1,0,3,2]
  s += dpp_f32<0x4E>(s);   // quad_perm [2,3,0,1]
  s += dpp_f32<0x141>(s);  // row_half_mirror
  s += dpp_f32<0x140>(s);  // row_mirror
  return s;
}

// MT rows of X (of the TR that `part` is laid out for) against `cols` weight rows.
template <int MT, int TR, bool PAIRS, class ROWS>
__device__ __forceinline__ void walk_rows(const Args &p, const ROWS &rows, const RowTile &t, int n0, int cols,
                                          int chunks, int rows_wg, float *part) {
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int groups = (int)(blockDim.x >> 6) / chunks;
  const int c = wave % chunks, g = wave / chunks;
  const int kb = p.K >> 5, kc = p.K >> 1;
  const int64_t first = (int64_t)t.e * p.N + (PAIRS ? n0 >> 1 : n0);
  const int wrows = PAIRS ? (p.N + cols) >> 1 : cols;  // weight rows the buffers span
  const uint8_t *const cbase = p.codes + first * kc, *const sbase = p.scales + first * kb;
  const __amdgpu_buffer_rsrc_t xrs =
      buffer(p.X + rows.base(t) * p.K, (int64_t)rows.whole(p, t) * p.K * 2);
  const int b = c * 64 + lane;
  const int out = b < kb ? 0 : kOutside;
  const int co = b * 16 | out, so = b | out;
  u32x4_t cw[kAhead];
  uint32_t sb[kAhead];
  // The row is the loads' uniform offset; past the last one the buffers are empty.
  const auto load = [&](int i, int n) __attribute__((always_inline)) {
    const bool in = n < cols;
    const int w = weight_row<PAIRS>(n, p.N);
    cw[i] = __builtin_amdgcn_raw_buffer_load_b128(buffer(cbase, in ? wrows * kc : 0), co, in ? w * kc : 0,
                                                  kLoadStream);
    sb[i] = __builtin_amdgcn_raw_buffer_load_b8(buffer(sbase, in ? wrows * kb : 0), so, in ? w * kb : 0, 0);
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) load(i, g + i * groups);
  u32x4_t x[MT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 4; ++j)
      x[m][j] = __builtin_amdgcn_raw_buffer_load_b128(
          xrs, (rows.place(t, m) * p.K * 2 + b * 64 + j * 16) | out, 0, 0);
  constexpr int RS = 4 / MT;  // weight rows summed together
  const int mine = (lane >> 4 & 1) * 2 + (lane >> 5);
  for (int n = g; n < cols; n += kAhead * groups) {
    float acc[4];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      float *a = acc + i % RS * MT;
#pragma unroll
      for (int m = 0; m < MT; ++m) a[m] = 0.f;
      const float sc = scale_of(sb[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const u32x4_t w = decode8(cw[i][j], sc);
#pragma unroll
        for (int h = 0; h < 4; ++h)
#pragma unroll
          for (int m = 0; m < MT; ++m)
            a[m] = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2_t, (uint32_t)w[h]),
                                                   __builtin_bit_cast(bf16x2_t, (uint32_t)x[m][j][h]),
                                                   a[m], false);
      }
      load(i, n + (kAhead + i) * groups);
      if (i % RS == RS - 1) {
        const float v = sum4(acc);
        const int r = n + (i - (RS - 1) + mine / MT) * groups;
        if ((lane & 15) == 0 && r < cols) part[(c * rows_wg + r) * TR + mine % MT] = v;
      }
    }
  }
}

template <int TR, typename OUT, class ROWS = SortedRows, class EPI = PlainOut>
__global__ void __launch_bounds__(1024)
    mx_gemv_kernel(Args p, int chunks, int rows_wg, ROWS rows, EPI epi) {
  extern __shared__ float part1[];  // [chunk][row of the workgroup][TR]
  int slot, block;
  if (!grid_item(p.grid, &slot, &block)) return;
  const RowTile t = rows.find(p, slot, TR, part1);
  if (t.rows <= 0) return;
  const int n0 = block * rows_wg;
  const int cols = min(rows_wg, p.N - n0);
  if (t.e >= 0) {
    if (t.rows == 1)
      walk_rows<1, TR, EPI::kPairs>(p, rows, t, n0, cols, chunks, rows_wg, part1);
    else if (TR > 2 && t.rows == 2)
      walk_rows<2, TR, EPI::kPairs>(p, rows, t, n0, cols, chunks, rows_wg, part1);
    else
      walk_rows<TR, TR, EPI::kPairs>(p, rows, t, n0, cols, chunks, rows_wg, part1);
  }
  __syncthreads();
  if constexpr (!EPI::kPlain) {
    epi.template rows_out<OUT>(p, rows, t, n0, cols, [&](int m, int r) __attribute__((always_inline)) {
      float v = part1[r * TR + m];
      for (int k = 1; k < chunks; ++k) v += part1[(k * rows_wg + r) * TR + m];
      return v;
    });
    return;
  }
  OUT *Y = reinterpret_cast<OUT *>(p.Y);
  for (int i = threadIdx.x; i < cols * t.rows; i += blockDim.x) {
    const int m = i / cols, r = i - m * cols;
    float v = 0.f;
    if (t.e >= 0) {
      v = part1[r * TR + m];
      for (int k = 1; k < chunks; ++k) v += part1[(k * rows_wg + r) * TR + m];
    }
    OUT *y = Y + (int64_t)(t.row0 + m) * p.N + n0 + r;
    if constexpr (sizeof(OUT) == 4)
      *y = v;
    else
      *y = (OUT)bf16_bits(v);
  }
}

// ----------------------------------------------------------- more rows ----
// A workgroup owns 16 MF rows x 16 NF WV columns; its waves form KG groups of WV that
// share out K, wave w of a group decoding columns 16 NF w .. into registers (no
// weight is decoded twice).  A stage is 64 KS values of k: the rows' tile of X goes
// straight into LDS, three stages in rotation (four or five measured the same), one
// barrier a stage.  Each wave's own
// codes come the same way, 64 KW values of k at a time (loads of whole 64- or 128-byte
// pieces of a row, where fragment-shaped loads from memory would touch a line a
// lane), and a lane's scale bytes for 256 k in one load.
// Bound by the load path into LDS and, for long prompts, by the matrix cores (67 % busy at
// the 2 GHz that the card then runs at).  Measured: 509 x 28672 x 4096 102-107 us (1.12-1.17
// PFLOP/s), 117 with weights from memory; 16382 rows of 8 experts of 14336 x 4096 1457-1538
// (1.25-1.32) from one card to the next; 1003 rows of 32 of 2048 x 2048 27, from memory 31.

// Permutation of a row's 16-byte chunks (XOR).  A 16-byte read is served 16 lanes at
// a time, lanes 0-3, 12-15, 20-27 and so on: rows 0-3 and 12-15 of one lane quarter
// with rows 4-11 of the next.  The permutations put these, too, into 16 different
// columns of the 256 bytes that LDS reads a cycle.  A row of X is 128 KS bytes.
template <int KS>
__device__ __forceinline__ int x_perm(int row) {
  return KS == 1 ? (row >> 1) & 7 : ((row >> 2) & 3) | (row & 3) << 2;
}
// The same for a row of 32 KW bytes of codes, read in words (KS = 1) or 16 bytes.
template <int KS, int KW>
__device__ __forceinline__ int w_perm(int row) {
  return KW == 4 ? (row >> 1) & 7 : KS == 1 ? (row >> 2) & 3 : -(row >> 2) & 3;
}

template <int MF, int NF, int WV, int KS, int KW, int KG, bool SVEC, typename OUT, class ROWS = SortedRows,
          class EPI = PlainOut>
__global__ void __launch_bounds__(64 * WV *KG, 2)
    mx_tile_kernel(Args p, ROWS rows, EPI epi) {
  constexpr bool PAIRS = EPI::kPairs;
  constexpr int BM = 16 * MF, BN = 16 * NF * WV;
  constexpr int SG = 4 / KS;                              // stages per scale load (256 k)
  constexpr int WS = KW / KS;                             // stages per block of codes
  constexpr int NX = 3, NW = WS == 1 ? NX : 2;            // buffers of X and of codes
  constexpr int XB = BM * 128 * KS, WB = BN * 32 * KW;    // bytes of one
  constexpr int XL = MF * KS * 2 / WV, WL = NF * KW / 2;  // loads a wave
  constexpr int XC = 8 * KS, WC = 2 * KW;                 // chunks a row
  // Scales of 256 k: through LDS as well, or (KS = 1, where LDS is full, and rows that
  // are not whole words) in registers
  constexpr bool SL = SVEC && KS > 1;
  constexpr int NS = SG == 1 ? 3 : 2, SB = NF > 2 ? 512 : 256, SLN = SB / 256;
  constexpr int S = SL ? SLN : 0;
  static_assert((WS == 1 || (WS == 2 && KS == 1)) && XL * WV == MF * KS * 2, "stages");
  __shared__ __attribute__((aligned(1024))) uint8_t
      shared[KG][NX * XB + NW * WB + (SL ? NS * SB * WV : 0)];
  int slot, block;
  if (!grid_item(p.grid, &slot, &block)) return;
  const RowTile t = rows.find(p, slot, BM, &shared[0][0]);
  if (t.rows <= 0) return;
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);
  const int wave = wave_all % WV, kg = wave_all / WV;
  const int l16 = lane & 15, q = lane >> 4;
  const int n0 = block * BN;
  const int cols = min(BN, p.N - n0);
  f32x4_t acc[NF][MF];
#pragma unroll
  for (int c = 0; c < NF; ++c)
#pragma unroll
    for (int r = 0; r < MF; ++r) acc[c][r] = f32x4_t{0.f, 0.f, 0.f, 0.f};

  if (t.e >= 0) {
    const int kb = p.K >> 5, kc = p.K >> 1;
    const int64_t first = (int64_t)t.e * p.N + (PAIRS ? n0 >> 1 : n0);
    const int wrows = PAIRS ? (p.N + cols) >> 1 : cols;  // weight rows the buffers span
    // scale groups (256 k), dealt to the K-groups in runs of `per`
    const int sgs = (kb + 7) >> 3, per = (sgs + KG - 1) / KG;
    const int g0 = kg * per;
    uint8_t *const xlds = shared[kg];
    uint8_t *const wlds = shared[kg] + NX * XB + wave * (WB / WV);  // + i * WB: buffer i
    uint8_t *const slds = shared[kg] + NX * XB + NW * WB + wave * (NS * SB);
    const uint32_t xaddr = lds_address(xlds), waddr = lds_address(wlds), saddr = lds_address(slds);
    // Voffsets are fixed; a stage moves the buffers' base.  Only in a stage that
    // K ends in (or past it) chunks are masked.
    int xo[XL], wo[WL];
#pragma unroll
    for (int i = 0; i < XL; ++i) {
      const int idx = (i * WV + wave) * 64 + lane, row = idx / XC;
      xo[i] = rows.place(t, row) * p.K * 2 + (idx % XC ^ x_perm<KS>(row)) * 16;
    }
#pragma unroll
    for (int i = 0; i < WL; ++i) {
      const int idx = i * 64 + lane, row = idx / WC;  // within the wave's own columns
      wo[i] = weight_row<PAIRS>(wave * 16 * NF + row, p.N) * kc + (idx % WC ^ w_perm<KS, KW>(row)) * 16;
    }
    const int xbytes = rows.whole(p, t) * p.K * 2, wbytes = wrows * kc;
    const uint8_t *xbase = reinterpret_cast<const uint8_t *>(p.X + rows.base(t) * p.K);
    const uint8_t *wbase = p.codes + first * kc;
    const auto load_x = [&](int buf, int s) {  // s: stage from the start of K
      const int adv = s * 128 * KS;
      const u32x4_t rs = buffer_words(xbase + adv, max(xbytes - adv, 0));
      const int left = kb * 4 - s * XC;  // chunks of the row from here on
      int o[XL];
#pragma unroll
      for (int i = 0; i < XL; ++i) {
        const int idx = (i * WV + wave) * 64 + lane, row = idx / XC;
        o[i] = xo[i];
        if (left < XC) o[i] = (idx % XC ^ x_perm<KS>(row)) < left ? o[i] : kOutside;
      }
      load_lds16xn<XL, WV * 1024>(rs, xaddr + buf * XB + wave * 1024, o);
    };
    const auto load_w = [&](int buf, int b) {  // b: block of codes
      const int adv = b * 32 * KW;
      const u32x4_t rs = buffer_words(wbase + adv, max(wbytes - adv, 0));
      const int left = kb - b * WC;
      int o[WL];
#pragma unroll
      for (int i = 0; i < WL; ++i) {
        const int idx = i * 64 + lane, row = idx / WC;
        o[i] = wo[i];
        if (left < WC) o[i] = (idx % WC ^ w_perm<KS, KW>(row)) < left ? o[i] : kOutside;
      }
      load_lds16xn<WL, 1024>(rs, waddr + buf * WB, o);
    };
    // Column c * 16 + l16 of the wave has 8 scale bytes a group.  In LDS: NS groups in
    // rotation.  In registers: the three words around them, or two.
    const uint8_t *sbase = p.scales + first * kb;
    const LooseWords loose(sbase, (int64_t)wrows * kb);
    constexpr int SWORDS = SVEC ? 2 : 3;
    u32x2_t sreg[NF];
    uint32_t snext[NF][SWORDS];
    const auto load_scales = [&](int buf, int g) {
      if constexpr (SL) {
        const u32x4_t rs = buffer_words(sbase + g * 8, max(wrows * kb - g * 8, 0));
#pragma unroll
        for (int i = 0; i < SLN; ++i) {
          const int col = i * 32 + (lane >> 1), w = lane & 1;  // 8 bytes a column
          const int o = weight_row<PAIRS>(wave * 16 * NF + col, p.N) * kb + w * 4;
          load_lds4(rs, saddr + buf * SB + i * 256,
                    col < 16 * NF && g * 8 + w * 4 < kb ? o : kOutside);
        }
      } else {
#pragma unroll
        for (int c = 0; c < NF; ++c)
#pragma unroll
          for (int i = 0; i < SWORDS; ++i)
            snext[c][i] =
                loose.fetch(weight_row<PAIRS>(wave * 16 * NF + c * 16 + l16, p.N) * kb + g * 8, i);
      }
    };
    const auto take_scales = [&](int buf, int g) {
      // bytes past the row's end are the next row's, perhaps NaN: as words they go
      const int left = kb - g * 8;
      const uint64_t own = left <= 0 ? 0 : left < 8 ? ~uint64_t(0) >> (64 - 8 * left) : ~uint64_t(0);
#pragma unroll
      for (int c = 0; c < NF; ++c) {
        if constexpr (SL) {
          sreg[c] = *reinterpret_cast<const u32x2_t *>(slds + buf * SB + (c * 16 + l16) * 8);
        } else if constexpr (SVEC) {
          sreg[c] = u32x2_t{snext[c][0], snext[c][1]};
        } else {
          const int o = weight_row<PAIRS>(wave * 16 * NF + c * 16 + l16, p.N) * kb + g * 8;
          sreg[c] = u32x2_t{loose.word(o, snext[c][0], snext[c][1]),
                            loose.word(o, snext[c][1], snext[c][2])};
        }
        if constexpr (!SL) sreg[c] &= u32x2_t{(uint32_t)own, (uint32_t)(own >> 32)};
      }
    };
    const int s0 = g0 * SG;
    load_scales(0, g0);
    load_x(0, s0);
    load_w(0, s0 / WS);
    if constexpr (SL && SG == 1) load_scales(1, g0 + 1);
    load_x(1, s0 + 1);
    if constexpr (WS == 1) load_w(1, s0 + 1);
    int buf = 0, wbuf = 0, sbuf = 0;
    for (int g = g0; g < g0 + per; ++g) {
      if constexpr (!SL) take_scales(0, g);
#pragma unroll
      for (int u = 0; u < SG; ++u) {
        const int s = g * SG + u;
        // in flight may stay what the last stage asked for, which is not of this one
        constexpr int one = XL + WL;
        if (WS == 1)
          SG == 1 || u == 1 ? lds_loads_but<S + one>() : lds_loads_but<one>();
        else
          u % 2 == 0 ? lds_loads_but<XL>() : lds_loads_but<one>();
        __syncthreads();  // stage s is in LDS; the buffer of the last one is free
        if (u == 0) {
          if constexpr (SL) take_scales(sbuf, g);
          if constexpr (SL && SG == 1)
            load_scales(sbuf == 0 ? 2 : sbuf - 1, g + 2);
          else
            load_scales(sbuf ^ 1, g + 1);
        }
        const auto ahead_x = [&]() __attribute__((always_inline)) {
          load_x(buf == 0 ? NX - 1 : buf - 1, s + NX - 1);
        };
        const auto ahead_w = [&]() __attribute__((always_inline)) {
          if constexpr (WS == 1)
            load_w(buf == 0 ? NX - 1 : buf - 1, s + NX - 1);
          else if (u % 2 == 0)
            load_w(wbuf ^ 1, s / 2 + 1);
        };
        const uint8_t *xt = xlds + buf * XB + l16 * 128 * KS;
        const uint8_t *wt = wlds + (WS == 1 ? buf : wbuf) * WB + l16 * 32 * KW;
        if constexpr (KS == 1) {
          // 64 k: MFMA j has k = 32 j + 8 q .. + 7, one word of block j.  The order is held:
          // four fragments of X are read ahead of their products, the second block is
          // decoded between the first one's, and the next stages' loads go out once the
          // matrix cores are fed (16382 rows of 8 experts of 14336 x 4096: 1520 -> 1450 us,
          // the loads alone 1515 -> 1450; 509 x 28672 x 4096: 123 -> 112).
          constexpr int half = KW == 1 ? 0 : 2, RB = 4;
          uint32_t w[NF][2];
#pragma unroll
          for (int c = 0; c < NF; ++c)
#pragma unroll
            for (int j = 0; j < 2; ++j)
              w[c][j] = *reinterpret_cast<const uint32_t *>(
                  wt + c * 512 * KW + ((u % 2 * half + j) ^ w_perm<KS, KW>(l16)) * 16 + q * 4);
          u32x4_t b[RB], a[2][NF];
          const auto read = [&](int t) __attribute__((always_inline)) {
            b[t % RB] = *reinterpret_cast<const u32x4_t *>(
                xt + t % MF * 2048 + ((t / MF * 4 + q) ^ x_perm<1>(l16)) * 16);
          };
          const auto decode = [&](int j, int c) __attribute__((always_inline)) {
            a[j][c] = decode8(w[c][j], scale_of((sreg[c][u >> 1] >> (16 * (u & 1) + 8 * j)) & 0xffu));
          };
          static_assert(MF >= NF && MF > 5, "the second block is decoded in the first one's time");
#pragma unroll
          for (int t = 0; t < RB; ++t) read(t);
#pragma unroll
          for (int c = 0; c < NF; ++c) decode(0, c);
#pragma unroll
          for (int t = 0; t < 2 * MF; ++t) {
#pragma unroll
            for (int c = 0; c < NF; ++c) acc[c][t % MF] = mfma16(a[t / MF][c], b[t % RB], acc[c][t % MF]);
            if (t + RB < 2 * MF) read(t + RB);
            if (t < NF) decode(1, t);
            if (t == 5) ahead_x();
            if (t == 8) ahead_w();
            __builtin_amdgcn_sched_barrier(0);
          }
        } else {
#pragma unroll
          for (int kk = 0; kk < KS / 2; ++kk) {  // 128 k: lane q has block q
            u32x4_t w[NF];
            float sc[NF];
#pragma unroll
            for (int c = 0; c < NF; ++c) {
              w[c] = *reinterpret_cast<const u32x4_t *>(
                  wt + c * 512 * KW + (((kk * 4 + q) ^ w_perm<KS, KW>(l16)) * 16));
              sc[c] = scale_of((sreg[c][KS == 4 ? kk : u] >> (8 * q)) & 0xffu);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              u32x4_t a[NF];
#pragma unroll
              for (int c = 0; c < NF; ++c) a[c] = decode8(w[c][j], sc[c]);
#pragma unroll
              for (int r = 0; r < MF; ++r) {
                const u32x4_t b = *reinterpret_cast<const u32x4_t *>(
                    xt + r * 2048 * KS + (((kk * 16 + q * 4 + j) ^ x_perm<KS>(l16)) * 16));
#pragma unroll
                for (int c = 0; c < NF; ++c) acc[c][r] = mfma16(a[c], b, acc[c][r]);
              }
              // the next stages' loads go out once the matrix cores are fed (256 x 28672 x
              // 4096 73.6 -> 70.3 us, 2000 x 4096 x 4096 74.5 -> 71)
              if (kk == 0 && j == 0) ahead_x();
              if (kk == 0 && j == 1) ahead_w();
            }
          }
        }
        buf = buf == NX - 1 ? 0 : buf + 1;
        if (u % 2 == 1) wbuf ^= 1;
      }
      sbuf = SG == 1 ? (sbuf == 2 ? 0 : sbuf + 1) : sbuf ^ 1;
    }
    lds_loads_but<0>();  // the loads past the end have landed, too
  }
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
    if constexpr (EPI::kPlain)
      if (kg > 0) return;
#pragma unroll
    for (int g = 0; g < KG - 1; ++g)
#pragma unroll
      for (int c = 0; c < NF; ++c)
#pragma unroll
        for (int r = 0; r < MF; ++r)
          acc[c][r] += part[((g * WV + wave) * NF * MF + c * MF + r) * 64 + lane];
  }
  if constexpr (!EPI::kPlain) {
    epi.template tile_out<MF, NF, WV, KG, OUT, sizeof(shared)>(p, rows, t, n0, wave, kg, acc, &shared[0][0]);
    return;
  }
  OUT *Y = reinterpret_cast<OUT *>(p.Y);
  const bool vec = (p.N & 3) == 0;
#pragma unroll
  for (int r = 0; r < MF; ++r) {
    const int m = r * 16 + l16;
    if (m >= t.rows) continue;
    OUT *row = Y + (int64_t)(t.row0 + m) * p.N;
#pragma unroll
    for (int c = 0; c < NF; ++c)
      store4<OUT>(row, n0 + (wave * NF + c) * 16 + q * 4, p.N, acc[c][r], vec);
  }
}

// A product with its rows and outputs, launched by the kernels below.  F32, B16: the
// output types that it is compiled for.
template <class ROWS, class EPI, bool F32, bool B16>
struct Product {
  Args a;
  bool grouped;
  int out_dtype;
  ROWS rows;
  EPI epi;
  hipStream_t s;
  static constexpr bool kPlain = EPI::kPlain;

  template <int TR, typename OUT>
  int gemv_as(unsigned n, int threads, size_t lds, int chunks, int wrows) {
    hipLaunchKernelGGL((mx_gemv_kernel<TR, OUT, ROWS, EPI>), dim3(n), dim3(threads), lds, s, a, chunks,
                       wrows, rows, epi);
    return launch_status(hipGetLastError());
  }
  template <int TR>
  int gemv() {
    const int64_t slots = slots_for(a.R, a.E, grouped, TR);
    // Weight rows a workgroup.  Dense 16 (4096 x 14336, M = 1: 9.3 us; 8 rows 9.6; 32 13.4).
    // Grouped, where tiles that turn out empty start workgroups as well: 128 (30 rows of 16
    // experts of 4096 x 4096: 28.3; 32 rows 29.7), or 32 where those would be few (8 of 8 of
    // 2048 x 2048: 6.3; 128 rows 11.5).
    const int wrows = !grouped ? 16 : slots * ((a.N + 127) / 128) >= 640 ? 128 : 32;
    const int chunks = (a.K + 2047) / 2048;
    // 8 waves, or 4 where there are plenty of workgroups: 28672 x 4096, M = 1: 13.7 us with
    // 4 waves, 14.8 with 8; 4096 x 4096: 5.8, 5.4
    const int waves = slots * a.N >= 8192 ? 4 : 8;
    const int groups = chunks >= waves ? 1 : waves / chunks;
    a.grid = make_grid(slots, (a.N + wrows - 1) / wrows, kRowTiles);
    const int64_t n = grid_size(a.grid);
    const int threads = 64 * chunks * groups;
    if (n * threads >= (int64_t(1) << 32)) return NF4_ERANGE;
    const size_t lds = (size_t)chunks * wrows * TR * 4;
    if constexpr (F32)
      if (out_dtype == NF4_F32) return gemv_as<TR, float>((unsigned)n, threads, lds, chunks, wrows);
    if constexpr (B16)
      if (out_dtype == NF4_BF16) return gemv_as<TR, uint16_t>((unsigned)n, threads, lds, chunks, wrows);
    return NF4_EINVAL;
  }

  template <int MF, int NF, int WV, int KS, int KW, int KG, bool SVEC>
  int tile_as() {
    a.grid = make_grid(slots_for(a.R, a.E, grouped, 16 * MF), (a.N + 16 * NF * WV - 1) / (16 * NF * WV), 8);
    const int64_t n = grid_size(a.grid);
    if (n * 64 * WV * KG >= (int64_t(1) << 32)) return NF4_ERANGE;
    if constexpr (F32)
      if (out_dtype == NF4_F32) {
        hipLaunchKernelGGL((mx_tile_kernel<MF, NF, WV, KS, KW, KG, SVEC, float, ROWS, EPI>),
                           dim3((unsigned)n), dim3(64 * WV * KG), 0, s, a, rows, epi);
        return launch_status(hipGetLastError());
      }
    if constexpr (B16)
      if (out_dtype == NF4_BF16) {
        hipLaunchKernelGGL((mx_tile_kernel<MF, NF, WV, KS, KW, KG, SVEC, uint16_t, ROWS, EPI>),
                           dim3((unsigned)n), dim3(64 * WV * KG), 0, s, a, rows, epi);
        return launch_status(hipGetLastError());
      }
    return NF4_EINVAL;
  }
  template <int MF, int NF, int WV, int KS, int KW, int KG>
  int tile() {
    if (a.K % 128 == 0 && aligned_to(a.scales, 4)) return tile_as<MF, NF, WV, KS, KW, KG, true>();
    return tile_as<MF, NF, WV, KS, KW, KG, false>();
  }
};

// The tiles of dense_tile().
template <class P>
static int launch_dense_tile(P &p) {
  switch (dense_tile(p.a.R, p.a.N, p.a.K)) {
    case 0: return p.template tile<8, 4, 4, 1, 2, 1>();
    case 1: return p.template tile<8, 3, 4, 1, 2, 1>();
    case 2: return p.template tile<8, 2, 4, 1, 2, 1>();
    case 3: return p.template tile<6, 2, 4, 1, 2, 1>();
    case 4: return p.template tile<4, 2, 4, 2, 2, 1>();
    case 5: return p.template tile<2, 2, 4, 2, 2, 1>();
    case 6: return p.template tile<2, 1, 4, 4, 4, 1>();
    case 7: return p.template tile<2, 1, 4, 4, 4, 2>();
    case 8: return p.template tile<1, 1, 4, 4, 4, 1>();
    case 9: return p.template tile<1, 1, 4, 4, 4, 2>();
    default: return p.template tile<1, 1, 2, 4, 4, 4>();
  }
}

// The kernel for a product: the largest tile that is not mostly empty and still gives the
// CUs enough of them, else a smaller one with K shared out inside the workgroup (K-groups).
// Measured, us, M x N x K or rows of experts of N x K, weights from memory (in brackets:
// tiles of the kind taken):
//   taken                    case                               others
//   row kernel, 2 rows       2 x 4096 x 14336          9.7      16 x 32: 14.7
//   row kernel, 4 rows       4 x 4096 x 14336         12.9      16 x 32: 15.0
//                            4 x 6144 x 4096           9.6      16 x 32: 7.2
//   128 x 256                2000 x 4096 x 4096 (256)   68      64 x 128: 74
//                            256 x 28672 x 4096 (224)   68      64 x 128: 74
//   128 x 256, grouped       1000 of 8 of 14336 x 4096 159      64 x 128: 171
//   64 x 128                 1500 x 4096 x 4096         58      128 x 256 (192): 65
//                            640 x 4096 x 4096 (320)  34.6      32 x 128: 35.8, 64 x 64: 41.2
//                            64 x 28672 x 4096 (224)  29.4      32 x 128: 32.6, 64 x 64: 32.8
//   64 x 128, grouped        800 of 8 of 14336 x 4096  137      128 x 256: 154, 32 x 128: 155
//   32 x 128, grouped        1003 of 32 of 2048 x 2048  31      64 x 128: 32.7, 32 x 64: 36.8
//   32 x 64                  256 x 4096 x 4096 (512)  18.4      64 x 128: 23.5, two K-groups: 20.7
//   32 x 64, two K-groups    100 x 4096 x 4096 (256)  11.7      one: 13.6, 16 x 64: 14.1
//   16 x 64                  16 x 28672 x 4096 (448)  20.8      two K-groups: 21.1
//   16 x 64, two K-groups    16 x 10240 x 4096 (160)   9.1      one: 11.1, 16 x 32: 12.6
//   16 x 32, four K-groups   16 x 8192 x 4096 (256)    8.0      16 x 64, two: 9.0
//                            8 x 4096 x 14336 (128)   15.8      16 x 64, two: 23.2; two: 19.3
template <class P>
static int launch_product(P &p) {
  const Args &a = p.a;
  const bool grouped = p.grouped;
  const auto tiles = [&](int bm, int bn) {
    return slots_for(a.R, a.E, grouped, bm) * ((a.N + bn - 1) / bn);
  };
  // rows an expert has on average; popular ones have more
  const int64_t mean = grouped ? (a.R + a.E - 1) / a.E : a.R;
  const int64_t rows = grouped ? mean + mean / 2 : mean;
  // Up to kRowTiles rows, in one group of the grid: an expert's weights come from memory
  // once even if every row has a tile of its own, and the tiles work side by side.  Beyond
  // that two groups on two XCDs would read them.  One row a tile against two, us, weights
  // from memory, experts drawn at random / with falling shares / all rows one expert's:
  //   28672 x 4096, 8 rows of 8:   61.9 59.6 43.3    64.7 64.5 44.2
  //                 9 rows of 8:   84.0 81.0 69.5    64.7 63.8 57.2
  //   4096 x 14336, 8 rows of 64:  38.9 36.7 24.4    41.1 40.8 25.2
  //                 9 rows of 64:  54.8 53.0 41.3    48.8 44.5 35.0
  //   2048 x 2048,  8 rows of 8:    6.3  6.1  5.7     6.8  6.7  6.4
  //                 9 rows of 8:    8.0  7.9  7.5     7.0  6.8  6.3
  // Fewer rows: between 20 % faster and 8 % slower, but for 5 rows that are all one
  // expert's (28672 x 4096: 34.2 against 28.0).
  if (mean <= 1 && a.R <= kRowTiles) return p.template gemv<1>();
  if (mean <= 2) return p.template gemv<2>();
  if (mean <= 4 && tiles(16, 64) < 256) return p.template gemv<4>();
  constexpr int kBig = 208, kFill = 384, kSplit = 192;
  if constexpr (!P::kPlain)
    if (!grouped && rows > 16) return launch_dense_tile(p);
  // grouped, each expert leaves one that is partly empty
  if (rows > (grouped ? 150 : 64) && tiles(128, 256) >= (grouped ? kFill : kBig))
    return p.template tile<8, 4, 4, 1, 2, 1>();
  if (rows > 48 && tiles(64, 128) >= kSplit) return p.template tile<4, 2, 4, 2, 2, 1>();
  if (rows > 16) {
    if (tiles(32, 128) >= kFill) return p.template tile<2, 2, 4, 2, 2, 1>();
    if (tiles(32, 64) >= kFill) return p.template tile<2, 1, 4, 4, 4, 1>();
    if (tiles(32, 64) >= kSplit) return p.template tile<2, 1, 4, 4, 4, 2>();
  }
  if (tiles(16, 64) >= kFill) return p.template tile<1, 1, 4, 4, 4, 1>();
  if (tiles(16, 32) > 256) return p.template tile<1, 1, 4, 4, 4, 2>();
  return p.template tile<1, 1, 2, 4, 4, 4>();
}

}  // namespace mx
}  // namespace nf4
