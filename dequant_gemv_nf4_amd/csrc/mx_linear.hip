// mx_linear.hip -- product of bf16 rows with a packed MXFP4 matrix, with bias, activation,
// gate and residual applied to the sums before they leave the workgroup (gfx950):
//   z[m][n] = sum_k X[m][k] v(n,k) + bias[n];  Y = act(z) + residual
// or, gated, Y[m][i] = act(z[m][i]) z[m][N/2 + i] + residual[m][i].
// The sums are those of mx_product.h.  A gated product takes the rows of both halves in
// turn, so that gate and gated value are neighbouring columns of one workgroup.
// Bound as the plain products are, the epilogue hides behind another workgroup's products.
// Us on six cards, from the caches and (in brackets) with weights from memory: 28672 x 4096,
// gated, M = 1: 14.3 (16.7, without the gate 13.9); M = 1021 with z kept: 197-210 (208-218;
// 1.1-1.22 PFLOP/s); 4096 x 4096 with residual, M = 1: 5.7 (5.8, without 4.9); 333 x 13824 x
// 5120 with bias and gelu in fp32: 60-65 (63-68; 0.7-0.78 PFLOP/s: 432 tiles of 96 x 128, of
// which the chip holds 512).
#include "mx_act.h"
#include "mx_product.h"

namespace nf4 {
namespace mx {

template <bool PAIRS>
struct LinearOut {
  static constexpr bool kPairs = PAIRS, kPlain = false;
  const void *bias;      // fp32 or bf16 [N], or null
  const void *residual;  // [M][columns of Y] of Y's type, or null
  uint16_t *Z;           // bf16 [M][N], or null
  int act, bias_bf16;

  __device__ __forceinline__ float bias_at(int n) const {
    return bias_bf16 ? __uint_as_float((uint32_t) reinterpret_cast<const uint16_t *>(bias)[n] << 16)
                     : reinterpret_cast<const float *>(bias)[n];
  }
  // The bias of four outputs from column n of Y on, and of what a gated one multiplies them with.
  struct Bias {
    f32x4_t z, zu;
  };
  __device__ __forceinline__ Bias bias_of(const Args &p, int n) const {
    Bias b{{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    if (bias) {
      const int cols = PAIRS ? p.N >> 1 : p.N;
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (n + i < cols) {
          b.z[i] = bias_at(n + i);
          if (PAIRS) b.zu[i] = bias_at(cols + n + i);
        }
    }
    return b;
  }
  // z[0 .. 3] at columns n .. n + 3 of row m of the matrix's N columns; adds the bias and keeps z
  __device__ __forceinline__ f32x4_t take(const Args &p, int64_t m, int n, int end, f32x4_t z, f32x4_t b,
                                          bool vec) const {
    if (bias) z += b;
    if (Z) {
      uint16_t *row = Z + m * p.N;
      store4<uint16_t>(row, n, end, z, vec);
    }
    return z;
  }
  template <typename OUT>
  __device__ __forceinline__ void put(const Args &p, int64_t m, int n, int cols, f32x4_t y, bool vec) const {
    if (residual) {
      const OUT *r = reinterpret_cast<const OUT *>(residual) + m * cols + n;
      if (vec) {
        if (n < cols) {
          if constexpr (sizeof(OUT) == 4) {
            y += *reinterpret_cast<const f32x4_t *>(r);
          } else {
            const u32x2_t w = *reinterpret_cast<const u32x2_t *>(r);
            y += f32x4_t{bf16_lo(w[0]), bf16_hi(w[0]), bf16_lo(w[1]), bf16_hi(w[1])};
          }
        }
      } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (n + i < cols) {
            if constexpr (sizeof(OUT) == 4)
              y[i] += r[i];
            else
              y[i] += __uint_as_float((uint32_t)r[i] << 16);
          }
      }
    }
    store4<OUT>(reinterpret_cast<OUT *>(p.Y) + m * cols, n, cols, y, vec);
  }
  // Four outputs from column n of Y on; zu: what a gated product multiplies them with.
  template <typename OUT>
  __device__ __forceinline__ void finish(const Args &p, int64_t m, int n, f32x4_t z, f32x4_t zu,
                                         const Bias &b) const {
    const int cols = PAIRS ? p.N >> 1 : p.N;
    const bool vec = (cols & 3) == 0;
    z = take(p, m, n, cols, z, b.z, vec);
    f32x4_t y = act_values(act, z);
    if constexpr (PAIRS) y *= take(p, m, cols + n, p.N, zu, b.zu, vec);
    put<OUT>(p, m, n, cols, y, vec);
  }

  template <typename OUT, class ROWS, class SUM>
  __device__ __forceinline__ void rows_out(const Args &p, const ROWS &, const RowTile &t, int n0, int cols,
                                           const SUM &sum) const {
    constexpr int W = PAIRS ? 8 : 4;  // columns of four outputs
    const int quads = (cols + W - 1) / W;
    for (int i = threadIdx.x; i < quads * t.rows; i += blockDim.x) {
      const int m = i / quads, r = (i - m * quads) * W;
      f32x4_t z = {0.f, 0.f, 0.f, 0.f}, zu = z;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int c = r + j * (W / 4);
        if (c < cols) z[j] = sum(m, c);
        if (PAIRS && c < cols) zu[j] = sum(m, c + 1);
      }
      const int n = (PAIRS ? n0 >> 1 : n0) + r / (W / 4);
      finish<OUT>(p, t.row0 + m, n, z, zu, bias_of(p, n));
    }
  }
  template <int MF, int NF, int WV, int KG, typename OUT, int BYTES, class ROWS>
  __device__ __forceinline__ void tile_out(const Args &p, const ROWS &, const RowTile &t, int n0, int wave,
                                           int kg, const f32x4_t (&acc)[NF][MF], uint8_t *lds) const {
    typedef TileRows<MF, NF, WV, KG, BYTES> T;
    T::each(wave, kg, acc, lds, [&](const float *z, int m0, int rows) __attribute__((always_inline)) {
      constexpr int W = PAIRS ? 8 : 4, quads = T::kCols / W, kThreads = 64 * WV * KG;
      const int n = min(rows, t.rows - m0) * quads;
      const auto first = [&](int r) __attribute__((always_inline)) { return PAIRS ? (n0 + r) >> 1 : n0 + r; };
      // a thread's columns are the same in all rows, but in tiles of 192: the bias is read once
      // (1021 x 28672 x 4096, gated, with bias, on one card: 227 us read for each row, 212 so;
      // 194-211 on four others, 193-209 without bias)
      constexpr bool kFixed = kThreads % quads == 0;
      Bias b = bias_of(p, first((int)threadIdx.x % quads * W));
#pragma unroll 1
      for (int i = threadIdx.x; i < n; i += kThreads) {
        const int m = i / quads, r = i % quads * W;
        if (n0 + r >= p.N) continue;
        if (!kFixed) b = bias_of(p, first(r));
        const float *s = z + m * T::kPitch + r;
        const f32x4_t a = *reinterpret_cast<const f32x4_t *>(s);
        if constexpr (PAIRS) {
          const f32x4_t c = *reinterpret_cast<const f32x4_t *>(s + 4);
          finish<OUT>(p, t.row0 + m0 + m, first(r), f32x4_t{a[0], a[2], c[0], c[2]},
                      f32x4_t{a[1], a[3], c[1], c[3]}, b);
        } else {
          finish<OUT>(p, t.row0 + m0 + m, first(r), a, a, b);
        }
      }
    });
  }
};

template <bool PAIRS>
static int linear(const Args &a, int out_dtype, const LinearOut<PAIRS> &epi, hipStream_t s) {
  Product<SortedRows, LinearOut<PAIRS>, true, true> p{a, false, out_dtype, {}, epi, s};
  return launch_product(p);
}

}  // namespace mx
}  // namespace nf4

extern "C" {

int nf4_mx_linear(const uint8_t *codes, const uint8_t *scales, int64_t N, int64_t K, const uint16_t *X,
                  int64_t M, const void *bias, int bias_dtype, int act, const void *residual, void *Y,
                  int out_dtype, uint16_t *Z, void *stream) {
  if (!codes || !scales || !X || !Y || !nf4::known_dtype(out_dtype) || !nf4::mx::known_act(act) ||
      (bias && !nf4::known_dtype(bias_dtype)))
    return NF4_EINVAL;
  if (int r = nf4::check_mx_shape(N, K)) return r;
  const bool gated = nf4::mx::is_gated(act);
  if (gated && N % 2 != 0) return NF4_EINVAL;
  if (M < 1 || M >= (int64_t(1) << 26)) return NF4_ERANGE;
  if (!nf4::aligned_to(codes, 16) || !nf4::aligned_to(X, 16) || !nf4::aligned_to(Y, 16) ||
      !nf4::aligned_to(residual, 16) || !nf4::aligned_to(Z, 16) ||
      !nf4::aligned_to(bias, bias_dtype == NF4_BF16 ? 2 : 4))
    return NF4_EALIGN;
  // with nothing after it the product itself: its kernels, and its bits
  if (act == NF4_ACT_NONE && !bias && !residual && !Z)
    return nf4_mx_gemm(codes, scales, N, K, X, M, Y, out_dtype, stream);
  if (int r = nf4::device_status()) return r;
  const nf4::mx::Args a{codes, scales, X, nullptr, Y, M, 1, (int)N, (int)K, {}};
  hipStream_t s = (hipStream_t)stream;
  if (gated)
    return nf4::mx::linear<true>(a, out_dtype, {bias, residual, Z, act, bias_dtype == NF4_BF16}, s);
  return nf4::mx::linear<false>(a, out_dtype, {bias, residual, Z, act, bias_dtype == NF4_BF16}, s);
}

}  // extern "C"
