// mx_loss.hip -- softmax cross entropy of X . dequant(W)^T, W a packed head of a large
// vocabulary, and its gradient in X, without the logits in memory (gfx950):
//   l[m][n] = sum_k X[m][k] v(n,k);  lse = log sum_n exp l;  loss = lse - l[target]
//   dX[m][k] = dloss[m] (sum_n exp(l - lse) v(n,k) - v(target,k))
//            = dloss[m] (sum_(n != target) exp(l - lse) v(n,k) - (1 - p) v(target,k)),
// p the target's probability.  The second form is the one computed, with 1 - p as the others'
// sum over the whole: for a token that the model predicts well both terms of the first are
// nearly one, and the gradient would be what their rounding leaves.  The loss is, for such a
// token, log(1 + the others' sum / the target's).
//
// The vocabulary goes in pieces.  Of each piece
//  1. the product's tiles (mx_product.h) take exp2(l log2(e) - c) of their logits, c a whole
//     number, at least the strip's largest exponent and the row's so far; the strip's c and
//     sum stay, and for the gradient the values, at most 1, in bf16, which is what the matrix
//     cores take (so each has its full relative precision however far below the row's maximum
//     its strip lies, and the gradient in bf16 is as near to 64 bits as one of fp32 values:
//     1.6e-3 of its norm); the target's is left out of both, its logit is kept;
//  2. a row's strips meet in the row's new c and sum; strips with a smaller c are moved to
//     it by a subtraction in the exponents of their values;
//  3. the values' product with the piece's matrix (mx_grad.hip) is added to the row's sum
//     over the vocabulary, which the change of c scales, exactly.
// So the logits are computed once, 4 M N K operations with the gradient where a second pass
// over them takes 6.  Last, the sums are divided by the row's, the target's row is taken
// off, and dloss applied.
// Bound by the products (the exponentials run beside another workgroup's matrix
// instructions).  Us of 128256 x 4096, on six cards: 1000 rows 757-811 (1.3-1.39 PFLOP/s; up to
// 832 in a trace); 2047 rows with the gradient, four pieces, 3380-3640 (1.18-1.27): 390-410 a
// piece the logits, 413-450 their product back, 9 the join, 13-17 moving strips (most of it in
// the first piece, where the maximum is found).  With the gradient, few rows, weights from
// memory: 1 row 150, 8 157, 64 195-209 (without 99), 200 460-485 (without 214-230); of 32000 x
// 4096 51, 50, 74 and 145.  32000 x 4096, 5 rows: 13.5-14.5 (4.8-5.1 TB/s) and 4-5.
#include "mx_grad.h"
#include "mx_product.h"

namespace nf4 {
namespace mx {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kNoMax = -3.4028234664e38f;  // c of a row before its first logit: nothing is below

struct Strip {
  float c, sum;
};

// Takes a tile's logits: strips of the 16 NF columns of a wave.
struct LossOut {
  static constexpr bool kPairs = false, kPlain = false;
  const int64_t *targets;  // of the rows
  int64_t first;           // the piece's first column
  const float *c;          // the rows' so far, or null
  float *target_logit;
  Strip *strips;  // [strip][M]
  uint16_t *P;    // [M][ld], or null
  int64_t ld;

  template <int MF, int NF, int WV, int KG, typename OUT, int BYTES, class ROWS>
  __device__ __forceinline__ void tile_out(const Args &p, const ROWS &, const RowTile &t, int n0, int wave,
                                           int kg, const f32x4_t (&acc)[NF][MF], uint8_t *) const {
    if (KG > 1 && kg > 0) return;
    const int lane = threadIdx.x & 63, l16 = lane & 15, q = lane >> 4;
    const int w0 = n0 + wave * 16 * NF;  // the strip's first column
    if (w0 >= p.N) return;
    const int end8 = (p.N + 7) & ~7;  // P is zero from N up to here
    Strip *const out = strips + (int64_t)(w0 / (16 * NF)) * p.R;
#pragma unroll
    for (int r = 0; r < MF; ++r) {
      const int m = r * 16 + l16;
      const bool in = m < t.rows;
      const int64_t row = t.row0 + m;
      f32x4_t l[NF];
      float top = -__builtin_inff();
#pragma unroll
      for (int k = 0; k < NF; ++k) {
        l[k] = acc[k][r];
        if (w0 + 16 * NF > p.N) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (w0 + k * 16 + q * 4 + i >= p.N) l[k][i] = -__builtin_inff();
        }
        top = fmaxf(fmaxf(top, fmaxf(l[k][0], l[k][1])), fmaxf(l[k][2], l[k][3]));
      }
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      const float ref = fmaxf(in && c ? c[row] : kNoMax, __builtin_ceilf(top * kLog2e));
      const int64_t at = in ? targets[row] - first - w0 : -1;
      if (at >= 0 && at < 16 * NF && w0 + at < p.N) {
#pragma unroll
        for (int k = 0; k < NF; ++k)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            if (k * 16 + q * 4 + i == at) {
              target_logit[row] = l[k][i];
              l[k][i] = -__builtin_inff();
            }
      }
      float sum = 0.f;
#pragma unroll
      for (int k = 0; k < NF; ++k) {
#pragma unroll
        for (int i = 0; i < 4; ++i) l[k][i] = __builtin_amdgcn_exp2f(__builtin_fmaf(l[k][i], kLog2e, -ref));
        sum += (l[k][0] + l[k][1]) + (l[k][2] + l[k][3]);
        if (P && in) {
          const int n = w0 + k * 16 + q * 4;
          if (n < end8)
            *reinterpret_cast<u32x2_t *>(P + row * ld + n) = u32x2_t{
                bf16_bits(l[k][0]) | (bf16_bits(l[k][1]) << 16), bf16_bits(l[k][2]) | (bf16_bits(l[k][3]) << 16)};
        }
      }
      sum += __shfl_xor(sum, 16, 64);
      sum += __shfl_xor(sum, 32, 64);
      if (in && q == 0) out[row] = Strip{ref, sum};
    }
  }
};

constexpr int kStrip = 16;  // columns of the narrowest strip
struct LossProduct : Product<SortedRows, LossOut, false, true> {
  int strip = 0;  // columns of a strip, set by the launch
  template <int MF, int NF, int WV, int KS, int KW, int KG>
  int tile() {
    strip = 16 * NF;
    return this->Product::template tile<MF, NF, WV, KS, KW, KG>();
  }
  // Up to two rows (four of a small head), where the plain product takes its row kernel.  Us,
  // one row, weights from memory, against one K-group, which five rows take: 32000 x 4096 22-24
  // and 21, 128256 x 4096 75 and 69, 50257 x 1600 28 and 21.
  template <int TR>
  int gemv() {
    return tile<1, 1, 4, 4, 4, 2>();
  }
};
// Two sums with their references, as one.
__device__ __forceinline__ Strip join(Strip a, Strip b) {
  const float c = fmaxf(a.c, b.c);
  return {c, a.sum * __builtin_amdgcn_exp2f(a.c - c) + b.sum * __builtin_amdgcn_exp2f(b.c - c)};
}

struct RowState {  // of a row of X, between pieces; sum: without the target
  float *c, *sum, *rescale, *target_logit, *total;
};

// A row's strips of a piece: ROWS rows a workgroup, which share out the strips.  Writes
// the row's c and sum, the factor for what is summed so far, and for each strip how far
// its exponents have to go down.  `loss` (after the last piece): the outputs.
// 16 rows read whole lines of the strips; of few rows four a workgroup, so that each has
// more threads: 5 rows of 32000 columns 3.9 us, with 16 11.
constexpr int kJoinThreads = 1024;
template <int ROWS>
__global__ void __launch_bounds__(kJoinThreads)
    mx_loss_join_kernel(const Strip *__restrict__ strips, int n, int M, int first_piece, RowState rows,
                        uint8_t *__restrict__ down, const int64_t *__restrict__ targets, int64_t N,
                        float *__restrict__ loss, float *__restrict__ lse, int32_t *status) {
  constexpr int kShares = kJoinThreads / ROWS;
  __shared__ Strip part[kShares][ROWS];
  const int r = threadIdx.x % ROWS, share = threadIdx.x / ROWS;
  const int m = blockIdx.x * ROWS + r;
  Strip v{kNoMax, 0.f};
  if (m < M)
    for (int i0 = share; i0 < n; i0 += 8 * kShares) {
      Strip s[8];  // loads that do not wait for one another
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int i = i0 + k * kShares;
        s[k] = i < n ? strips[(int64_t)i * M + m] : Strip{kNoMax, 0.f};
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) v = join(v, s[k]);
    }
  part[share][r] = v;
  __syncthreads();
#pragma unroll
  for (int d = kShares / 2; d > 0; d >>= 1) {
    if (share < d) part[share][r] = join(part[share][r], part[share + d][r]);
    __syncthreads();
  }
  Strip all = part[0][r];
  float before = kNoMax;
  if (!first_piece && m < M) {
    before = rows.c[m];
    all = join(Strip{before, rows.sum[m]}, all);
  }
  __syncthreads();  // every thread of the row has read c before it changes
  if (m >= M) return;
  if (share == 0) {
    rows.c[m] = all.c;
    rows.sum[m] = all.sum;
    rows.rescale[m] = __builtin_amdgcn_exp2f(before - all.c);
    if (loss) {
      const int64_t t = targets[m];
      const bool counts = t >= 0 && t < N;
      const float l = counts ? rows.target_logit[m] : 0.f;
      const float own = counts ? __builtin_amdgcn_exp2f(__builtin_fmaf(l, kLog2e, -all.c)) : 0.f;
      const float total = all.sum + own;
      const float log = __builtin_fmaf(__builtin_amdgcn_logf(total), kLn2, all.c * kLn2);
      rows.total[m] = total;
      lse[m] = log;
      loss[m] = !counts ? 0.f : all.sum < own ? log1pf(all.sum / own) : log - l;
      if (t >= N && status) atomicOr(status, NF4_LOSS_BAD_TARGET);
    }
  }
  if (down)
    for (int i = share; i < n; i += kShares)
      down[(int64_t)m * n + i] = (uint8_t)fminf(all.c - strips[(int64_t)i * M + m].c, 255.f);
}

// Values of strips that are to go down: their exponents less `down`, at least 0.
__global__ void __launch_bounds__(256)
    mx_loss_down_kernel(const uint8_t *__restrict__ down, int n, int width, uint16_t *__restrict__ P, int64_t ld) {
  typedef uint16_t u16x8 __attribute__((ext_vector_type(8)));
  const int64_t m = blockIdx.y;
  const int i = blockIdx.x * 256 + threadIdx.x;  // 8 columns
  const int strip = i * 8 / width;  // (a multiple of 16 columns)
  if (strip >= n || i * 8 >= ld) return;
  const uint32_t d = down[m * n + strip];
  if (d == 0) return;
  u16x8 *at = reinterpret_cast<u16x8 *>(P + m * ld) + i;
  u16x8 v = *at, s = (uint16_t)(d << 7);
  *at = __builtin_elementwise_sub_sat(v, s);
}

// dX = (sum of the parts - the others' sum * the target's row) / the row's whole sum * dloss
template <typename OUT>
__global__ void __launch_bounds__(256)
    mx_loss_grad_kernel(const float *__restrict__ parts, int splits, int64_t M, int K, const float *__restrict__ sum,
                        const float *__restrict__ total, const int64_t *__restrict__ targets, int64_t N, const float *__restrict__ dloss,
                        const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales,
                        OUT *__restrict__ dX) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;  // 8 columns
  const int per = K >> 3;
  const int64_t m = i / per;
  if (m >= M) return;
  const int k = (int)(i - m * per) * 8;
  const int64_t t = targets[m];
  f32x4_t lo = {0.f, 0.f, 0.f, 0.f}, hi = lo;
  if (t >= 0 && t < N) {
    const f32x4_t *at = reinterpret_cast<const f32x4_t *>(parts + m * K + k);
    lo = at[0];
    hi = at[1];
#pragma unroll 4
    for (int s = 1; s < splits; ++s) {
      at += M * K / 4;
      lo += at[0];
      hi += at[1];
    }
    const uint32_t w = *reinterpret_cast<const uint32_t *>(codes + t * (K >> 1) + (k >> 1));
    const u32x4_t v = decode8(w, scale_of(scales[t * (K >> 5) + (k >> 5)]));
    const float inv = 1.f / total[m], rest = sum[m], d = dloss[m];
    lo = (lo - rest * f32x4_t{bf16_lo(v[0]), bf16_hi(v[0]), bf16_lo(v[1]), bf16_hi(v[1])}) * inv * d;
    hi = (hi - rest * f32x4_t{bf16_lo(v[2]), bf16_hi(v[2]), bf16_lo(v[3]), bf16_hi(v[3])}) * inv * d;
  }
  store4<OUT>(dX + m * K, k, K, lo, true);
  store4<OUT>(dX + m * K, k + 4, K, hi, true);
}

__global__ void mx_loss_clear_kernel(int32_t *status) { *status = 0; }

// Rows and columns of a piece, and what of the workspace is whose.
struct LossPlan {
  int64_t rows, cols, ld, splits;
  int64_t p, parts, strips, down, state, bytes;  // offsets; state: 5 floats a row
};
// Up to kLossRows rows at a time, and as many columns as keep the values under kLossBytes,
// which with the piece of the matrix fits the 256 MB of the last cache; without the values,
// the strips' sums, half a byte a logit where strips are narrowest.
constexpr int64_t kLossRows = 4096, kLossBytes = int64_t(128) << 20;
static LossPlan loss_plan(int64_t N, int64_t K, int64_t M, bool grad) {
  LossPlan d;
  const int64_t turns = (M + kLossRows - 1) / kLossRows;
  d.rows = turns == 1 ? M : ((M + turns - 1) / turns + 127) / 128 * 128;
  const int64_t most = kLossBytes * (grad ? 1 : 4) / (2 * d.rows) / 256 * 256;
  const int64_t pieces = (N + most - 1) / most;
  d.cols = pieces == 1 ? N : ((N + pieces - 1) / pieces + 255) / 256 * 256;
  d.ld = (d.cols + 63) / 64 * 64;
  d.splits = grad ? grad_splits(d.rows, d.cols, K) : 0;
  const int64_t n = (d.cols + kStrip - 1) / kStrip;
  int64_t at = 0;
  const auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  d.p = take(grad ? d.rows * d.ld * 2 : 0);
  d.parts = take(d.splits * d.rows * K * 4);
  d.strips = take(n * d.rows * (int64_t)sizeof(Strip));
  d.down = take(grad ? n * d.rows : 0);
  d.state = take(5 * d.rows * 4);
  d.bytes = at;
  return d;
}

static int loss_rows(const LossPlan &d, const uint8_t *codes, const uint8_t *scales, int64_t N, int64_t K,
                     const uint16_t *X, const int64_t *targets, int64_t M, float *loss, float *lse,
                     const float *dloss, void *dX, int out_dtype, uint8_t *ws, int32_t *status, hipStream_t s) {
  float *const state = reinterpret_cast<float *>(ws + d.state);
  const RowState rows{state, state + M, state + 2 * M, state + 3 * M, state + 4 * M};
  Strip *const strips = reinterpret_cast<Strip *>(ws + d.strips);
  uint16_t *const P = dX ? reinterpret_cast<uint16_t *>(ws + d.p) : nullptr;
  uint8_t *const down = dX ? ws + d.down : nullptr;
  float *const parts = reinterpret_cast<float *>(ws + d.parts);
  for (int64_t n0 = 0; n0 < N; n0 += d.cols) {
    const int64_t cols = N - n0 < d.cols ? N - n0 : d.cols;
    const bool first = n0 == 0, last = n0 + cols == N;
    const uint8_t *const pc = codes + n0 * (K / 2), *const ps = scales + n0 * (K / 32);
    LossProduct p;
    p.a = Args{pc, ps, X, nullptr, nullptr, M, 1, (int)cols, (int)K, {}};
    p.grouped = false;
    p.out_dtype = NF4_BF16;
    p.epi = LossOut{targets, n0, first ? nullptr : rows.c, rows.target_logit, strips, P, d.ld};
    p.s = s;
    if (int r = launch_product(p)) return r;
    const int n = (int)((cols + p.strip - 1) / p.strip);
    if (M >= 512)
      hipLaunchKernelGGL((mx_loss_join_kernel<16>), dim3((unsigned)((M + 15) / 16)), dim3(kJoinThreads), 0, s,
                         strips, n, (int)M, first, rows, down, targets, N, last ? loss : nullptr, lse, status);
    else
      hipLaunchKernelGGL((mx_loss_join_kernel<4>), dim3((unsigned)((M + 3) / 4)), dim3(kJoinThreads), 0, s, strips,
                         n, (int)M, first, rows, down, targets, N, last ? loss : nullptr, lse, status);
    if (int r = launch_status(hipGetLastError())) return r;
    if (!dX) continue;
    hipLaunchKernelGGL(mx_loss_down_kernel, dim3((unsigned)((d.ld / 8 + 255) / 256), (unsigned)M), dim3(256), 0, s,
                       down, n, p.strip, P, d.ld);
    if (int r = launch_status(hipGetLastError())) return r;
    if (int r = launch_grad_parts(
            {pc, ps, cols, K, d.rows, d.cols, P, d.ld, M, parts, first ? nullptr : rows.rescale}, s))
      return r;
  }
  if (!dX) return NF4_OK;
  const unsigned blocks = (unsigned)((M * (K / 8) + 255) / 256);
  const int splits = (int)d.splits;
  if (out_dtype == NF4_F32)
    hipLaunchKernelGGL((mx_loss_grad_kernel<float>), dim3(blocks), dim3(256), 0, s, parts, splits, M, (int)K,
                       rows.sum, rows.total, targets, N, dloss, codes, scales, static_cast<float *>(dX));
  else
    hipLaunchKernelGGL((mx_loss_grad_kernel<uint16_t>), dim3(blocks), dim3(256), 0, s, parts, splits, M, (int)K,
                       rows.sum, rows.total, targets, N, dloss, codes, scales, static_cast<uint16_t *>(dX));
  return launch_status(hipGetLastError());
}

}  // namespace mx
}  // namespace nf4

extern "C" {

int64_t nf4_mx_cross_entropy_workspace_bytes(int64_t N, int64_t K, int64_t M, int grad) {
  if (nf4::check_mx_shape(N, K) || N > (int64_t(1) << 23) || M < 1 || M >= (int64_t(1) << 26)) return -1;
  return nf4::mx::loss_plan(N, K, M, grad != 0).bytes;
}

int nf4_mx_cross_entropy(const uint8_t *codes, const uint8_t *scales, int64_t N, int64_t K, const uint16_t *X,
                         const int64_t *targets, int64_t M, float *loss, float *lse, const float *dloss, void *dX,
                         int out_dtype, void *workspace, int64_t workspace_bytes, int32_t *dev_status,
                         void *stream) {
  using namespace nf4::mx;
  if (!codes || !scales || !X || !targets || !loss || !lse || !dX != !dloss || (dX && !nf4::known_dtype(out_dtype)))
    return NF4_EINVAL;
  if (int r = nf4::check_mx_shape(N, K)) return r;
  if (M < 1 || M >= (int64_t(1) << 26) || N > (int64_t(1) << 23)) return NF4_ERANGE;
  if (!nf4::aligned_to(codes, 16) || !nf4::aligned_to(X, 16) || !nf4::aligned_to(dX, 16) ||
      !nf4::aligned_to(targets, 8) || !nf4::aligned_to(loss, 4) || !nf4::aligned_to(lse, 4) ||
      !nf4::aligned_to(dloss, 4) || !nf4::aligned_to(dev_status, 4) || !nf4::aligned_to(workspace, 256))
    return NF4_EALIGN;
  const LossPlan d = loss_plan(N, K, M, dX != nullptr);
  if (!workspace || workspace_bytes < d.bytes) return NF4_ERANGE;
  if (int r = nf4::device_status()) return r;
  hipStream_t s = (hipStream_t)stream;
  if (dev_status) {
    hipLaunchKernelGGL(mx_loss_clear_kernel, dim3(1), dim3(1), 0, s, dev_status);
    if (int r = nf4::launch_status(hipGetLastError())) return r;
  }
  for (int64_t m = 0; m < M; m += d.rows) {
    const int64_t rows = M - m < d.rows ? M - m : d.rows;
    uint8_t *const out = dX ? static_cast<uint8_t *>(dX) + m * K * (out_dtype == NF4_F32 ? 4 : 2) : nullptr;
    if (int r = loss_rows(d, codes, scales, N, K, X + m * K, targets + m, rows, loss + m, lse + m,
                          dloss ? dloss + m : nullptr, out, out_dtype, static_cast<uint8_t *>(workspace),
                          dev_status, s))
      return r;
  }
  return NF4_OK;
}

}  // extern "C"
