// mx_gemm.hip -- products of bf16 rows with packed MXFP4 matrices, dense and
// grouped by expert (gfx950):
//   Y[i][n] = sum_k X[i][k] * v(e(i), n, k),  v = element * 2^(scale - 127).
#include "mx_product.h"

namespace nf4 {
namespace mx {

using PlainProduct = Product<SortedRows, PlainOut, true, true>;

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
  nf4::mx::PlainProduct p{{codes, scales, X, nullptr, Y, M, 1, (int)N, (int)K, {}}, false, out_dtype, {}, {},
                          (hipStream_t)stream};
  return nf4::mx::launch_product(p);
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
  nf4::mx::PlainProduct p{{codes, scales, X, offsets, Y, R, (int)E, (int)N, (int)K, {}}, true, out_dtype, {}, {},
                          (hipStream_t)stream};
  return nf4::mx::launch_product(p);
}

}  // extern "C"
