// Host sanitizer run of the argument checks of the MXFP4 and routing entry points:
// sizes around every limit, null and misaligned pointers, built (host code only)
// with AddressSanitizer and UndefinedBehaviorSanitizer.  Without a GPU every call
// that passes its checks stops at the device check, so no kernel is launched;
// pointers are fake addresses that are never dereferenced.
#include <cstdint>
#include <cstdio>

#include "nf4.h"

static int bad = 0;
static void expect(const char *what, int64_t got, int64_t want) {
  if (got != want) {
    std::printf("%s: got %lld, want %lld\n", what, (long long)got, (long long)want);
    bad = 1;
  }
}
static void refused(const char *what, int got) {
  if (got == NF4_OK || got == NF4_ELAUNCH) {
    std::printf("%s: passed the device check without a device (%d)\n", what, got);
    bad = 1;
  }
}

int main() {
  auto P = reinterpret_cast<void *>(uintptr_t(0x100000));
  auto *c = static_cast<uint8_t *>(P);
  auto *h = static_cast<uint16_t *>(P);
  auto *i = static_cast<int32_t *>(P);
  auto *id = static_cast<int64_t *>(P);
  auto *f = static_cast<float *>(P);
  const int64_t top = INT64_MAX;
  const int64_t Ns[] = {-top, -1, 0, 1, 8, 4096, int64_t(1) << 23, int64_t(1) << 31, top};
  const int64_t Ks[] = {-32, 0, 31, 32, 96, 4096, 32768, 32800, top - 31, top};
  const int64_t Rs[] = {-top, -1, 0, 1, 512, (int64_t(1) << 26) - 1, int64_t(1) << 26, top};
  for (int64_t N : Ns)
    for (int64_t K : Ks)
      for (int dtype : {-1, 0, 1, 2}) {
        refused("pack", nf4_mx_pack(P, dtype, N, K, c, c, i, nullptr));
        refused("unpack", nf4_mx_unpack(c, c, N, K, P, dtype, nullptr));
        for (int64_t R : Rs) {
          refused("gemm", nf4_mx_gemm(c, c, N, K, h, R, P, dtype, nullptr));
          refused("packed", nf4_mx_gemm_packed(c, c, N, K, c, c, R, P, dtype, nullptr));
          for (int64_t E : {int64_t(-1), int64_t(1), int64_t(512), int64_t(513), top}) {
            refused("grouped", nf4_mx_gemm_grouped(c, c, E, N, K, h, i, R, P, dtype, nullptr));
            refused("grad", nf4_mx_gemm_grouped_grad(c, c, E, N, K, h, i, R, P, dtype, nullptr));
          }
        }
      }
  const int64_t Ts[] = {-top, -1, 0, 1, (int64_t(1) << 24) - 1, int64_t(1) << 24, top};
  for (int64_t T : Ts)
    for (int64_t topk : {-top, int64_t(0), int64_t(1), int64_t(64), int64_t(512), int64_t(513), top}) {
      for (int64_t E : {-top, int64_t(0), int64_t(1), int64_t(512), int64_t(513), top})
        refused("sort", nf4_moe_sort(id, T, topk, E, i, i, i, i, nullptr));
      for (int64_t H : {-top, int64_t(0), int64_t(1), int64_t(1) << 20, (int64_t(1) << 20) + 1, top})
        for (int dtype : {0, 1, 5}) {
          refused("gather", nf4_moe_gather(P, dtype, i, T, topk, H, P, nullptr));
          refused("combine", nf4_moe_combine(P, dtype, i, nullptr, T, topk, H, P, nullptr));
          refused("combine_grad",
                  nf4_moe_combine_grad(P, P, dtype, i, f, T, topk, H, P, f, nullptr));
        }
    }
  expect("gemm null X", nf4_mx_gemm(c, c, 4, 32, nullptr, 1, P, 0, nullptr), NF4_EINVAL);
  expect("gemm odd codes", nf4_mx_gemm(c + 8, c, 4, 32, h, 1, P, 0, nullptr), NF4_EALIGN);
  expect("grad N % 8", nf4_mx_gemm_grouped_grad(c, c, 1, 12, 32, h, i, 1, P, 0, nullptr), NF4_EINVAL);
  expect("sort odd ids", nf4_moe_sort(reinterpret_cast<int64_t *>(i + 1), 1, 1, 1, i, i, i, nullptr,
                                      nullptr), NF4_EALIGN);
  expect("combine odd rows", nf4_moe_combine(c + 1, 1, i, f, 1, 1, 8, P, nullptr), NF4_EALIGN);
  std::printf("mx abi sanitizer run: %s\n", bad ? "FAILED" : "ok");
  return bad;
}
