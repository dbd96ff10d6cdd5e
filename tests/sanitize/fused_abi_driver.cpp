// Host sanitizer run of the argument checks and workspace sizes of the fused MXFP4 entry
// points: sizes around and far beyond every limit, null and misaligned pointers, built (host
// code only) with AddressSanitizer and UndefinedBehaviorSanitizer.  Without a GPU every call
// that passes its checks stops at the device check, so no kernel is launched; pointers are
// fake addresses that are never dereferenced.
#include <cstdint>
#include <cstdio>

#include "nf4.h"

static int bad = 0;
static void refused(const char *what, int got) {
  if (got == NF4_OK || got == NF4_ELAUNCH) {
    std::printf("%s: passed the device check without a device (%d)\n", what, got);
    bad = 1;
  }
}
static void sane(const char *what, int64_t got) {
  if (got < -1 || got > (int64_t(1) << 44)) {
    std::printf("%s: %lld bytes\n", what, (long long)got);
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
  const int64_t Ns[] = {-top, -1, 0, 1, 8, 4096, 128256, int64_t(1) << 23, (int64_t(1) << 23) + 8, int64_t(1) << 31, top};
  const int64_t Ks[] = {-32, 0, 31, 32, 96, 4096, 32768, 32800, top - 31, top};
  const int64_t Ms[] = {-top, -1, 0, 1, 17, 512, 4096, 4097, int64_t(1) << 21, (int64_t(1) << 26) - 1, int64_t(1) << 26, top};
  for (int64_t N : Ns)
    for (int64_t K : Ks)
      for (int64_t M : Ms) {
        sane("linear_grad", nf4_mx_linear_grad_workspace_bytes(N, K, M));
        for (int grad : {0, 1}) sane("loss", nf4_mx_cross_entropy_workspace_bytes(N, K, M, grad));
        for (int64_t bytes : {int64_t(-1), int64_t(0), top}) {
          for (int act = -1; act <= 7; ++act) {
            refused("linear_grad", nf4_mx_linear_grad(c, c, N, K, h, h, act, M, h, f, P, 1, P, bytes, nullptr));
            refused("linear", nf4_mx_linear(c, c, N, K, h, M, P, act & 1, act, P, P, 0, h, nullptr));
          }
          refused("loss", nf4_mx_cross_entropy(c, c, N, K, h, id, M, f, f, nullptr, nullptr, 0, P, bytes, i, nullptr));
          refused("loss grad", nf4_mx_cross_entropy(c, c, N, K, h, id, M, f, f, f, P, 1, P, bytes, i, nullptr));
        }
      }
  const int64_t Hs[] = {-32, 0, 32, 48, 4096, 32768, 32800, top};
  for (int64_t H : Hs)
    for (int64_t I : Hs)
      for (int64_t E : {-top, int64_t(0), int64_t(1), int64_t(8), int64_t(512), int64_t(513), top})
        for (int64_t T : {-top, int64_t(1), int64_t(16), int64_t(17), int64_t(64), int64_t(65), top})
          for (int64_t topk : {-top, int64_t(0), int64_t(1), int64_t(512), int64_t(513), top})
            for (int act : {-1, 0, 5, 7}) {
              sane("moe", nf4_moe_mlp_workspace_bytes(E, H, I, act, T, topk));
              refused("moe", nf4_moe_mlp(c, c, c, c, E, H, I, h, id, f, T, topk, act, P, P, 0, P, top, nullptr));
            }
  std::printf("fused abi sanitizer run: %s\n", bad ? "FAILED" : "ok");
  return bad;
}
