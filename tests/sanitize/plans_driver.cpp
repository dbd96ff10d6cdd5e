// The host's choices of tiles (mx_plan.h), for the sizes on standard input: "t M N K" a dense
// product with an epilogue, "g M N K" a dense gradient.
#include <cstdio>

#include "mx_plan.h"

int main() {
  char kind;
  long long M, N, K;
  while (std::scanf(" %c %lld %lld %lld", &kind, &M, &N, &K) == 4) {
    if (kind == 't') {
      std::printf("%d\n", nf4::mx::dense_tile(M, N, K));
    } else {
      const nf4::mx::DensePlan d = nf4::mx::plan_dense(M, N, K);
      std::printf("%d %d %d %d\n", d.mf, d.wv, d.kg, d.splits);
    }
  }
}
