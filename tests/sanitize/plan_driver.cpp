// Driver for the attention's launch plan and layouts (decode_plan.hpp), on the host
// alone (test infrastructure).
#include <cstdio>

#include "../../sparse_gemm_linears_amd/csrc/decode_plan.hpp"

using namespace fp8lin;

static int g_bad = 0;
#define EXPECT(cond)                                                        \
  do {                                                                      \
    if (!(cond)) {                                                          \
      std::fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
      g_bad = 1;                                                            \
    }                                                                       \
  } while (0)

// Every head of every wave starts on 16 bytes (its accesses are that wide), and
// the three parts neither overlap nor leave the allocation.
template <int D>
static void boxes() {
  constexpr int kHead = RowBoxOf<D>::kHead;
  EXPECT(kHead >= D && kHead % 4 == 0);
  for (int waves : {1, 2, 4, 8}) {
    for (int heads = 1; heads <= 32; heads++) {
      const RowBox box = RowBoxOf<D>::at(waves, heads);
      const int n = waves * heads;
      const int begin[3] = {box.o, box.m, box.l}, size[3] = {n * kHead, n, n};
      if (box.o % 4) std::fprintf(stderr, "D %d, %d waves of %d heads: o at float %d\n", D, waves, heads, box.o);
      EXPECT(box.o % 4 == 0);
      for (int i = 0; i < 3; i++) {
        EXPECT(begin[i] >= 0 && begin[i] + size[i] <= box.floats);
        for (int j = 0; j < i; j++) EXPECT(begin[i] >= begin[j] + size[j] || begin[j] >= begin[i] + size[i]);
      }
    }
  }
}

int main() {
  boxes<64>();
  boxes<128>();
  boxes<256>();
  if (!g_bad) std::printf("decode plan driver: ok\n");
  return g_bad;
}
