// Driver for the attention's launch plan and layouts (decode_plan.hpp), on the host
// alone (test infrastructure).
#include <cstdio>
#include <cstdlib>

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

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A plan's kernel exists, its parts cover the longest row, its counts fit their
// types and grids; and every kernel that exists is some plan's.
static void plans() {
  long checked = 0;
  bool met[3][3][9] = {}, by_row[3][3] = {}, by_share[3][3] = {};  // [D 64, 128, 256][sets of heads][waves]
  const int lens[] = {0, 1, 32, 33, 64, 65, 96, 97, 128, 300, 512, 513, 800, 1025, 3000, 4096, 20000, 100000, 1 << 30};
  for (int cus : {32, 64, 256, 304}) {
    for (int B : {1, 2, 3, 17, 64, 255, 300, 4096, 65535}) {
      for (int Hkv : {1, 2, 8, 40, 1024}) {
        for (int group : {1, 4, 16, 17, 32, 33, 128}) {
          if (Hkv * group > 1024) continue;
          for (int d = 0; d < 3; d++) {
            for (int len : lens) {
              for (int window : {0, 1, 17, 18, 50, 1000, 4000, 2147483647}) {
                for (int fp8 = 0; fp8 < 2; fp8++) {
                  float scale = 0.f;
                  DecodeArgs a{};
                  a.B = B;
                  a.Hq = Hkv * group;
                  a.Hkv = Hkv;
                  a.D = 64 << d;
                  a.max_len = len;
                  a.window = window;
                  if (fp8) a.k_scale = a.v_scale = &scale;
                  const DecodePlan p = plan_decode(a, cus);
                  const int RT = row_tiles(a);
                  checked++;
                  int64_t tiles = 1;  // of the longest row, wherever its window ends in a half tile
                  for (int n = len; n > 0 && n > len - 16; n--) {
                    const int64_t t = ceil_div((int64_t)n - first_token(n, window), kTile);
                    tiles = t > tiles ? t : tiles;
                  }
                  EXPECT(p.rows == (int64_t)B * Hkv * ceil_div(group, 16 * RT));
                  EXPECT(p.owners > 0 && p.first_row == 0);
                  if (p.row_waves) {
                    EXPECT(has_row_form(a.D, RT, p.row_waves));
                    EXPECT(p.splits >= 1 && p.per >= 1 && p.splits * p.per >= tiles);
                    EXPECT(p.owners == p.rows * p.splits && p.by_row == (p.splits > 1));
                    EXPECT(p.splits == 1 || p.owners <= kRowGrid);
                    const int heads = group < 16 * RT ? group : 16 * RT;
                    const RowBox box = a.D == 64    ? RowBoxOf<64>::at(p.row_waves, heads)
                                       : a.D == 128 ? RowBoxOf<128>::at(p.row_waves, heads)
                                                    : RowBoxOf<256>::at(p.row_waves, heads);
                    EXPECT(box.floats * 4 <= 160 * 1024);  // a compute unit's LDS
                    met[d][RT][p.row_waves] = true;
                  } else {
                    EXPECT(p.owners == 1 << p.log2_parts && p.by_row == (p.rows <= p.owners));
                    (p.by_row ? by_row : by_share)[d][RT] = true;
                  }
                }
              }
            }
          }
        }
      }
    }
  }
  for (int d = 0; d < 3; d++) {
    for (int RT = 1; RT <= (d < 2 ? 2 : 1); RT++) {
      EXPECT(by_row[d][RT] && by_share[d][RT]);
      for (int waves = 1; waves <= 8; waves *= 2) {
        if (has_row_form(64 << d, RT, waves) != met[d][RT][waves])
          std::fprintf(stderr, "D %d, %d sets of heads, %d waves: built %d, planned %d\n", 64 << d, RT, waves,
                       has_row_form(64 << d, RT, waves), met[d][RT][waves]);
        EXPECT(has_row_form(64 << d, RT, waves) == met[d][RT][waves]);
      }
    }
  }
  std::printf("attention plans: %ld\n", checked);
}

// Arguments B Hq Hkv D e4m3 max_len window: prints the plan for 256 compute units.
static int one(char **v) {
  float scale = 0.f;
  DecodeArgs a{};
  a.B = std::atoi(v[0]);
  a.Hq = std::atoi(v[1]);
  a.Hkv = std::atoi(v[2]);
  a.D = std::atoi(v[3]);
  if (std::atoi(v[4])) a.k_scale = a.v_scale = &scale;
  a.max_len = std::atoi(v[5]);
  a.window = std::atoi(v[6]);
  const DecodePlan p = plan_decode(a, 256);
  std::printf("%d %d %d\n", p.row_waves, p.splits, (int)p.by_row);
  return 0;
}

int main(int argc, char **argv) {
  if (argc == 8) return one(argv + 1);
  plans();
  boxes<64>();
  boxes<128>();
  boxes<256>();
  if (!g_bad) std::printf("decode plan driver: ok\n");
  return g_bad;
}
