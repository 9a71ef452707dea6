// Driver for the address / undefined-behaviour sanitizer build of the prompt and chunk
// calls' host code (test infrastructure): argument validation with extreme values, the
// device check without a GPU, and the attention's launch plan over a sweep of batches: its parts
// cover every tile, its blocks every row, its partials stay small.  No kernel is launched.
#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdio>
#include <limits>

#include "../../include/fp8lin.h"
#include "../../sparse_gemm_linears_amd/csrc/prompt_plan.hpp"

static int g_bad = 0;
#define EXPECT(cond)                                                        \
  do {                                                                      \
    if (!(cond)) {                                                          \
      std::fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
      g_bad = 1;                                                            \
    }                                                                       \
  } while (0)

template <class T>
static T *fake(uintptr_t i) {
  return reinterpret_cast<T *>(i << 42);
}

static const int64_t kWild[] = {std::numeric_limits<int64_t>::min(), -8, 0, 1, 3, 16, 48, 64, 128, 256, 65536,
                                int64_t(1) << 24, int64_t(1) << 31, int64_t(1) << 36, int64_t(1) << 40,
                                std::numeric_limits<int64_t>::max()};

static bool known(fp8l_status s) {
  return s == FP8L_OK || s == FP8L_ERR_SHAPE || s == FP8L_ERR_DEVICE || s == FP8L_ERR_ALIAS;
}

// Pairs of arguments take every two wild values while the others are ordinary: a status
// comes back, with no overflow on the way.
template <int N, class Call>
static void pairs(const int64_t (&ordinary)[N], Call call) {
  for (int64_t x : kWild)
    for (int64_t y : kWild)
      for (int i = 0; i < N; i++)
        for (int j = 0; j < N; j++) {
          int64_t w[N];
          for (int k = 0; k < N; k++) w[k] = k == i ? x : k == j ? y : ordinary[k];
          EXPECT(known(call(w)));
        }
}

static void wild() {
  const int64_t append[8] = {4, 8, 2, 128, 128, 64, 8, 16};  // T, Hq, Hkv, D, rot, max_pos, pages, page
  pairs(append, [](const int64_t *w) {
    return kv_norm_rope_append_fp8(fake<uint16_t>(1), fake<uint16_t>(2), fake<uint16_t>(3), 1e-5f, fake<int32_t>(4),
                                   fake<int64_t>(5), fake<float>(6), w[0], w[1], w[2], w[3], w[4], 0, w[5], w[6], w[7],
                                   fake<uint16_t>(7), fake<uint16_t>(8), fake<uint8_t>(9), fake<uint8_t>(10),
                                   fake<float>(11), fake<float>(12), nullptr);
  });
  // B, T, Hq, Hkv, D, six strides, window
  const int64_t prompt[12] = {3, 64, 8, 2, 128, 1024, 128, 256, 128, 256, 128, 0};
  pairs(prompt, [](const int64_t *w) {
    return prompt_attention(fake<uint16_t>(1), fake<uint16_t>(2), fake<uint16_t>(3), fake<int32_t>(4), w[0], w[1], w[2],
                            w[3], w[4], w[5], w[6], w[7], w[8], w[9], w[10], 0.1f, 0.f, w[11], 1, fake<uint16_t>(5),
                            fake<float>(6), nullptr);
  });
  // B, T, Hq, Hkv, D, pages, page, max_pages, max_len, window
  const int64_t chunk[10] = {3, 64, 8, 2, 128, 8, 16, 4, 64, 0};
  pairs(chunk, [](const int64_t *w) {
    return paged_chunk_attention(fake<uint16_t>(1), fake<uint16_t>(2), fake<uint16_t>(3), fake<int32_t>(4),
                                 fake<int32_t>(5), fake<int32_t>(6), w[0], w[1], w[2], w[3], w[4], w[5], w[6], w[7],
                                 w[8], 0.1f, 0.f, w[9], fake<uint16_t>(7), fake<float>(8), nullptr);
  });
}

// The blocks of sequences of these lengths have numbers of their own, below the plan's count.
static void blocks_of(const fp8lin::PromptPlan &p, int64_t T, int64_t B, int group) {
  for (int kind = 0; kind < 3; kind++) {
    int64_t start = 0, last = -1;
    for (int64_t b = 0; b < B; b++) {
      const int64_t n = kind == 0 ? (b == 0 ? T : 0) : kind == 1 ? (b == B - 1 ? T : 0) : T * (b + 1) / B - T * b / B;
      const int64_t first = fp8lin::first_block(start, b, group), next = fp8lin::first_block(start + n, b + 1, group);
      const int64_t blocks = (n * group + fp8lin::kBlockRows - 1) / fp8lin::kBlockRows;
      EXPECT(first > last && first + blocks <= next && next <= p.blocks);
      last = first + blocks - 1 > last ? first + blocks - 1 : first;
      start += n;
    }
  }
}

static void plans() {
  size_t worst = 0;
  long checked = 0;
  static int32_t table;
  static float scale;
  for (int cus : {32, 64, 256, 304})
    for (int64_t B : {1, 2, 3, 17, 64, 255, 4096, 65535})
      for (int64_t T : {int64_t(1), int64_t(7), int64_t(64), int64_t(500), int64_t(4093), int64_t(100000), int64_t(1) << 24})
        for (int Hkv : {1, 2, 8, 40, 1024})
          for (int group : {1, 4, 16, 33, 128})
            for (int D : {64, 128, 256}) {
              if (Hkv * group > 1024 || T * Hkv * group * D > int64_t(1) << 36) continue;
              for (int64_t len : {int64_t(0), int64_t(1), int64_t(777), int64_t(32768), int64_t(1) << 30})
                for (int window : {0, 1, 1000, 1 << 30})
                  for (int kind = 0; kind < 3; kind++) {
                    fp8lin::PromptArgs a{};
                    a.B = (int)B;
                    a.T = (int)T;
                    a.Hq = Hkv * group;
                    a.Hkv = Hkv;
                    a.D = D;
                    a.window = window;
                    a.causal = true;
                    a.max_len = (int)(kind ? len : T);
                    a.block_table = kind ? &table : nullptr;
                    a.k_scale = kind == 2 ? &scale : nullptr;
                    if (!kind && len) continue;
                    const fp8lin::PromptPlan p = fp8lin::plan_prompt(a, cus);
                    // the keys that a block can see
                    int64_t keys = a.max_len;
                    const int64_t seen = (int64_t)window + (fp8lin::kBlockRows + group - 1) / group + 15;
                    if (window && seen < keys) keys = seen;
                    EXPECT(p.splits >= 1 && p.per >= 1 && p.blocks >= 1 && p.filled >= 1);
                    EXPECT((int64_t)p.splits * p.per * fp8lin::tile_keys(D) >= keys);
                    EXPECT(fp8lin::prompt_parts(p, a.Hkv) < (int64_t(1) << 31));
                    // with shares every block has one at least
                    EXPECT(p.shares == 0 || (p.shares >= p.blocks && p.splits == 1 && kind && B <= 256));
                    // the join is one launch
                    EXPECT(!fp8lin::prompt_joins(p) || fp8lin::prompt_parts(p, a.Hkv) * 256 < int64_t(1) << 22);
                    const size_t bytes = !fp8lin::prompt_joins(p) ? 0
                                                                  : (size_t)fp8lin::prompt_parts(p, a.Hkv) *
                                                                        fp8lin::prompt_part_floats(D) * sizeof(float);
                    worst = bytes > worst ? bytes : worst;
                    EXPECT(bytes < size_t(1) << 30);
                    checked++;
                  }
              fp8lin::PromptArgs a{};
              a.B = (int)B;
              a.T = (int)T;
              a.Hq = Hkv * group;
              a.Hkv = Hkv;
              a.D = D;
              a.max_len = (int)T;
              if (B <= 4096 && cus == 256) blocks_of(fp8lin::plan_prompt(a, cus), T, B, group);
            }
  std::printf("prompt plans: %ld, largest partials %zu bytes\n", checked, worst);
}

int main() {
  int n = 0;
  if (hipGetDeviceCount(&n) != hipSuccess || n == 0) {  // with a GPU the ordinary values would launch
    (void)hipGetLastError();
    wild();
  }
  plans();
  if (!g_bad) std::printf("prompt host sanitizer driver: ok\n");
  return g_bad;
}
