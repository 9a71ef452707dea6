// Driver for the address / undefined-behaviour sanitizer build of the
// decoder-layer calls' host code (test infrastructure): argument validation with
// extreme values, the device check without a GPU, and the attention's launch plan
// over a sweep of batches.  No kernel is launched.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <cstdio>
#include <limits>

#include "../../include/fp8lin.h"
#include "../../sparse_gemm_linears_amd/csrc/launch_layer.hpp"

static int g_bad = 0;
#define EXPECT(cond)                                                        \
  do {                                                                      \
    if (!(cond)) {                                                          \
      std::fprintf(stderr, "%s:%d: check failed: %s\n", __FILE__, __LINE__, #cond); \
      g_bad = 1;                                                            \
    }                                                                       \
  } while (0)

template <class T>
static T *fake(uintptr_t i, uintptr_t off = 0) {
  return reinterpret_cast<T *>((i << 42) + off);
}

static const int64_t kWild[] = {std::numeric_limits<int64_t>::min(), -1, 0, 1, 3, 16, 48, 64, 100, 128, 256,
                                65536, int64_t(1) << 24, int64_t(1) << 31, int64_t(1) << 40,
                                std::numeric_limits<int64_t>::max()};

static bool known(fp8l_status s) {
  return s == FP8L_OK || s == FP8L_ERR_SHAPE || s == FP8L_ERR_DEVICE || s == FP8L_ERR_ALIAS;
}

// Every argument takes every wild value while the others are ordinary, and pairs of
// them do: a status comes back, with no overflow on the way.
static void wild() {
  for (int64_t x : kWild) {
    for (int64_t y : kWild) {
      EXPECT(known(fp8_add_rmsnorm(fake<uint16_t>(1), fake<uint16_t>(2), fake<uint16_t>(3), 1e-5f, x, y,
                                   fake<uint16_t>(4), fake<uint16_t>(5), fake<uint8_t>(6), fake<float>(7), nullptr)));
      int64_t v[8] = {4, 8, 2, 128, 128, 64, 8, 16};  // T, Hq, Hkv, D, rot, max_pos, pages, page
      for (int i = 0; i < 8; i++) {
        for (int j = 0; j < 8; j++) {
          int64_t w[8];
          for (int k = 0; k < 8; k++) w[k] = k == i ? x : k == j ? y : v[k];
          EXPECT(known(kv_rope_append_fp8(fake<uint16_t>(1), fake<int32_t>(2), fake<int64_t>(3), fake<float>(4), w[0],
                                          w[1], w[2], w[3], w[4], 0, w[5], w[6], w[7], fake<uint16_t>(5),
                                          fake<uint8_t>(6), fake<uint8_t>(7), fake<float>(8), fake<float>(9),
                                          nullptr)));
        }
      }
      int64_t u[9] = {3, 8, 2, 128, 8, 16, 4, 64, 0};  // B, Hq, Hkv, D, pages, page, max_pages, max_len, window
      for (int i = 0; i < 9; i++) {
        for (int j = 0; j < 9; j++) {
          int64_t w[9];
          for (int k = 0; k < 9; k++) w[k] = k == i ? x : k == j ? y : u[k];
          EXPECT(known(paged_decode_attention(fake<uint16_t>(1), fake<uint16_t>(2), fake<uint16_t>(3),
                                              fake<int32_t>(4), fake<int32_t>(5), w[0], w[1], w[2], w[3], w[4], w[5],
                                              w[6], w[7], 0.1f, 0.f, w[8], fake<uint16_t>(6), fake<float>(7),
                                              nullptr)));
        }
      }
    }
  }
  EXPECT(fp8_add_rmsnorm(fake<uint16_t>(1), nullptr, fake<uint16_t>(3), std::nanf(""), 4, 128, nullptr,
                         fake<uint16_t>(5), nullptr, nullptr, nullptr) == FP8L_ERR_SHAPE);
}

static void plans() {
  size_t worst = 0;
  long checked = 0;
  for (int cus : {32, 64, 256, 304}) {
    for (int64_t B : {1, 2, 3, 17, 64, 255, 4096, 65535}) {
      for (int Hkv : {1, 2, 8, 40, 1024}) {
        for (int group : {1, 4, 16, 17, 32, 33, 128}) {
          if (Hkv * group > 1024) continue;
          for (int D : {64, 128, 256}) {
            for (int64_t len : {int64_t(0), int64_t(1), int64_t(512), int64_t(513), int64_t(1025), int64_t(100000),
                                int64_t(1) << 30}) {
              for (int window : {0, 1, 1000, std::numeric_limits<int>::max()}) {
                fp8lin::DecodeArgs a{};
                a.B = (int)B;
                a.Hq = Hkv * group;
                a.Hkv = Hkv;
                a.D = D;
                a.max_len = (int)len;
                a.window = window;
                const size_t bytes = fp8lin::paged_decode_partial_bytes(a, cus);
                worst = bytes > worst ? bytes : worst;
                checked++;
                if (len <= 1) EXPECT(bytes == 0);
                EXPECT(bytes < size_t(256) << 20);
              }
            }
          }
        }
      }
    }
  }
  std::printf("attention plans: %ld, largest partials %zu bytes\n", checked, worst);
}

int main() {
  int n = 0;
  if (hipGetDeviceCount(&n) != hipSuccess || n == 0) {  // with a GPU the ordinary values would launch
    (void)hipGetLastError();
    wild();
  }
  plans();
  if (!g_bad) std::printf("decoder-layer host sanitizer driver: ok\n");
  return g_bad;
}
