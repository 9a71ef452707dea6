// The bounds that the attention's launch plan states for its divisions (test infrastructure), over
// a sweep of batches: at most kMostPartialBytes of partials, and at most 8 workgroups a compute
// unit, or 1.25 times the blocks and a round of two a compute unit more where lengths divide
// them.  No kernel is launched.
#include <cstdint>
#include <cstdio>

#include "../../sparse_gemm_linears_amd/csrc/prompt_plan.hpp"

int main() {
  int bad = 0;
  long checked = 0, divided = 0;
  int64_t worst = 0;
  double most = 0;
  static int32_t table;
  static float scale;
  for (int cus : {32, 256, 304})
    for (int B = 1; B <= 300; B += B < 20 ? 1 : 3)
      for (int each : {1, 4, 8, 19, 64, 300})
        for (int Hkv : {1, 2, 3, 8, 32, 100, 1024})
          for (int group : {1, 4, 16, 64})
            for (int D : {64, 128, 256})
              for (int len : {300, 4096, 1 << 20})
                for (int kind = 0; kind < 3; kind++) {
                  if (Hkv * group > 1024 || each * B > (1 << 16)) continue;
                  fp8lin::PromptArgs a{};
                  a.B = B;
                  a.T = B * each;
                  a.Hq = Hkv * group;
                  a.Hkv = Hkv;
                  a.D = D;
                  a.causal = true;
                  a.max_len = kind ? len : a.T;
                  a.block_table = kind ? &table : nullptr;
                  a.k_scale = kind == 2 ? &scale : nullptr;
                  const fp8lin::PromptPlan p = fp8lin::plan_prompt(a, cus);
                  checked++;
                  if (!fp8lin::prompt_joins(p)) continue;
                  divided++;
                  const int64_t parts = fp8lin::prompt_parts(p, Hkv), found = (int64_t)p.blocks * Hkv;
                  const int64_t bytes = parts * fp8lin::prompt_part_floats(D) * 4;
                  const int64_t limit = p.shares > 0 ? found * 5 / 4 + 2 * cus : 8 * cus;
                  if (bytes > worst) worst = bytes;
                  if ((double)parts / cus > most) most = (double)parts / cus;
                  // (parts of shares come in whole rounds, times 5/4 where blocks are large)
                  const bool ok = bytes <= fp8lin::kMostPartialBytes &&
                                  parts <= (p.shares > 0 && p.filled > fp8lin::kWaveRows ? limit * 5 / 4 : limit) &&
                                  (p.shares == 0 || p.shares >= p.blocks);
                  if (!ok) {
                    if (!bad)
                      std::fprintf(stderr, "cus %d B %d T %d heads %d / %d of %d, %d keys: %lld workgroups, %lld bytes\n",
                                   cus, B, a.T, a.Hq, Hkv, D, a.max_len, (long long)parts, (long long)bytes);
                    bad++;
                  }
                }
  std::printf("prompt bounds: %ld plans, %ld divided, at most %.1f workgroups a compute unit and %lld bytes\n", checked,
              divided, most, (long long)worst);
  if (!bad) std::printf("prompt bounds: ok\n");
  return bad ? 1 : 0;
}
