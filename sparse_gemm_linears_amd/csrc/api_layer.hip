// C entry points of the decoder-layer operators: the residual norm with e4m3
// output, the rotary append to a paged cache and the attention over it, of one
// token or several, or of prompts over their own keys.  The checks run in the
// order of api.hip: shapes (an empty call returns here), NULL pointers,
// alignment, aliasing, device; then scratch memory; then the launches.
#include <cmath>

#include "api_common.hpp"
#include "launch_layer.hpp"

namespace {

using namespace fp8lin;  // the shared checks

constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxPage = 65536;
constexpr int64_t kMaxSlots = (int64_t(1) << 31) - 1;  // cache lines of one head: pages * page_size
constexpr int64_t kMaxTokens = int64_t(1) << 30;          // of one sequence: max_pages * page_size
constexpr int64_t kMaxBatch = 65535;
constexpr int64_t kMaxCacheElems = int64_t(1) << 40;

fp8l_status add_rmsnorm(const NormArgs &a, int64_t K, ScaleKind kind, hipStream_t stream) {
  if (bad_mk(a.M, K) || !(a.eps >= 0.0f) || std::isinf(a.eps)) return FP8L_ERR_SHAPE;
  if (a.M == 0) return FP8L_OK;
  if (!a.x || !a.w || (!a.res != !a.h) || (!a.q != !a.scales) || (!a.y && !a.q)) return FP8L_ERR_NULL;
  const void *ptrs[] = {a.x, a.res, a.w, a.h, a.y, a.q, a.scales};
  for (const void *p : ptrs)
    if (!aligned16(p)) return FP8L_ERR_ALIGN;
  const int64_t n = a.M * K, scale_bytes = n / 128 * (kind == ScaleKind::kFp32 ? 4 : 1);
  // h may be res itself (the residual stream updated in place), else it overlaps no input
  const bool in_place = a.h && a.h == a.res;
  const Range ins[] = {{a.x, n * 2}, {a.w, K * 2}, {a.res, a.res && !in_place ? n * 2 : 0}};
  const Range outs[] = {{a.h, a.h ? n * 2 : 0}, {a.y, a.y ? n * 2 : 0}, {a.q, a.q ? n : 0},
                        {a.scales, a.q ? scale_bytes : 0}};
  if (any_alias(outs, 4, ins, 3)) return FP8L_ERR_ALIAS;
  if (fp8l_status st = check_device()) return st;
  return launched(launch_add_rmsnorm(a, kind, stream));
}

bool bad_cache(int64_t Hq, int64_t Hkv, int64_t D, int64_t pages, int64_t page_size) {
  return Hq <= 0 || Hkv <= 0 || Hq > kMaxHeads || Hkv > kMaxHeads || (D != 64 && D != 128 && D != 256) ||
         pages <= 0 || pages > kMaxSlots || page_size <= 0 || page_size % 16 != 0 || page_size > kMaxPage ||
         pages * page_size > kMaxSlots || pages * page_size * Hkv * D > kMaxCacheElems;
}

fp8l_status rope_append(AppendArgs a, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t rot, int64_t max_pos,
                        int64_t pages, int64_t page_size, bool fp8, hipStream_t stream) {
  if (bad_cache(Hq, Hkv, D, pages, page_size) || T < 0 || T > kMaxDim || T * (Hq + 2 * Hkv) * D > kMaxElems ||
      rot < 0 || rot > D || rot % 16 != 0 || max_pos < (rot > 0) || max_pos > kMaxDim || !(a.eps >= 0.0f) ||
      std::isinf(a.eps))
    return FP8L_ERR_SHAPE;
  if (T == 0) return FP8L_OK;
  if (!a.qkv || !a.slots || !a.q_out || !a.k_cache || !a.v_cache || (rot > 0 && (!a.positions || !a.cos_sin)) ||
      (fp8 && (!a.k_scale || !a.v_scale)))
    return FP8L_ERR_NULL;
  const void *ptrs[] = {a.qkv,     a.cos_sin, a.q_out,   a.k_cache,  a.v_cache,
                        a.k_scale, a.v_scale, a.k_out,   a.q_weight, a.k_weight};
  for (const void *p : ptrs)
    if (!aligned16(p)) return FP8L_ERR_ALIGN;
  if (((uintptr_t)a.positions & 3u) || ((uintptr_t)a.slots & 7u)) return FP8L_ERR_ALIGN;
  const int64_t lines = pages * page_size * Hkv, cache_bytes = lines * D * (fp8 ? 1 : 2);
  const Range ins[] = {{a.qkv, T * (Hq + 2 * Hkv) * D * 2},
                       {a.positions, rot > 0 ? T * 4 : 0},
                       {a.slots, T * 8},
                       {a.cos_sin, max_pos * rot * 4},
                       {a.q_weight, a.q_weight ? D * 2 : 0},
                       {a.k_weight, a.k_weight ? D * 2 : 0}};
  const Range outs[] = {{a.q_out, T * Hq * D * 2},
                        {a.k_out, a.k_out ? T * Hkv * D * 2 : 0},
                        {a.k_cache, cache_bytes},
                        {a.v_cache, cache_bytes},
                        {a.k_scale, fp8 ? lines * 4 : 0},
                        {a.v_scale, fp8 ? lines * 4 : 0}};
  if (any_alias(outs, 6, ins, 6)) return FP8L_ERR_ALIAS;
  if (fp8l_status st = check_device()) return st;
  a.T = T;
  a.Hq = (int)Hq;
  a.Hkv = (int)Hkv;
  a.D = (int)D;
  a.rot = (int)rot;
  a.max_pos = (int)max_pos;
  a.n_slots = (uint32_t)(pages * page_size);
  a.page_size = (uint32_t)page_size;
  return launched(launch_kv_rope_append(a, stream));
}

fp8l_status decode(const DecodeArgs &in, int64_t B, int64_t Hq, int64_t Hkv, int64_t D, int64_t pages,
                   int64_t page_size, int64_t max_pages, int64_t max_len, int64_t window, bool fp8,
                   hipStream_t stream) {
  if (bad_cache(Hq, Hkv, D, pages, page_size) || Hq % Hkv != 0 || B < 0 || B > kMaxBatch || max_pages <= 0 ||
      max_pages > kMaxTokens || max_pages * page_size > kMaxTokens || max_len < 0 || max_len > max_pages * page_size ||
      window < 0 || !std::isfinite(in.scale) || !(in.softcap >= 0.0f) || std::isinf(in.softcap))
    return FP8L_ERR_SHAPE;
  if (B == 0) return FP8L_OK;
  if (!in.q || !in.k_cache || !in.v_cache || !in.block_table || !in.seq_lens || !in.o ||
      (fp8 && (!in.k_scale || !in.v_scale)))
    return FP8L_ERR_NULL;
  const void *ptrs[] = {in.q, in.k_cache, in.v_cache, in.k_scale, in.v_scale, in.o};
  for (const void *p : ptrs)
    if (!aligned16(p)) return FP8L_ERR_ALIGN;
  if (((uintptr_t)in.block_table & 3u) || ((uintptr_t)in.seq_lens & 3u) || ((uintptr_t)in.lse & 3u))
    return FP8L_ERR_ALIGN;
  const int64_t lines = pages * page_size * Hkv, cache_bytes = lines * D * (fp8 ? 1 : 2);
  const Range ins[] = {{in.q, B * Hq * D * 2},
                       {in.k_cache, cache_bytes},
                       {in.v_cache, cache_bytes},
                       {in.k_scale, fp8 ? lines * 4 : 0},
                       {in.v_scale, fp8 ? lines * 4 : 0},
                       {in.block_table, B * max_pages * 4},
                       {in.seq_lens, B * 4}};
  const Range outs[] = {{in.o, B * Hq * D * 2}, {in.lse, in.lse ? B * Hq * 4 : 0}};
  if (any_alias(outs, 2, ins, 7)) return FP8L_ERR_ALIAS;
  if (fp8l_status st = check_device()) return st;
  DecodeArgs a = in;
  a.B = (int)B;
  a.Hq = (int)Hq;
  a.Hkv = (int)Hkv;
  a.D = (int)D;
  a.pages = (int)pages;
  a.page_size = (int)page_size;
  a.max_pages = (int)max_pages;
  a.max_len = (int)max_len;
  a.window = (int)(window < kMaxSlots ? window : kMaxSlots);
  // a smaller cap has no reciprocal, and leaves scores that no exponential tells from 0 either
  if (a.softcap > 0.0f && a.softcap < 1e-30f) a.softcap = 1e-30f;
  CallScratch sc;
  if (hipError_t e = sc.acquire(paged_decode_partial_bytes(a, device_cu_count()), 0, stream)) return launched(e);
  const hipError_t e = launch_paged_decode(a, sc.partials(), stream);
  return finished(e, sc);
}

constexpr int64_t kMaxHeadStride = int64_t(1) << 36, kMaxTokenStride = int64_t(1) << 24;  // 16 tokens by 32-bit offsets
constexpr float kMaxScale = 0x1p100f;

bool bad_scores(float scale, float softcap, int64_t window) {
  return !(std::fabs(scale) <= kMaxScale) || !(softcap >= 0.0f) || std::isinf(softcap) || window < 0;
}

bool bad_strides(int64_t token, int64_t head) {
  return token < 0 || token > kMaxTokenStride || token % 8 != 0 || head < 0 || head > kMaxHeadStride || head % 8 != 0;
}

// The attention of several tokens: the arguments that both calls have, already checked.
fp8l_status prompt(PromptArgs a, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t window,
                   hipStream_t stream) {
  if (fp8l_status st = check_device()) return st;
  a.B = (int)B;
  a.T = (int)T;
  a.Hq = (int)Hq;
  a.Hkv = (int)Hkv;
  a.D = (int)D;
  a.window = (int)(window < kMaxTokens ? window : kMaxTokens);
  // scores of a scale of 0 are 0 under any cap; without one 0 times the -infinity of a hidden key would be a NaN
  if (a.scale == 0.0f) a.softcap = 1.0f;
  if (a.softcap > 0.0f) {
    // The kernel multiplies q.k by scale / softcap, which has to be a normal number.  A smaller cap than
    // 2^-127 |scale| (2^-27 at most) leaves scores that no exponential tells from 0 either, nor does one below
    // 1e-30; a larger one than 2^126 |scale| is as good as none while |q.k| < 2^113.
    const float size = std::fabs(a.scale);
    if (a.softcap > 1e38f) a.softcap = 1e38f;  // log2(e) times it is finite
    if (a.softcap * 0x1p-126f > size) a.softcap = size * 0x1p126f;
    const float least = size * 0x1p-127f > 1e-30f ? size * 0x1p-127f : 1e-30f;
    if (a.softcap < least) a.softcap = least;
  }
  CallScratch sc;
  if (hipError_t e = sc.acquire(prompt_partial_bytes(a, device_cu_count()), 0, stream)) return launched(e);
  const hipError_t e = launch_prompt_attention(a, sc.partials(), stream);
  return finished(e, sc);
}

bool bad_tokens(int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D) {
  return Hq % Hkv != 0 || B < 0 || B > kMaxBatch || T < 0 || T > kMaxDim || T * Hq * D > kMaxElems;
}

fp8l_status chunk(PromptArgs a, int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t pages,
                  int64_t page_size, int64_t max_pages, int64_t max_len, int64_t window, bool fp8,
                  hipStream_t stream) {
  if (bad_cache(Hq, Hkv, D, pages, page_size) || bad_tokens(B, T, Hq, Hkv, D) || max_pages <= 0 ||
      max_pages > kMaxTokens || max_pages * page_size > kMaxTokens || max_len < 0 || max_len > max_pages * page_size ||
      bad_scores(a.scale, a.softcap, window))
    return FP8L_ERR_SHAPE;
  if (B == 0 || T == 0) return FP8L_OK;
  if (!a.q || !a.k || !a.v || !a.block_table || !a.seq_lens || !a.starts || !a.o ||
      (fp8 && (!a.k_scale || !a.v_scale)))
    return FP8L_ERR_NULL;
  const void *ptrs[] = {a.q, a.k, a.v, a.k_scale, a.v_scale, a.o};
  for (const void *p : ptrs)
    if (!aligned16(p)) return FP8L_ERR_ALIGN;
  if (((uintptr_t)a.block_table & 3u) || ((uintptr_t)a.seq_lens & 3u) || ((uintptr_t)a.starts & 3u) ||
      ((uintptr_t)a.lse & 3u))
    return FP8L_ERR_ALIGN;
  const int64_t lines = pages * page_size * Hkv, cache_bytes = lines * D * (fp8 ? 1 : 2);
  const Range ins[] = {{a.q, T * Hq * D * 2},
                       {a.k, cache_bytes},
                       {a.v, cache_bytes},
                       {a.k_scale, fp8 ? lines * 4 : 0},
                       {a.v_scale, fp8 ? lines * 4 : 0},
                       {a.block_table, B * max_pages * 4},
                       {a.seq_lens, B * 4},
                       {a.starts, (B + 1) * 4}};
  const Range outs[] = {{a.o, T * Hq * D * 2}, {a.lse, a.lse ? T * Hq * 4 : 0}};
  if (any_alias(outs, 2, ins, 8)) return FP8L_ERR_ALIAS;
  a.q_token = Hq * D;
  a.q_head = D;
  a.pages = (int)pages;
  a.page_size = (int)page_size;
  a.max_pages = (int)max_pages;
  a.max_len = (int)max_len;
  a.causal = true;
  return prompt(a, B, T, Hq, Hkv, D, window, stream);
}

}  // namespace

extern "C" {

fp8l_status fp8_add_rmsnorm(const uint16_t *x, const uint16_t *res, const uint16_t *w, float eps, int64_t M,
                            int64_t K, uint16_t *h, uint16_t *y, uint8_t *q, float *s, hipStream_t stream) {
  return add_rmsnorm(NormArgs{x, res, w, eps, M, (int)K, h, y, q, s}, K, ScaleKind::kFp32, stream);
}

fp8l_status fp8_add_rmsnorm_ue8m0(const uint16_t *x, const uint16_t *res, const uint16_t *w, float eps, int64_t M,
                                  int64_t K, uint16_t *h, uint16_t *y, uint8_t *q, uint8_t *e, hipStream_t stream) {
  return add_rmsnorm(NormArgs{x, res, w, eps, M, (int)K, h, y, q, e}, K, ScaleKind::kUe8m0, stream);
}

fp8l_status kv_rope_append(const uint16_t *qkv, const int32_t *positions, const int64_t *slots, const float *cos_sin,
                           int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t rot, int interleaved,
                           int64_t max_pos, int64_t pages, int64_t page_size, uint16_t *q_out, uint16_t *k_cache,
                           uint16_t *v_cache, hipStream_t stream) {
  AppendArgs a{};
  a.qkv = qkv;
  a.positions = positions;
  a.slots = slots;
  a.cos_sin = cos_sin;
  a.interleaved = interleaved != 0;
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  return rope_append(a, T, Hq, Hkv, D, rot, max_pos, pages, page_size, false, stream);
}

fp8l_status kv_rope_append_fp8(const uint16_t *qkv, const int32_t *positions, const int64_t *slots,
                               const float *cos_sin, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t rot,
                               int interleaved, int64_t max_pos, int64_t pages, int64_t page_size, uint16_t *q_out,
                               uint8_t *k_cache, uint8_t *v_cache, float *k_scale, float *v_scale,
                               hipStream_t stream) {
  AppendArgs a{};
  a.qkv = qkv;
  a.positions = positions;
  a.slots = slots;
  a.cos_sin = cos_sin;
  a.interleaved = interleaved != 0;
  a.q_out = q_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return rope_append(a, T, Hq, Hkv, D, rot, max_pos, pages, page_size, true, stream);
}

fp8l_status kv_norm_rope_append(const uint16_t *qkv, const uint16_t *q_weight, const uint16_t *k_weight, float eps,
                                const int32_t *positions, const int64_t *slots, const float *cos_sin, int64_t T,
                                int64_t Hq, int64_t Hkv, int64_t D, int64_t rot, int interleaved, int64_t max_pos,
                                int64_t pages, int64_t page_size, uint16_t *q_out, uint16_t *k_out, uint16_t *k_cache,
                                uint16_t *v_cache, hipStream_t stream) {
  AppendArgs a{};
  a.qkv = qkv;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.positions = positions;
  a.slots = slots;
  a.cos_sin = cos_sin;
  a.interleaved = interleaved != 0;
  a.q_out = q_out;
  a.k_out = k_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  return rope_append(a, T, Hq, Hkv, D, rot, max_pos, pages, page_size, false, stream);
}

fp8l_status kv_norm_rope_append_fp8(const uint16_t *qkv, const uint16_t *q_weight, const uint16_t *k_weight, float eps,
                                    const int32_t *positions, const int64_t *slots, const float *cos_sin, int64_t T,
                                    int64_t Hq, int64_t Hkv, int64_t D, int64_t rot, int interleaved, int64_t max_pos,
                                    int64_t pages, int64_t page_size, uint16_t *q_out, uint16_t *k_out,
                                    uint8_t *k_cache, uint8_t *v_cache, float *k_scale, float *v_scale,
                                    hipStream_t stream) {
  AppendArgs a{};
  a.qkv = qkv;
  a.q_weight = q_weight;
  a.k_weight = k_weight;
  a.eps = eps;
  a.positions = positions;
  a.slots = slots;
  a.cos_sin = cos_sin;
  a.interleaved = interleaved != 0;
  a.q_out = q_out;
  a.k_out = k_out;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  return rope_append(a, T, Hq, Hkv, D, rot, max_pos, pages, page_size, true, stream);
}

fp8l_status paged_decode_attention(const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache,
                                   const int32_t *block_table, const int32_t *seq_lens, int64_t B, int64_t Hq,
                                   int64_t Hkv, int64_t D, int64_t pages, int64_t page_size, int64_t max_pages,
                                   int64_t max_len, float scale, float softcap, int64_t window, uint16_t *o,
                                   float *lse, hipStream_t stream) {
  DecodeArgs a{};
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.scale = scale;
  a.softcap = softcap;
  a.o = o;
  a.lse = lse;
  return decode(a, B, Hq, Hkv, D, pages, page_size, max_pages, max_len, window, false, stream);
}

fp8l_status paged_decode_attention_fp8(const uint16_t *q, const uint8_t *k_cache, const uint8_t *v_cache,
                                       const float *k_scale, const float *v_scale, const int32_t *block_table,
                                       const int32_t *seq_lens, int64_t B, int64_t Hq, int64_t Hkv, int64_t D,
                                       int64_t pages, int64_t page_size, int64_t max_pages, int64_t max_len,
                                       float scale, float softcap, int64_t window, uint16_t *o, float *lse,
                                       hipStream_t stream) {
  DecodeArgs a{};
  a.q = q;
  a.k_cache = k_cache;
  a.v_cache = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.scale = scale;
  a.softcap = softcap;
  a.o = o;
  a.lse = lse;
  return decode(a, B, Hq, Hkv, D, pages, page_size, max_pages, max_len, window, true, stream);
}

fp8l_status prompt_attention(const uint16_t *q, const uint16_t *k, const uint16_t *v, const int32_t *starts, int64_t B,
                             int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t q_token, int64_t q_head,
                             int64_t k_token, int64_t k_head, int64_t v_token, int64_t v_head, float scale,
                             float softcap, int64_t window, int causal, uint16_t *o, float *lse, hipStream_t stream) {
  if (bad_cache(Hq, Hkv, D, 1, 16) || bad_tokens(B, T, Hq, Hkv, D) || bad_scores(scale, softcap, window) ||
      (window > 0 && !causal) || bad_strides(q_token, q_head) || bad_strides(k_token, k_head) ||
      bad_strides(v_token, v_head))
    return FP8L_ERR_SHAPE;
  if (B == 0 || T == 0) return FP8L_OK;
  if (!q || !k || !v || !starts || !o) return FP8L_ERR_NULL;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(o) || ((uintptr_t)starts & 3u) ||
      ((uintptr_t)lse & 3u))
    return FP8L_ERR_ALIGN;
  const Range ins[] = {{q, ((T - 1) * q_token + (Hq - 1) * q_head + D) * 2},
                       {k, ((T - 1) * k_token + (Hkv - 1) * k_head + D) * 2},
                       {v, ((T - 1) * v_token + (Hkv - 1) * v_head + D) * 2},
                       {starts, (B + 1) * 4}};
  const Range outs[] = {{o, T * Hq * D * 2}, {lse, lse ? T * Hq * 4 : 0}};
  if (any_alias(outs, 2, ins, 4)) return FP8L_ERR_ALIAS;
  PromptArgs a{};
  a.q = q;
  a.q_token = q_token;
  a.q_head = q_head;
  a.k = k;
  a.v = v;
  a.k_token = k_token;
  a.k_head = k_head;
  a.v_token = v_token;
  a.v_head = v_head;
  a.starts = starts;
  a.max_len = (int)T;
  a.scale = scale;
  a.softcap = softcap;
  a.causal = causal != 0;
  a.o = o;
  a.lse = lse;
  return prompt(a, B, T, Hq, Hkv, D, window, stream);
}

fp8l_status paged_chunk_attention(const uint16_t *q, const uint16_t *k_cache, const uint16_t *v_cache,
                                  const int32_t *block_table, const int32_t *seq_lens, const int32_t *starts,
                                  int64_t B, int64_t T, int64_t Hq, int64_t Hkv, int64_t D, int64_t pages,
                                  int64_t page_size, int64_t max_pages, int64_t max_len, float scale, float softcap,
                                  int64_t window, uint16_t *o, float *lse, hipStream_t stream) {
  PromptArgs a{};
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.starts = starts;
  a.scale = scale;
  a.softcap = softcap;
  a.o = o;
  a.lse = lse;
  return chunk(a, B, T, Hq, Hkv, D, pages, page_size, max_pages, max_len, window, false, stream);
}

fp8l_status paged_chunk_attention_fp8(const uint16_t *q, const uint8_t *k_cache, const uint8_t *v_cache,
                                      const float *k_scale, const float *v_scale, const int32_t *block_table,
                                      const int32_t *seq_lens, const int32_t *starts, int64_t B, int64_t T, int64_t Hq,
                                      int64_t Hkv, int64_t D, int64_t pages, int64_t page_size, int64_t max_pages,
                                      int64_t max_len, float scale, float softcap, int64_t window, uint16_t *o,
                                      float *lse, hipStream_t stream) {
  PromptArgs a{};
  a.q = q;
  a.k = k_cache;
  a.v = v_cache;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.block_table = block_table;
  a.seq_lens = seq_lens;
  a.starts = starts;
  a.scale = scale;
  a.softcap = softcap;
  a.o = o;
  a.lse = lse;
  return chunk(a, B, T, Hq, Hkv, D, pages, page_size, max_pages, max_len, window, true, stream);
}

}  // extern "C"
