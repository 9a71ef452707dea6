// Launchers of the decoder-layer kernels (norm.hip, kv_append.hip,
// paged_decode.hip) behind the entry points in api_layer.hip.  Arguments are
// already validated; each returns the runtime's launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace fp8lin {

// Scales of an e4m3 output: fp32 amax / 448, or UE8M0 exponent bytes.
enum class ScaleKind { kFp32, kUe8m0 };

struct NormArgs {
  const uint16_t *x, *res, *w;  // res may be NULL
  float eps;
  int64_t M;
  int K;
  uint16_t *h, *y;  // each may be NULL
  uint8_t *q;       // may be NULL (then scales too)
  void *scales;     // float or uint8_t, by ScaleKind
};
hipError_t launch_add_rmsnorm(const NormArgs &a, ScaleKind kind, hipStream_t stream);

struct AppendArgs {
  const uint16_t *qkv;
  const int32_t *positions;
  const int64_t *slots;
  const float *cos_sin;
  int64_t T;
  int Hq, Hkv, D, rot;
  bool interleaved;
  int max_pos;
  uint32_t n_slots, page_size;
  uint16_t *q_out;
  void *k_cache, *v_cache;    // bf16, or e4m3 codes when the scales are given
  float *k_scale, *v_scale;   // both NULL for a bf16 cache
};
hipError_t launch_kv_rope_append(const AppendArgs &a, hipStream_t stream);

struct DecodeArgs {
  const uint16_t *q;
  const void *k_cache, *v_cache;
  const float *k_scale, *v_scale;  // both NULL for a bf16 cache
  const int32_t *block_table, *seq_lens;
  int B, Hq, Hkv, D;
  int pages, page_size, max_pages, max_len;
  float scale, softcap;  // softcap 0: none
  int window;            // 0: none
  uint16_t *o;
  float *lse;  // may be NULL
};
hipError_t launch_paged_decode(const DecodeArgs &a, float *part, hipStream_t stream);
// Bytes of fp32 partials that call needs on a device with `cus` compute units
// (0 where one workgroup covers a whole sequence).
size_t paged_decode_partial_bytes(const DecodeArgs &a, int cus);

}  // namespace fp8lin
