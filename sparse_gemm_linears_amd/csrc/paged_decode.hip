// Attention of one new token of each sequence over a paged key-value cache.
//
// For query head n of sequence b, over the live tokens t (the last `window` of
// the sequence, or all): score_t = scale q.k_t, capped as c tanh(score / c) when
// a cap is given, o = sum_t softmax(score)_t v_t and lse = log sum_t exp(score_t).
// One pass over keys and values with a running maximum and sum.
#include "device_common.hpp"
#include "launch_layer.hpp"

namespace fp8lin {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

__device__ __forceinline__ float e4m3_value(uint32_t code) {
  return __builtin_amdgcn_cvt_f32_fp8((int)code, 0);
}

// One workgroup for each query head; a wave takes every fourth token, its
// lanes across the head's D values.
template <int D, bool FP8>
__global__ __launch_bounds__(256) void decode_head_kernel(DecodeArgs a) {
  constexpr int E = D / 64;
  __shared__ float wave_m[4], wave_l[4], wave_o[4][D];
  const int n = blockIdx.x, b = blockIdx.y, kvh = n / (a.Hq / a.Hkv);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int len = min(max(a.seq_lens[b], 0), a.max_len);
  const int first = a.window > 0 ? max(0, len - a.window) : 0;
  float q[E], o[E] = {}, m = -INFINITY, l = 0.f;
  for (int e = 0; e < E; e++) q[e] = bf16_to_f32(a.q[((int64_t)b * a.Hq + n) * D + e * 64 + lane]);
  for (int t = first + wave; t < len; t += 4) {
    int page = a.block_table[(int64_t)b * a.max_pages + t / a.page_size];
    page = min(max(page, 0), a.pages - 1);
    const int64_t line = ((int64_t)page * a.Hkv + kvh) * a.page_size + t % a.page_size;
    float s = 0.f, v[E];
    for (int e = 0; e < E; e++) {
      const int64_t at = line * D + e * 64 + lane;
      if (FP8) {
        s += q[e] * e4m3_value(static_cast<const uint8_t *>(a.k_cache)[at]);
        v[e] = e4m3_value(static_cast<const uint8_t *>(a.v_cache)[at]) * a.v_scale[line];
      } else {
        s += q[e] * bf16_to_f32(static_cast<const uint16_t *>(a.k_cache)[at]);
        v[e] = bf16_to_f32(static_cast<const uint16_t *>(a.v_cache)[at]);
      }
    }
    for (int off = 32; off; off >>= 1) s += __shfl_xor(s, off, 64);
    s *= a.scale;
    if (FP8) s *= a.k_scale[line];
    if (a.softcap > 0.f) s = a.softcap * tanhf(s / a.softcap);
    const float top = fmaxf(m, s), shrink = m == top ? 1.f : exp2f((m - top) * kLog2e);
    const float p = s == -INFINITY ? 0.f : exp2f((s - top) * kLog2e);
    l = l * shrink + p;
    for (int e = 0; e < E; e++) o[e] = o[e] * shrink + p * v[e];
    m = top;
  }
  if (lane == 0) wave_m[wave] = m, wave_l[wave] = l;
  for (int e = 0; e < E; e++) wave_o[wave][e * 64 + lane] = o[e];
  __syncthreads();
  float top = -INFINITY, total = 0.f;
  for (int w = 0; w < 4; w++) top = fmaxf(top, wave_m[w]);
  float f[4];
  for (int w = 0; w < 4; w++) {
    f[w] = wave_l[w] == 0.f ? 0.f : exp2f((wave_m[w] - top) * kLog2e);
    total += f[w] * wave_l[w];
  }
  for (int d = threadIdx.x; d < D; d += 256) {
    float sum = 0.f;
    for (int w = 0; w < 4; w++) sum += f[w] * wave_o[w][d];
    a.o[((int64_t)b * a.Hq + n) * D + d] = (uint16_t)f32_to_bf16_rne(total == 0.f ? 0.f : sum / total);
  }
  if (a.lse && threadIdx.x == 0)
    a.lse[(int64_t)b * a.Hq + n] = total == 0.f ? -INFINITY : top + kLn2 * log2f(total);
}

template <int D>
void launch_heads(const DecodeArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)a.Hq, (unsigned)a.B), block(256);
  if (a.k_scale)
    hipLaunchKernelGGL((decode_head_kernel<D, true>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((decode_head_kernel<D, false>), grid, block, 0, stream, a);
}

}  // namespace

size_t paged_decode_partial_bytes(const DecodeArgs &, int) { return 0; }

hipError_t launch_paged_decode(const DecodeArgs &a, float *, hipStream_t stream) {
  if (a.D == 64)
    launch_heads<64>(a, stream);
  else if (a.D == 128)
    launch_heads<128>(a, stream);
  else
    launch_heads<256>(a, stream);
  return hipGetLastError();
}

}  // namespace fp8lin
