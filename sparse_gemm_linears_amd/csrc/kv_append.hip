// Rotary position embedding of the query and key heads of a QKV projection and
// the append of the keys and values to a paged cache.
//
// A rotated pair (a, b) becomes (a cos - b sin, b cos + a sin), in fp32, rounded
// once: to bf16, or for an e4m3 cache to codes with one fp32 scale
// amax / 448 for each token and head.  HBM-bound for many tokens (each value
// is read once and written once), two memory latencies and the launch for one.
#include "device_common.hpp"
#include "launch_layer.hpp"

namespace fp8lin {
namespace {

// Largest over aligned sets of L lanes (4, 8 or 16), in every lane of the set.
template <int L>
__device__ __forceinline__ uint32_t lanes_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));  // quad_perm 1,0,3,2
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false));  // quad_perm 2,3,0,1
  if (L >= 8) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x141, 0xF, 0xF, false));  // half mirror
  if (L >= 16) v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x140, 0xF, 0xF, false));  // mirror
  return v;
}

// D / 16 lanes hold one head: two chunks of eight values each, which are the
// two halves of eight pairs where the lane rotates.  A workgroup covers one
// token, 256 * 16 / D heads at a time.
template <int D>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a) {
  constexpr int L = D / 16;
  const int64_t token = blockIdx.x;
  const int u = threadIdx.x % L;
  const int heads = a.Hq + 2 * a.Hkv;
  const int turning = a.rot / 16;  // lanes of a head that rotate
  int c0, c1;                      // columns of the two chunks
  if (a.interleaved || u >= turning) {
    c0 = 16 * u;
    c1 = 16 * u + 8;
  } else {
    c0 = 8 * u;
    c1 = 8 * u + a.rot / 2;
  }
  float cs[8], sn[8];
  if (u < turning) {
    const int p = min(max(a.positions[token], 0), a.max_pos - 1);
    const float4 *row = reinterpret_cast<const float4 *>(a.cos_sin + (int64_t)p * a.rot + 8 * u);
    const float4 *row2 = reinterpret_cast<const float4 *>(a.cos_sin + (int64_t)p * a.rot + a.rot / 2 + 8 * u);
    const float4 k0 = row[0], k1 = row[1], s0 = row2[0], s1 = row2[1];
    cs[0] = k0.x; cs[1] = k0.y; cs[2] = k0.z; cs[3] = k0.w; cs[4] = k1.x; cs[5] = k1.y; cs[6] = k1.z; cs[7] = k1.w;
    sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w; sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
  }
  const int64_t slot = a.slots[token];
  const bool stored = slot >= 0 && slot < (int64_t)a.n_slots;
  const uint32_t page = stored ? (uint32_t)slot / a.page_size : 0, off = stored ? (uint32_t)slot % a.page_size : 0;
  for (int h = threadIdx.x / L; h < heads; h += 256 / L) {
    const uint16_t *src = a.qkv + (token * heads + h) * D;
    float f0[8], f1[8];
    unpack8(*reinterpret_cast<const uint4 *>(src + c0), f0);
    unpack8(*reinterpret_cast<const uint4 *>(src + c1), f1);
    if (h < a.Hq + a.Hkv && u < turning) {
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const float x0 = f0[2 * j], y0 = f0[2 * j + 1], x1 = f1[2 * j], y1 = f1[2 * j + 1];
          f0[2 * j] = x0 * cs[j] - y0 * sn[j];
          f0[2 * j + 1] = y0 * cs[j] + x0 * sn[j];
          f1[2 * j] = x1 * cs[4 + j] - y1 * sn[4 + j];
          f1[2 * j + 1] = y1 * cs[4 + j] + x1 * sn[4 + j];
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const float x = f0[j], y = f1[j];
          f0[j] = x * cs[j] - y * sn[j];
          f1[j] = y * cs[j] + x * sn[j];
        }
      }
    }
    if (h < a.Hq) {
      uint16_t *dst = a.q_out + (token * a.Hq + h) * D;
      *reinterpret_cast<uint4 *>(dst + c0) = pack8(f0);
      *reinterpret_cast<uint4 *>(dst + c1) = pack8(f1);
      continue;
    }
    const bool value = h >= a.Hq + a.Hkv;
    const int kvh = h - a.Hq - (value ? a.Hkv : 0);
    const int64_t line = ((int64_t)page * a.Hkv + kvh) * a.page_size + off;
    if (a.k_scale) {
      uint32_t m = 0;
#pragma unroll
      for (int j = 0; j < 8; j++)
        m = max(m, max(__float_as_uint(f0[j]) & 0x7FFFFFFFu, __float_as_uint(f1[j]) & 0x7FFFFFFFu));
      m = lanes_max<L>(m);
      float s;
      const uint2 q0 = quantize8_f32(f0, m, s), q1 = quantize8_f32(f1, m, s);
      if (stored) {
        uint8_t *dst = static_cast<uint8_t *>(value ? a.v_cache : a.k_cache) + line * D;
        *reinterpret_cast<uint2 *>(dst + c0) = q0;
        *reinterpret_cast<uint2 *>(dst + c1) = q1;
        if (u == 0) (value ? a.v_scale : a.k_scale)[line] = s;
      }
    } else if (stored) {
      uint16_t *dst = static_cast<uint16_t *>(value ? a.v_cache : a.k_cache) + line * D;
      *reinterpret_cast<uint4 *>(dst + c0) = pack8(f0);
      *reinterpret_cast<uint4 *>(dst + c1) = pack8(f1);
    }
  }
}

}  // namespace

hipError_t launch_kv_rope_append(const AppendArgs &a, hipStream_t stream) {
  const dim3 grid((unsigned)a.T), block(256);
  if (a.D == 64)
    hipLaunchKernelGGL(append_kernel<64>, grid, block, 0, stream, a);
  else if (a.D == 128)
    hipLaunchKernelGGL(append_kernel<128>, grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL(append_kernel<256>, grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace fp8lin
