// Rotary position embedding of the query and key heads of a QKV projection and
// the append of the keys and values to a paged cache; before the rotation, on
// request, the root-mean-square norm of each query and key head.
//
// A rotated pair (a, b) becomes (a cos - b sin, b cos + a sin), in fp32, rounded
// once: to bf16, or for an e4m3 cache to codes with one fp32 scale
// amax / 448 for each token and head.  HBM-bound for many tokens (each value
// is read once and written once): 8192 tokens of 48 heads of 128 into an e4m3
// cache, 189 MB in 33.8 us, 5.6 TB/s.  One token is bound by two memory
// latencies and the launch: 3.0 us.  (Times in this file: one call of a replayed graph of
// twelve over three sets of inputs in turn.  Issued one by one, calls take 37.5 and
// 5.3 us.)  With the norms and the keys kept in bf16 the 8192 tokens move 206 MB in 43.3 us, issued one by
// one (4.8 TB/s; 37.5 without), one token takes 5.4 to 5.7 us: the norm adds 16 products and a sum over
// a head's lanes to each head, which the loads in flight cover.
#include <type_traits>

#include "device_common.hpp"
#include "launch.hpp"
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

// The pair (x, y) turned.  Which product is fused is written out, so that every form of
// the kernel gives the same bits.
template <bool NEIGHBOURS>
__device__ __forceinline__ void turn(float x, float y, float c, float s, float &a, float &b) {
  a = __builtin_fmaf(x, c, -(y * s));
  b = NEIGHBOURS ? __builtin_fmaf(y, c, x * s) : __builtin_fmaf(x, s, y * c);
}

// Sum over aligned sets of L lanes (4, 8 or 16), in every lane of the set.
template <int L>
__device__ __forceinline__ float lanes_sum(float v) {
  auto from = [&](auto ctrl) {
    return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), decltype(ctrl)::value, 0xF, 0xF, false));
  };
  v += from(std::integral_constant<int, 0xB1>());
  v += from(std::integral_constant<int, 0x4E>());
  if constexpr (L >= 8) v += from(std::integral_constant<int, 0x141>());
  if constexpr (L >= 16) v += from(std::integral_constant<int, 0x140>());
  return v;
}

// x / sqrt(mean x^2 + eps) * w of a head of D values, 16 in each of D / 16 lanes, in fp32
// (an infinite mean leaves 0 of finite values, like the residual norm).
template <int D>
__device__ __forceinline__ void norm_head(float (&f0)[8], float (&f1)[8], const uint4 &w0, const uint4 &w1, float eps) {
  float sum = 0.f;
#pragma unroll
  for (int j = 0; j < 8; j++) sum = __builtin_fmaf(f0[j], f0[j], __builtin_fmaf(f1[j], f1[j], sum));
  const float r = 1.0f / sqrtf(lanes_sum<D / 16>(sum) * (1.0f / D) + eps);
  float g0[8], g1[8];
  unpack8(w0, g0);
  unpack8(w1, g1);
#pragma unroll
  for (int j = 0; j < 8; j++) {
    f0[j] = f0[j] * r * g0[j];
    f1[j] = f1[j] * r * g1[j];
  }
}

// D / 16 lanes hold one head: two chunks of eight values each, which are the
// two halves of eight pairs where the lane rotates.  A workgroup covers 2^tokens_log2
// tokens; a set of lanes keeps one token, with its angles in registers, and takes
// its heads in strides of 256 16 / D >> tokens_log2.  MORE: heads may be normed, and
// the turned keys are stored in bf16 too where the caller wants them.
template <int D, bool FP8, bool MORE>
__global__ __launch_bounds__(256) void append_kernel(AppendArgs a, int tokens_log2) {
  constexpr int L = D / 16;
  const int u = threadIdx.x % L, set = threadIdx.x / L;
  const int64_t token = ((int64_t)blockIdx.x << tokens_log2) + (set & ((1 << tokens_log2) - 1));
  const int stride = 256 / L >> tokens_log2;
  if (token >= a.T) return;  // whole sets of lanes
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
  const uint16_t *row = a.qkv + token * heads * D;
  const int64_t slot = a.slots[token];
  float cs[8], sn[8];
  if (u < turning) {
    const int p = min(max(a.positions[token], 0), a.max_pos - 1);
    const float4 *cosines = reinterpret_cast<const float4 *>(a.cos_sin + (int64_t)p * a.rot + 8 * u);
    const float4 *sines = reinterpret_cast<const float4 *>(a.cos_sin + (int64_t)p * a.rot + a.rot / 2 + 8 * u);
    const float4 k0 = cosines[0], k1 = cosines[1], s0 = sines[0], s1 = sines[1];
    cs[0] = k0.x; cs[1] = k0.y; cs[2] = k0.z; cs[3] = k0.w; cs[4] = k1.x; cs[5] = k1.y; cs[6] = k1.z; cs[7] = k1.w;
    sn[0] = s0.x; sn[1] = s0.y; sn[2] = s0.z; sn[3] = s0.w; sn[4] = s1.x; sn[5] = s1.y; sn[6] = s1.z; sn[7] = s1.w;
  }
  uint4 qw[2], kw[2];  // weights of the lane's columns
  if constexpr (MORE) {
#pragma unroll
    for (int i = 0; i < 2; i++) {
      const int at = i ? c1 : c0;
      qw[i] = a.q_weight ? *reinterpret_cast<const uint4 *>(a.q_weight + at) : make_uint4(0, 0, 0, 0);
      kw[i] = a.k_weight ? *reinterpret_cast<const uint4 *>(a.k_weight + at) : make_uint4(0, 0, 0, 0);
    }
  }
  const bool stored = slot >= 0 && slot < (int64_t)a.n_slots;
  const uint32_t page = stored ? (uint32_t)slot / a.page_size : 0, off = stored ? (uint32_t)slot % a.page_size : 0;
  // turns, rounds and stores head h
  auto use = [&](const uint4(&r)[2], int h) {
    float f0[8], f1[8];
    unpack8(r[0], f0);
    unpack8(r[1], f1);
    if constexpr (MORE) {
      if (h < a.Hq) {
        if (a.q_weight) norm_head<D>(f0, f1, qw[0], qw[1], a.eps);
      } else if (h < a.Hq + a.Hkv) {
        if (a.k_weight) norm_head<D>(f0, f1, kw[0], kw[1], a.eps);
      }
    }
    if (h < a.Hq + a.Hkv && u < turning) {
      if (a.interleaved) {
#pragma unroll
        for (int j = 0; j < 4; j++) {
          const float x0 = f0[2 * j], y0 = f0[2 * j + 1], x1 = f1[2 * j], y1 = f1[2 * j + 1];
          turn<true>(x0, y0, cs[j], sn[j], f0[2 * j], f0[2 * j + 1]);
          turn<true>(x1, y1, cs[4 + j], sn[4 + j], f1[2 * j], f1[2 * j + 1]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const float x = f0[j], y = f1[j];
          turn<false>(x, y, cs[j], sn[j], f0[j], f1[j]);
        }
      }
    }
    if (h < a.Hq) {
      uint16_t *dst = a.q_out + (token * a.Hq + h) * D;
      *reinterpret_cast<uint4 *>(dst + c0) = pack8(f0);
      *reinterpret_cast<uint4 *>(dst + c1) = pack8(f1);
      return;
    }
    const bool value = h >= a.Hq + a.Hkv;
    const int kvh = h - a.Hq - (value ? a.Hkv : 0);
    if constexpr (MORE) {
      if (a.k_out && !value) {
        uint16_t *dst = a.k_out + (token * a.Hkv + kvh) * D;
        *reinterpret_cast<uint4 *>(dst + c0) = pack8(f0);
        *reinterpret_cast<uint4 *>(dst + c1) = pack8(f1);
      }
    }
    const int64_t line = ((int64_t)page * a.Hkv + kvh) * a.page_size + off;
    if constexpr (FP8) {
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
  };
  for (int h = set >> tokens_log2; h < heads; h += stride) {
    const uint16_t *src = row + h * D;
    const uint4 r[2] = {*reinterpret_cast<const uint4 *>(src + c0), *reinterpret_cast<const uint4 *>(src + c1)};
    use(r, h);
  }
}

// Tokens of a workgroup (log2): more of them leave fewer of its lanes idle, but make
// the workgroups fewer and their loops longer, so a number is taken if it needs a
// fifth fewer lane steps than the last one taken, loops of five at most, and leaves
// two workgroups for each compute unit.  With 1, 2, 4, 8, 16 tokens (* the choice): 12603
// tokens of 34 heads of 64 (e4m3 cache) 23.3 20.9 19.8* 20.0 23.4 us, 9000 of 56 (bf16)
// 26.0* 25.9 27.8 29.2 33.1, 30000 of 10 34.1 23.6 16.1 14.6 14.5*; of 128, 8192 of 48
// 35.2 33.8* 36.5 36.5 37.7, 1100 of 48 7.2 7.2* 8.6 12.4 20.9, 600 of 48 5.4* 5.7 7.2 11.7.
// It gives away a few percent where the next number's saving is just under a fifth: 6000 of
// 18 of 128 (bf16) 12.5 12.6 11.3* 10.6 13.4, 8000 of 10 of 256 16.2 15.3 15.0* 14.6 15.0.
int tokens_log2(const AppendArgs &a, int cus) {
  const int heads = a.Hq + 2 * a.Hkv, sets = 256 / (a.D / 16);
  int best = 0;
  int64_t best_cost = 0;
  for (int lg = 0; (sets >> lg) > 0; lg++) {
    const int stride = sets >> lg;
    const int steps = (heads + stride - 1) / stride;
    const int64_t cost = ((int64_t)steps << 16) >> lg;  // lane steps of a token
    const bool fits = a.T >> best < 1 << 23;  // a grid's threads are counted in 32 bits
    if (lg > 0 && fits && ((a.T >> lg) < 2 * cus || steps > 5 || 5 * cost > 4 * best_cost)) continue;
    best = lg;
    best_cost = cost;
  }
  return best;
}

template <int D>
void launch_append(const AppendArgs &a, hipStream_t stream) {
  const int lg = tokens_log2(a, device_cu_count());
  const dim3 grid((unsigned)((a.T + (1 << lg) - 1) >> lg)), block(256);
  const bool more = a.q_weight || a.k_weight || a.k_out;
  if (a.k_scale && more)
    hipLaunchKernelGGL((append_kernel<D, true, true>), grid, block, 0, stream, a, lg);
  else if (a.k_scale)
    hipLaunchKernelGGL((append_kernel<D, true, false>), grid, block, 0, stream, a, lg);
  else if (more)
    hipLaunchKernelGGL((append_kernel<D, false, true>), grid, block, 0, stream, a, lg);
  else
    hipLaunchKernelGGL((append_kernel<D, false, false>), grid, block, 0, stream, a, lg);
}

}  // namespace

hipError_t launch_kv_rope_append(const AppendArgs &a, hipStream_t stream) {
  if (a.D == 64)
    launch_append<64>(a, stream);
  else if (a.D == 128)
    launch_append<128>(a, stream);
  else
    launch_append<256>(a, stream);
  return hipGetLastError();
}

}  // namespace fp8lin
