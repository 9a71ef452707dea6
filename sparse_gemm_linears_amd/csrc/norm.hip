// Residual addition, root-mean-square norm and e4m3 quantization of one row:
//   h = x + res,  y = h / sqrt(mean(h^2) + eps) * w,
//   codes and scale of each 128 channels of y.
//
// One pass over HBM: a row is held in fp32 registers between the sum of
// squares and the output, so x and res are read once and h, the codes and the
// scales written once (7.03 bytes per element with a residual).  HBM-bound
// for many rows: 8192 x 7168 with a residual, 413 MB in 66 us, 6.3 TB/s.  One row
// is bound by two memory latencies and the launch: 1 x 4096 in 2.9 us.  (Times in this
// file: one call of a replayed graph of twelve over three sets of inputs in turn.  Issued
// one by one, calls take 75 and 7 us.)
//
// Numbers: h is exact in fp32 up to one rounding; the sum of squares is taken
// in fp32 over the unrounded h, each lane's elements in order and the lanes in
// a fixed tree, so results are deterministic.  y is not rounded to bf16 before
// it is quantized: each code is one rounding of an fp32 value.
#include "device_common.hpp"
#include "launch_layer.hpp"

namespace fp8lin {
namespace {

// Sum over the wave's 64 lanes in a fixed order, in every lane: four steps
// inside each DPP row, then the four row sums.
__device__ __forceinline__ float wave_sum(float v) {
  auto add = [](float x, int moved) { return x + __int_as_float(moved); };
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0xB1, 0xF, 0xF, false));   // quad_perm 1,0,3,2
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x4E, 0xF, 0xF, false));   // quad_perm 2,3,0,1
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x124, 0xF, 0xF, false));  // row_ror 4
  v = add(v, __builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xF, 0xF, false));  // row_ror 8
  const float r0 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 0));
  const float r1 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 16));
  const float r2 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 32));
  const float r3 = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 48));
  return (r0 + r1) + (r2 + r3);
}

__device__ __forceinline__ uint4 ld16(const uint16_t *p) { return *reinterpret_cast<const uint4 *>(p); }

template <bool STREAM>
__device__ __forceinline__ uint4 load16(const uint16_t *p) {
  return STREAM ? ldg16_stream(p) : ld16(p);
}

// Output of eight values of one row at column 8c: y, and the codes and scale
// of the group that this lane and its 15 neighbours (one DPP row) hold.  The
// 16 lanes are all active or all inactive, because K is a multiple of 128.
__device__ __forceinline__ void emit8(const NormArgs &a, ScaleKind kind, int64_t row, int c, const float (&v)[8]) {
  const int64_t at = row * a.K + 8 * (int64_t)c;
  if (a.y) *reinterpret_cast<uint4 *>(a.y + at) = pack8(v);
  if (!a.q) return;
  uint32_t m = 0;
#pragma unroll
  for (int j = 0; j < 8; j++) m = max(m, __float_as_uint(v[j]) & 0x7FFFFFFFu);
  m = row16_max(m);
  uint2 codes;
  const int64_t group = row * (a.K / kGroup) + (c >> 4);
  if (kind == ScaleKind::kUe8m0) {
    // a group with an infinity or a NaN gets the scale byte that stands for NaN
    const bool finite = m < 0x7F800000u;
    const uint32_t e = finite ? ue8m0_exponent(m) : 255u;
    const float inv = finite ? ue8m0_inverse(e) : 0.0f;
    codes = make_uint2(e4m3_pack4(v[0] * inv, v[1] * inv, v[2] * inv, v[3] * inv),
                       e4m3_pack4(v[4] * inv, v[5] * inv, v[6] * inv, v[7] * inv));
    if ((c & 15) == 0) static_cast<uint8_t *>(a.scales)[group] = (uint8_t)e;
  } else {
    float s;
    codes = quantize8_f32(v, m, s);
    if ((c & 15) == 0) static_cast<float *>(a.scales)[group] = s;
  }
  *reinterpret_cast<uint2 *>(a.q + at) = codes;
}

// TEAM threads hold one row, V chunks of eight elements each (K <= 8 TEAM V).
// STREAM: x and res bypass the caches.
template <int TEAM, int V, bool STREAM>
__global__ __launch_bounds__(TEAM < 256 ? 256 : TEAM) void rmsnorm_kernel(NormArgs a, ScaleKind kind) {
  constexpr int kRows = TEAM < 256 ? 256 / TEAM : 1;
  constexpr int kWaves = TEAM / 64;
  const int t = threadIdx.x % TEAM;
  const int64_t row = (int64_t)blockIdx.x * kRows + threadIdx.x / TEAM;
  if (row >= a.M) return;  // whole waves, and only in the one-wave form, which has no barrier
  const int chunks = a.K / 8;
  const int64_t base = row * a.K;
  uint4 xr[V], wr[V];
#pragma unroll
  for (int i = 0; i < V; i++) {
    const int c = i * TEAM + t;
    xr[i] = load16<STREAM>(a.x + base + 8 * (int64_t)(c < chunks ? c : 0));
  }
  float h[V][8];
  if (a.res) {
    uint4 rr[V];
#pragma unroll
    for (int i = 0; i < V; i++) {
      const int c = i * TEAM + t;
      rr[i] = load16<STREAM>(a.res + base + 8 * (int64_t)(c < chunks ? c : 0));
    }
#pragma unroll
    for (int i = 0; i < V; i++) {
      const int c = i * TEAM + t;
      wr[i] = ld16(a.w + 8 * (c < chunks ? c : 0));
    }
#pragma unroll
    for (int i = 0; i < V; i++) {
      float r[8];
      unpack8(xr[i], h[i]);
      unpack8(rr[i], r);
#pragma unroll
      for (int j = 0; j < 8; j++) h[i][j] += r[j];
      const int c = i * TEAM + t;
      if (c < chunks) *reinterpret_cast<uint4 *>(a.h + base + 8 * (int64_t)c) = pack8(h[i]);
    }
  } else {
#pragma unroll
    for (int i = 0; i < V; i++) {
      const int c = i * TEAM + t;
      wr[i] = ld16(a.w + 8 * (c < chunks ? c : 0));
    }
#pragma unroll
    for (int i = 0; i < V; i++) unpack8(xr[i], h[i]);
  }
  float ss = 0.f;
#pragma unroll
  for (int i = 0; i < V; i++) {
    float part = 0.f;
#pragma unroll
    for (int j = 0; j < 8; j++) part = __builtin_fmaf(h[i][j], h[i][j], part);
    ss += i * TEAM + t < chunks ? part : 0.f;
  }
  ss = wave_sum(ss);
  if constexpr (kWaves > 1) {
    __shared__ float wave_ss[kWaves];
    if ((t & 63) == 0) wave_ss[t >> 6] = ss;
    __syncthreads();
    ss = 0.f;
#pragma unroll
    for (int i = 0; i < kWaves; i++) ss += wave_ss[i];
  }
  const float rinv = 1.0f / sqrtf(ss / (float)a.K + a.eps);
#pragma unroll
  for (int i = 0; i < V; i++) {
    const int c = i * TEAM + t;
    if (c >= chunks) continue;
    float w[8];
    unpack8(wr[i], w);
#pragma unroll
    for (int j = 0; j < 8; j++) h[i][j] = h[i][j] * rinv * w[j];
    emit8(a, kind, row, c, h[i]);
  }
}

// Rows longer than the register forms hold: two passes over the row, the
// second from the caches where it fits them.  h is written in the second pass
// only, because it may be the same memory as res.
__global__ __launch_bounds__(1024) void rmsnorm_long_kernel(NormArgs a, ScaleKind kind) {
  __shared__ float wave_ss[16];
  const int t = threadIdx.x;
  const int64_t row = blockIdx.x, base = row * a.K;
  const int chunks = a.K / 8;
  auto load = [&](int c, float (&h)[8]) {
    unpack8(ld16(a.x + base + 8 * (int64_t)c), h);
    if (a.res) {
      float r[8];
      unpack8(ld16(a.res + base + 8 * (int64_t)c), r);
#pragma unroll
      for (int j = 0; j < 8; j++) h[j] += r[j];
    }
  };
  float ss = 0.f;
  for (int c = t; c < chunks; c += 1024) {
    float h[8], part = 0.f;
    load(c, h);
#pragma unroll
    for (int j = 0; j < 8; j++) part = __builtin_fmaf(h[j], h[j], part);
    ss += part;
  }
  ss = wave_sum(ss);
  if ((t & 63) == 0) wave_ss[t >> 6] = ss;
  __syncthreads();
  ss = 0.f;
#pragma unroll
  for (int i = 0; i < 16; i++) ss += wave_ss[i];
  const float rinv = 1.0f / sqrtf(ss / (float)a.K + a.eps);
  for (int c = t; c < chunks; c += 1024) {
    float h[8], w[8];
    load(c, h);
    unpack8(ld16(a.w + 8 * (int64_t)c), w);
    if (a.res) *reinterpret_cast<uint4 *>(a.h + base + 8 * (int64_t)c) = pack8(h);
#pragma unroll
    for (int j = 0; j < 8; j++) h[j] = h[j] * rinv * w[j];
    emit8(a, kind, row, c, h);
  }
}

// Inputs that the caches cannot hold (256 MB for all of a launch's data) are read
// past them: 8192 x 7168 with a residual 73.5 -> 65.8 us, 16384 x 3584 74.2 -> 65.7.
// Smaller ones may be there from the call that made them: 2048 x 16384 with a
// residual 41.2 -> 42.7 us, 4093 x 4096 without (bf16 output too) 15.8 -> 17.8 us so.
constexpr int64_t kStreamBytes = int64_t(192) << 20;
bool streams(const NormArgs &a) { return a.M * a.K * (a.res ? 4 : 2) > kStreamBytes; }

template <int TEAM, int V>
void launch_rows(const NormArgs &a, ScaleKind kind, hipStream_t stream) {
  constexpr int kRows = TEAM < 256 ? 256 / TEAM : 1;
  const dim3 grid((unsigned)((a.M + kRows - 1) / kRows)), block(TEAM < 256 ? 256 : TEAM);
  if (streams(a))
    hipLaunchKernelGGL((rmsnorm_kernel<TEAM, V, true>), grid, block, 0, stream, a, kind);
  else
    hipLaunchKernelGGL((rmsnorm_kernel<TEAM, V, false>), grid, block, 0, stream, a, kind);
}

void launch_matrix(const NormArgs &a, ScaleKind kind, hipStream_t stream) {
  // Threads of a row, measured with a residual: 4096 wide, one row 512 threads 2.85
  // us, 256 3.29, 1024 2.98, 64 5.56, and 2048 rows 12.2 / 12.7 / 13.0 / 14.2; 8192
  // wide, 512 rows 512 threads 8.5, 256 8.8, 1024 8.3; 16384 wide, 1024 rows 1024
  // threads 21.5, 512 22.6; 2048 wide, 4096 rows 256 threads 12.0, 64 13.0, 512
  // 12.1; 512 wide, 4096 rows 64 threads 4.7, 256 5.7.
  if (a.K <= 512)
    launch_rows<64, 1>(a, kind, stream);
  else if (a.K <= 1024)
    launch_rows<64, 2>(a, kind, stream);
  else if (a.K <= 2048)
    launch_rows<256, 1>(a, kind, stream);
  else if (a.K <= 4096 && streams(a))  // 16384 rows of 3584: 256 threads 65.6 us, 512 69.3
    launch_rows<256, 2>(a, kind, stream);
  else if (a.K <= 4096)
    launch_rows<512, 1>(a, kind, stream);
  else if (a.K <= 8192)
    launch_rows<512, 2>(a, kind, stream);
  else if (a.K <= 16384)
    launch_rows<1024, 2>(a, kind, stream);
  else if (a.K <= 32768)
    launch_rows<1024, 4>(a, kind, stream);
  else
    hipLaunchKernelGGL(rmsnorm_long_kernel, dim3((unsigned)a.M), dim3(1024), 0, stream, a, kind);
}

// Rows of one launch: a grid's threads are counted in 32 bits.
constexpr int64_t kLaunchRows = int64_t(1) << 21;

}  // namespace

hipError_t launch_add_rmsnorm(const NormArgs &a, ScaleKind kind, hipStream_t stream) {
  for (int64_t row = 0; row < a.M; row += kLaunchRows) {
    const int64_t at = row * a.K, scale_at = at / 128 * (kind == ScaleKind::kFp32 ? 4 : 1);
    NormArgs p = a;
    p.M = a.M - row < kLaunchRows ? a.M - row : kLaunchRows;
    p.x = a.x + at;
    if (a.res) p.res = a.res + at, p.h = a.h + at;
    if (a.y) p.y = a.y + at;
    if (a.q) p.q = a.q + at, p.scales = static_cast<uint8_t *>(a.scales) + scale_at;
    launch_matrix(p, kind, stream);
    if (hipError_t e = hipGetLastError()) return e;
  }
  return hipSuccess;
}

}  // namespace fp8lin
