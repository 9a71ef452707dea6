// Attention of one new token of each sequence over a paged key-value cache.
//
// For query head n of sequence b, over the live tokens t (the last `window` of
// the sequence, or all): score_t = scale q.k_t, capped as c tanh(score / c) when
// a cap is given, o = sum_t softmax(score)_t v_t and lse = log sum_t exp(score_t).
// One pass over keys and values with a running maximum and sum, so each cache
// line is read once for all query heads that share it.
//
// Bound: the cache's bytes.  A token of one key head costs 4 D bytes (bf16)
// against 4 D flops for each query head, far below the matrix rate, so the
// kernel spends matrix instructions freely: the 16 columns of a product hold
// the query heads of one key head (unused ones are zero), and the softmax
// weights enter the second product as two bf16 numbers each.
//
// A workgroup takes one key head, up to 16 RT of its query heads and `chunk`
// tokens; its waves take 32-token tiles in turn, each with a softmax state of
// its own, joined through LDS.  Sequences longer than a chunk leave fp32 partials that
// join_kernel adds in chunk order.
//
// Layouts (v_mfma_f32_16x16x32_bf16: lane l, n = l % 16, g = l / 16):
//   scores   A = K: row n is token n of a half tile, B = Q: column n is a query
//            head; the product over D may take its D values in any order, and
//            lane group g holds values 64 c + 16 g .. + 15, which it loads as 16
//            or 32 contiguous bytes of a token's line;
//   weights  the scores come out with column n = query head and rows 4 g .. + 3 =
//            tokens, which is the B layout of the second product if its 32
//            tokens are counted as (4 g + j of the first half, then of the
//            second): no movement between lanes;
//   values   A = V transposed: lane n loads D / 16 contiguous values of each of
//            its group's 8 tokens (a wave reads whole lines) and v_perm gathers
//            one value of 8 tokens; row n of product i is value (D / 16) n + i.
#include "device_common.hpp"
#include "launch.hpp"
#include "launch_layer.hpp"

namespace fp8lin {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr int kTile = 32;  // tokens of a wave's tile

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));

__device__ __forceinline__ v8bf as_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(v8bf, (v4u{a, b, c, d}));
}

// Two e4m3 codes (the low or the high half of w) as packed bf16, exactly.
template <bool HIGH>
__device__ __forceinline__ uint32_t e4m3x2_to_bf16(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
}

// One tile of a wave as it was loaded.
template <int D, bool FP8>
struct Tile {
  static constexpr int kBytes = FP8 ? 1 : 2;     // of a value
  static constexpr int kK = D * kBytes / 64;     // 16-byte loads of a lane's token in a half tile
  static constexpr int kV = D * kBytes / 16 / 4;  // words of a lane's part of one value line
  uint4 k[2][kK];
  uint32_t v[8][kV];
  float4 ks[2], vs[2];
};

template <int D, bool FP8>
__device__ __forceinline__ void load_tile(Tile<D, FP8> &t, const DecodeArgs &a, const int64_t (&line)[2], int n,
                                          int g) {
  using T = Tile<D, FP8>;
  constexpr int kLine = D * T::kBytes;
#pragma unroll
  for (int hh = 0; hh < 2; hh++) {
    const char *kp = static_cast<const char *>(a.k_cache) + line[hh] * kLine;
    const int at = n * kLine + (FP8 ? 16 : 32) * g;
#pragma unroll
    for (int c = 0; c < T::kK; c++) {
      // bf16: 32 contiguous bytes of each 128; e4m3: 16 of each 64
      const int off = FP8 ? 64 * c : 128 * (c >> 1) + 16 * (c & 1);
      t.k[hh][c] = *reinterpret_cast<const uint4 *>(kp + (at + off));
    }
  }
  if constexpr (FP8) {
#pragma unroll
    for (int hh = 0; hh < 2; hh++) {
      t.ks[hh] = *reinterpret_cast<const float4 *>(a.k_scale + line[hh] + 4 * g);
      t.vs[hh] = *reinterpret_cast<const float4 *>(a.v_scale + line[hh] + 4 * g);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; j++) {
    const char *vp = static_cast<const char *>(a.v_cache) + line[j >> 2] * kLine;
    const int at = (4 * g + (j & 3)) * kLine + n * (kLine / 16);
    if constexpr (T::kV == 1) {
      t.v[j][0] = *reinterpret_cast<const uint32_t *>(vp + at);
    } else if constexpr (T::kV == 2) {
      const uint2 x = *reinterpret_cast<const uint2 *>(vp + at);
      t.v[j][0] = x.x;
      t.v[j][1] = x.y;
    } else {
#pragma unroll
      for (int c = 0; c < T::kV / 4; c++) {
        const uint4 x = *reinterpret_cast<const uint4 *>(vp + (at + 16 * c));
        t.v[j][4 * c] = x.x;
        t.v[j][4 * c + 1] = x.y;
        t.v[j][4 * c + 2] = x.z;
        t.v[j][4 * c + 3] = x.w;
      }
    }
  }
}

// Softmax state of one set of 16 query heads (column n), spread over the lane
// groups: m (log2 units) is the same in all four, l and o are partial.
template <int D>
struct State {
  float m, l;
  v4f o[D / 16];
};

// One tile for the query heads in qf: scores, weights and the product with V.
// t0: the tile's first token; tokens outside [lo, len) count for nothing.
template <int D, bool FP8, int RT>
__device__ __forceinline__ void use_tile(Tile<D, FP8> &t, const DecodeArgs &a, const v8bf (&qf)[RT][D / 32],
                                         State<D> (&st)[RT], int t0, int lo, int len, int g) {
  using T = Tile<D, FP8>;
  v4f s[RT][2];
#pragma unroll
  for (int r = 0; r < RT; r++) s[r][0] = s[r][1] = v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int hh = 0; hh < 2; hh++) {
#pragma unroll
    for (int c = 0; c < D / 32; c++) {
      v8bf kf;
      if constexpr (FP8) {
        const uint4 &raw = t.k[hh][c >> 1];
        const uint32_t w0 = (c & 1) ? raw.z : raw.x, w1 = (c & 1) ? raw.w : raw.y;
        kf = as_bf16x8(e4m3x2_to_bf16<false>(w0), e4m3x2_to_bf16<true>(w0), e4m3x2_to_bf16<false>(w1),
                       e4m3x2_to_bf16<true>(w1));
      } else {
        const uint4 &raw = t.k[hh][c];
        kf = as_bf16x8(raw.x, raw.y, raw.z, raw.w);
      }
#pragma unroll
      for (int r = 0; r < RT; r++) s[r][hh] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, qf[r][c], s[r][hh], 0, 0, 0);
    }
  }
  float factor[8], vs[8];
#pragma unroll
  for (int j = 0; j < 8; j++) {
    factor[j] = a.scale;
    vs[j] = 1.f;
    if constexpr (FP8) {
      factor[j] *= reinterpret_cast<const float *>(&t.ks[j >> 2])[j & 3];
      vs[j] = reinterpret_cast<const float *>(&t.vs[j >> 2])[j & 3];
    }
  }
  uint32_t live = 0xFFu;  // bit j: token j of this lane group counts
  if (t0 < lo || t0 + kTile > len) {
    live = 0;
#pragma unroll
    for (int j = 0; j < 8; j++) {
      const int token = t0 + 16 * (j >> 2) + 4 * g + (j & 3);
      if (token >= lo && token < len) live |= 1u << j;
    }
    // dead lines may hold anything, and 0 times a NaN is one
#pragma unroll
    for (int j = 0; j < 8; j++) {
      if (!(live >> j & 1u)) {
        vs[j] = 0.f;
#pragma unroll
        for (int w = 0; w < T::kV; w++) t.v[j][w] = 0;
      }
    }
  }
  v8bf hi[RT], lo_[RT];
#pragma unroll
  for (int r = 0; r < RT; r++) {
    float x[8];
#pragma unroll
    for (int j = 0; j < 8; j++) x[j] = s[r][j >> 2][j & 3] * factor[j];
    if (a.softcap > 0.f) {
      // c tanh(x / c), with tanh z = 1 - 2 / (1 + exp 2z)
      const float rate = 2.f * kLog2e / a.softcap;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        const float e = __builtin_amdgcn_exp2f(x[j] * rate);
        x[j] = a.softcap - 2.f * a.softcap * __builtin_amdgcn_rcpf(1.f + e);
      }
    }
#pragma unroll
    for (int j = 0; j < 8; j++) x[j] = live >> j & 1u ? x[j] * kLog2e : -INFINITY;
    float top = fmaxf(fmaxf(fmaxf(x[0], x[1]), fmaxf(x[2], x[3])), fmaxf(fmaxf(x[4], x[5]), fmaxf(x[6], x[7])));
    // The reference of the exponents follows the maximum only when some score
    // passes it by 2^8: weights stay below 2^8 and sums far below overflow, and
    // most tiles need no exchange between the lane groups.
    if (__any(top > (st[r].m == -INFINITY ? -INFINITY : st[r].m + 8.f))) {
      top = fmaxf(top, __shfl_xor(top, 16, 64));
      top = fmaxf(top, __shfl_xor(top, 32, 64));
      top = fmaxf(top, st[r].m);
      const float shrink = top == st[r].m ? 1.f : __builtin_amdgcn_exp2f(st[r].m - top);
      st[r].m = top;
      st[r].l *= shrink;
#pragma unroll
      for (int i = 0; i < D / 16; i++) st[r].o[i] *= shrink;
    }
    const float base = st[r].m == -INFINITY ? 0.f : st[r].m;
    float p[8];
#pragma unroll
    for (int j = 0; j < 8; j++) p[j] = __builtin_amdgcn_exp2f(x[j] - base);
    st[r].l += ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
    if constexpr (FP8) {
#pragma unroll
      for (int j = 0; j < 8; j++) p[j] *= vs[j];
    }
    uint32_t h[4], low[4];
#pragma unroll
    for (int j = 0; j < 4; j++) {
      h[j] = pack_bf16x2(p[2 * j], p[2 * j + 1]);
      low[j] = pack_bf16x2(p[2 * j] - bf16_to_f32(h[j] & 0xFFFFu), p[2 * j + 1] - __uint_as_float(h[j] & 0xFFFF0000u));
    }
    hi[r] = as_bf16x8(h[0], h[1], h[2], h[3]);
    lo_[r] = as_bf16x8(low[0], low[1], low[2], low[3]);
  }
  // V: pairs of values (2w, 2w + 1) of all eight tokens, then one product each
#pragma unroll
  for (int w = 0; w < D / 32; w++) {
    uint32_t pair[8];
#pragma unroll
    for (int j = 0; j < 8; j++) {
      if constexpr (FP8)
        pair[j] = (w & 1) ? e4m3x2_to_bf16<true>(t.v[j][w >> 1]) : e4m3x2_to_bf16<false>(t.v[j][w >> 1]);
      else
        pair[j] = t.v[j][w];
    }
#pragma unroll
    for (int e = 0; e < 2; e++) {
      uint32_t f[4];
#pragma unroll
      for (int j = 0; j < 4; j++)
        f[j] = __builtin_amdgcn_perm(pair[2 * j + 1], pair[2 * j], e ? 0x07060302u : 0x05040100u);
      const v8bf vf = as_bf16x8(f[0], f[1], f[2], f[3]);
#pragma unroll
      for (int r = 0; r < RT; r++) {
        v4f &o = st[r].o[2 * w + e];
        o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, hi[r], o, 0, 0, 0);
        o = __builtin_amdgcn_mfma_f32_16x16x32_bf16(vf, lo_[r], o, 0, 0, 0);
      }
    }
  }
}

// Partials of one (sequence, chunk): o [Hq][D], then m and l [Hq] each.
__host__ __device__ inline size_t partial_floats(int Hq, int D) { return (size_t)Hq * (D + 2); }

__host__ __device__ inline int first_token(int len, int window) {
  const int lo = window > 0 && len > window ? len - window : 0;
  return lo & ~(kTile - 1);
}

// Whether a wave loads its next tile before it uses the present one: where two
// tiles and the state fit the registers of two waves on a SIMD (or one, for D = 256).
template <int D, int RT>
constexpr bool kAhead = D * RT <= 128 || RT == 1;

template <int D, bool FP8, int RT, int NW>
__global__ __launch_bounds__(64 * NW, D <= 128 ? 2 : 1) void decode_kernel(DecodeArgs a, int chunk, int splits, float *part) {
  constexpr int kPad = D + 4;  // a row of LDS, off the bank period
  extern __shared__ __align__(16) char lds[];
  int64_t *lines = reinterpret_cast<int64_t *>(lds);  // first cache line of each half tile
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, n = lane & 15, g = lane >> 4;
  const int split = blockIdx.x, b = blockIdx.z;
  const int group = a.Hq / a.Hkv, bands = (group + 16 * RT - 1) / (16 * RT);
  const int kvh = blockIdx.y / bands, head0 = (blockIdx.y % bands) * 16 * RT;
  const int heads = min(group - head0, 16 * RT);  // query heads of this workgroup
  const int64_t q0 = (int64_t)b * a.Hq + kvh * group + head0;
  const int len = min(max(a.seq_lens[b], 0), a.max_len);
  const int lo = a.window > 0 ? max(0, len - a.window) : 0;
  const int begin = first_token(len, a.window) + split * chunk;
  const int end = min(len, begin + chunk);
  if (begin >= end && !(split == 0)) return;  // chunks past the sequence; the first one writes its zeros
  const int halves = begin < end ? (end - begin + 15) / 16 : 0;
  for (int i = threadIdx.x; i < (halves + 1) / 2 * 2; i += 64 * NW) {
    const int token = begin + 16 * min(i, halves - 1);  // the odd last half tile repeats, its tokens are dead
    const int at = token / a.page_size;
    const int page = min(max(a.block_table[(int64_t)b * a.max_pages + at], 0), a.pages - 1);
    lines[i] = ((int64_t)page * a.Hkv + kvh) * a.page_size + (token - at * a.page_size);
  }
  v8bf qf[RT][D / 32];
#pragma unroll
  for (int r = 0; r < RT; r++) {
#pragma unroll
    for (int c = 0; c < D / 32; c++) {
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (16 * r + n < heads)
        raw = *reinterpret_cast<const uint4 *>(a.q + (q0 + 16 * r + n) * D + 64 * (c >> 1) + 16 * g + 8 * (c & 1));
      qf[r][c] = as_bf16x8(raw.x, raw.y, raw.z, raw.w);
    }
  }
  State<D> st[RT];
#pragma unroll
  for (int r = 0; r < RT; r++) {
    st[r].m = -INFINITY;
    st[r].l = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; i++) st[r].o[i] = v4f{0.f, 0.f, 0.f, 0.f};
  }
  __syncthreads();
  const int tiles = (halves + 1) / 2;
  auto load = [&](Tile<D, FP8> &t, int i) {
    int64_t line[2];
#pragma unroll
    for (int hh = 0; hh < 2; hh++) {
      const int64_t x = lines[2 * i + hh];
      line[hh] = (int64_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)x) |
                 (int64_t)__builtin_amdgcn_readfirstlane((int)(x >> 32)) << 32;
    }
    load_tile<D, FP8>(t, a, line, n, g);
  };
  Tile<D, FP8> ta;
  if constexpr (kAhead<D, RT>) {
    Tile<D, FP8> tb;
    int i = wave;
    if (i < tiles) load(ta, i);
    while (i < tiles) {
      if (i + NW < tiles) load(tb, i + NW);
      use_tile<D, FP8, RT>(ta, a, qf, st, begin + kTile * i, lo, end, g);
      i += NW;
      if (i >= tiles) break;
      if (i + NW < tiles) load(ta, i + NW);
      use_tile<D, FP8, RT>(tb, a, qf, st, begin + kTile * i, lo, end, g);
      i += NW;
    }
  } else {
    for (int i = wave; i < tiles; i += NW) {
      load(ta, i);
      use_tile<D, FP8, RT>(ta, a, qf, st, begin + kTile * i, lo, end, g);
    }
  }
#pragma unroll
  for (int r = 0; r < RT; r++) {
    st[r].l += __shfl_xor(st[r].l, 16, 64);
    st[r].l += __shfl_xor(st[r].l, 32, 64);
  }
  // join the waves' states pairwise, in a fixed order, through LDS
  float *box_o = reinterpret_cast<float *>(lds);
  float *box_m = box_o + NW / 2 * 16 * RT * kPad, *box_l = box_m + NW / 2 * 16 * RT;
#pragma unroll
  for (int half = NW / 2; half >= 1; half /= 2) {
    __syncthreads();
    if (wave >= half && wave < 2 * half) {
#pragma unroll
      for (int r = 0; r < RT; r++) {
        const int row = (wave - half) * 16 * RT + 16 * r + n;
#pragma unroll
        for (int k = 0; k < 4; k++) {
#pragma unroll
          for (int e = 0; e < D / 16; e++) box_o[row * kPad + D / 16 * (4 * g + k) + e] = st[r].o[e][k];
        }
        if (g == 0) {
          box_m[row] = st[r].m;
          box_l[row] = st[r].l;
        }
      }
    }
    __syncthreads();
    if (wave < half) {
#pragma unroll
      for (int r = 0; r < RT; r++) {
        const int row = wave * 16 * RT + 16 * r + n;
        const float m2 = box_m[row], top = fmaxf(st[r].m, m2);
        const float f1 = st[r].m == top ? 1.f : __builtin_amdgcn_exp2f(st[r].m - top);
        const float f2 = m2 == top ? 1.f : __builtin_amdgcn_exp2f(m2 - top);
        st[r].m = top;
        st[r].l = st[r].l * f1 + box_l[row] * f2;
#pragma unroll
        for (int k = 0; k < 4; k++) {
#pragma unroll
          for (int e = 0; e < D / 16; e++)
            st[r].o[e][k] = st[r].o[e][k] * f1 + box_o[row * kPad + D / 16 * (4 * g + k) + e] * f2;
        }
      }
    }
  }
  if (wave != 0) return;
#pragma unroll
  for (int r = 0; r < RT; r++) {
    const int head = 16 * r + n;
    if (head >= heads) continue;
    if (splits == 1) {
      const float inv = st[r].l == 0.f ? 0.f : 1.f / st[r].l;
      uint16_t *dst = a.o + (q0 + head) * D;
#pragma unroll
      for (int k = 0; k < 4; k++) {
#pragma unroll
        for (int e = 0; e < D / 16; e += 4)
          *reinterpret_cast<uint2 *>(dst + D / 16 * (4 * g + k) + e) =
              make_uint2(pack_bf16x2(st[r].o[e][k] * inv, st[r].o[e + 1][k] * inv),
                         pack_bf16x2(st[r].o[e + 2][k] * inv, st[r].o[e + 3][k] * inv));
      }
      if (a.lse && g == 0) a.lse[q0 + head] = st[r].l == 0.f ? -INFINITY : kLn2 * (st[r].m + log2f(st[r].l));
    } else {
      float *base = part + ((size_t)b * splits + split) * partial_floats(a.Hq, D);
      const int at = kvh * group + head0 + head;
#pragma unroll
      for (int k = 0; k < 4; k++) {
#pragma unroll
        for (int e = 0; e < D / 16; e += 4)
          *reinterpret_cast<float4 *>(base + (size_t)at * D + D / 16 * (4 * g + k) + e) =
              make_float4(st[r].o[e][k], st[r].o[e + 1][k], st[r].o[e + 2][k], st[r].o[e + 3][k]);
      }
      if (g == 0) {
        base[(size_t)a.Hq * D + at] = st[r].m;
        base[(size_t)a.Hq * (D + 1) + at] = st[r].l;
      }
    }
  }
}

// Joins the chunks of one query head, in chunk order.
template <int D>
__global__ __launch_bounds__(64) void join_kernel(DecodeArgs a, int chunk, int splits, const float *part) {
  constexpr int E = D / 64;
  const int head = blockIdx.x, b = blockIdx.y, lane = threadIdx.x;
  const int len = min(max(a.seq_lens[b], 0), a.max_len);
  const int live = max(1, (len - first_token(len, a.window) + chunk - 1) / chunk);
  const size_t stride = partial_floats(a.Hq, D);
  const float *base = part + (size_t)b * splits * stride;
  float top = -INFINITY;
  for (int s = lane; s < live; s += 64) top = fmaxf(top, base[s * stride + (size_t)a.Hq * D + head]);
  for (int off = 32; off; off >>= 1) top = fmaxf(top, __shfl_xor(top, off, 64));
  float l = 0.f, o[E] = {};
  for (int s = 0; s < live; s++) {
    const float *p = base + s * stride;
    const float m = p[(size_t)a.Hq * D + head];
    const float f = m == top ? 1.f : __builtin_amdgcn_exp2f(m - top);
    l += p[(size_t)a.Hq * (D + 1) + head] * f;
#pragma unroll
    for (int e = 0; e < E; e++) o[e] += p[(size_t)head * D + E * lane + e] * f;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
  const int64_t at = (int64_t)b * a.Hq + head;
#pragma unroll
  for (int e = 0; e < E; e++) a.o[at * D + E * lane + e] = (uint16_t)f32_to_bf16_rne(o[e] * inv);
  if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : kLn2 * (top + log2f(l));
}

constexpr int kWaves = 4;

// Tokens of a chunk and the chunks of the longest sequence: enough workgroups
// to cover the compute units a few times, in whole rounds of the waves' tiles.
struct Plan {
  int chunk, splits;
};

Plan plan_decode(const DecodeArgs &a, int cus) {
  const int round = kWaves * kTile;
  // live tokens of a sequence, from the tile that holds the first one
  int64_t tokens = a.max_len;
  if (a.window > 0) tokens = tokens < (int64_t)a.window + kTile ? tokens : (int64_t)a.window + kTile;
  if (tokens < 1) tokens = 1;
  const int64_t rows = (int64_t)a.B * a.Hkv * ((a.Hq / a.Hkv + 15) / 16);
  const int64_t want = (4 * (int64_t)cus + rows - 1) / rows;  // chunks of a sequence
  int64_t chunk = (tokens + want - 1) / want;
  chunk = (chunk + round - 1) / round * round;
  if (chunk < 2 * round) chunk = 2 * round;
  if (chunk > 16384) chunk = 16384;  // its page table stays below 16 KB of LDS
  return Plan{(int)chunk, (int)((tokens + chunk - 1) / chunk)};
}

template <int D, bool FP8, int RT>
hipError_t launch_decode(const DecodeArgs &a, const Plan &p, float *part, hipStream_t stream) {
  constexpr int NW = kWaves;
  const int group = a.Hq / a.Hkv, bands = (group + 16 * RT - 1) / (16 * RT);
  const size_t join = (size_t)NW / 2 * 16 * RT * (D + 6) * sizeof(float);
  const size_t lines = (size_t)(p.chunk / 16) * sizeof(int64_t);
  const size_t lds = join > lines ? join : lines;
  auto *kernel = decode_kernel<D, FP8, RT, NW>;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  hipLaunchKernelGGL(kernel, dim3((unsigned)p.splits, (unsigned)(a.Hkv * bands), (unsigned)a.B), dim3(64 * NW), lds,
                     stream, a, p.chunk, p.splits, part);
  if (p.splits > 1)
    hipLaunchKernelGGL(join_kernel<D>, dim3((unsigned)a.Hq, (unsigned)a.B), dim3(64), 0, stream, a, p.chunk, p.splits,
                       (const float *)part);
  return hipGetLastError();
}

template <int D, bool FP8>
hipError_t launch_rows(const DecodeArgs &a, const Plan &p, float *part, hipStream_t stream) {
  if (a.Hq / a.Hkv <= 16) return launch_decode<D, FP8, 1>(a, p, part, stream);
  return launch_decode<D, FP8, 2>(a, p, part, stream);
}

template <int D>
hipError_t launch_dim(const DecodeArgs &a, const Plan &p, float *part, hipStream_t stream) {
  return a.k_scale ? launch_rows<D, true>(a, p, part, stream) : launch_rows<D, false>(a, p, part, stream);
}

}  // namespace

size_t paged_decode_partial_bytes(const DecodeArgs &a, int cus) {
  const Plan p = plan_decode(a, cus);
  return p.splits > 1 ? (size_t)a.B * p.splits * partial_floats(a.Hq, a.D) * sizeof(float) : 0;
}

hipError_t launch_paged_decode(const DecodeArgs &a, float *part, hipStream_t stream) {
  const Plan p = plan_decode(a, device_cu_count());
  if (a.D == 64) return launch_dim<64>(a, p, part, stream);
  if (a.D == 128) return launch_dim<128>(a, p, part, stream);
  return launch_dim<256>(a, p, part, stream);
}

}  // namespace fp8lin
