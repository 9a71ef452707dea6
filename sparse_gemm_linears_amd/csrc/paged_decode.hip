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
// A row is one key head of one sequence with up to 16 RT of its query heads, and
// work is counted in tiles of 32 tokens.  Lengths are known on the device only,
// and a grid made for the longest sequence leaves most of it without work in a
// ragged batch.  So a fixed number of waves divides the batch into even shares:
// each finds its share from the lengths and takes the rows in it in turn, alone,
// without barriers; eight waves on a compute unit (four for D = 256) keep its loads going.  A wave
// leaves a partial for the row that its share begins inside and for the one that it
// ends inside, and join_kernel adds the partials of a row in order.  Short
// sequences, one sequence alone, windows, and batches that give each wave a few tiles
// at most are divided by the grid, without the search (row_kernel).
//
// Measured with 8 key heads of 128 (medians of a kernel trace): 131072 tokens of one
// sequence in bf16, 537 MB in 84 us, 6.4 TB/s, and 5 us for the join; 64 sequences of 1
// to 8192 tokens in e4m3, 373 MB in 68 us, 5.5 TB/s, and 6 us; 777 tokens of one sequence
// 5.7 us and 4 us.
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
#include "decode_plan.hpp"
#include "device_common.hpp"
#include "launch.hpp"
#include "launch_layer.hpp"

namespace fp8lin {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

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
      const v2u x = __builtin_nontemporal_load(reinterpret_cast<const v2u *>(vp + at));
      t.v[j][0] = x[0];
      t.v[j][1] = x[1];
    } else {
#pragma unroll
      for (int c = 0; c < T::kV / 4; c++) {
        const uint4 x = ldg16_stream(vp + (at + 16 * c));
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
      // c tanh(x / c).  tanh z = 1 - 2 / (1 + exp 2z), but below 1/4, where that
      // would lose a small score's low bits, its power series (2^-26 of it is left out).
      const float rate = 1.f / a.softcap;
      float z[8], most = 0.f;
#pragma unroll
      for (int j = 0; j < 8; j++) {
        z[j] = x[j] * rate;
        const float u = z[j] * z[j];
        float t = __builtin_fmaf(u, 62.f / 2835.f, -17.f / 315.f);
        t = __builtin_fmaf(u, t, 2.f / 15.f);
        t = __builtin_fmaf(u, t, -1.f / 3.f);
        x[j] = a.softcap * __builtin_fmaf(z[j] * u, t, z[j]);
        most = fmaxf(most, fabsf(z[j]));
      }
      if (__any(most >= 0.25f)) {
#pragma unroll
        for (int j = 0; j < 8; j++) {
          const float m = fabsf(z[j]), e = __builtin_amdgcn_exp2f(2.f * kLog2e * m);
          if (m >= 0.25f) x[j] = a.softcap * copysignf(1.f - 2.f * __builtin_amdgcn_rcpf(1.f + e), z[j]);
        }
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

constexpr int kWaves = 4;  // of a workgroup; each works alone
constexpr int kThreads = 64 * kWaves;
constexpr int kListed = 64;  // tiles that a wave lists at a time, one in each lane

__device__ __forceinline__ int length_of(const DecodeArgs &a, int b) {
  return b < a.B ? min(max(a.seq_lens[b], 0), a.max_len) : 0;
}

// Tiles of a sequence (an empty one has a tile without live tokens, which
// writes its zeros).
__device__ __forceinline__ int tiles_of(const DecodeArgs &a, int len) {
  return max(1, (len - first_token(len, a.window) + kTile - 1) / kTile);
}

// A row that is divided (slot < 0: none): its parts are in `slot` and in slot 0 of
// the owners that follow `owner`: `parts` of them in all, or (parts == 0) as many
// as have shares that start before row_end.
struct Cut {
  int64_t total, row_end;
  int b, band, slot, parts;
  int owner, pad;
};

// A unit of the batch: tile `tile` of row `band` of sequence b, or (tile ==
// tiles_of) the row's end.
struct Place {
  int b, band, tile, len;
};

// All units of the batch; before and upto: those of the sequences before this
// lane's run of sequences, and with it.
__device__ __forceinline__ int64_t batch_units(const DecodeArgs &a, int rows, int lane, int64_t &before,
                                               int64_t &upto) {
  const int per = (a.B + 63) / 64, b0 = lane * per, b1 = min(a.B, b0 + per);
  int64_t mine = 0;
  for (int i = b0; i < b1; i++) mine += tiles_of(a, length_of(a, i)) + 1;
  mine *= rows;
  upto = mine;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int64_t x = __shfl_up(upto, off, 64);
    if (lane >= off) upto += x;
  }
  before = upto - mine;
  return __shfl(upto, 63, 64);
}

// A row: key head kvh of sequence b with `heads` query heads from q0 of all on.
struct Row {
  int kvh, heads;
  int64_t q0;
  __device__ Row(const DecodeArgs &a, int b, int band, int RT) {
    const int group = a.Hq / a.Hkv, bands = (group + 16 * RT - 1) / (16 * RT);
    kvh = band / bands;
    const int head0 = (band - kvh * bands) * 16 * RT;
    heads = min(group - head0, 16 * RT);
    q0 = (int64_t)b * a.Hq + kvh * group + head0;
  }
};

template <int D, bool FP8, int RT>
__device__ __forceinline__ void load_queries(v8bf (&qf)[RT][D / 32], const DecodeArgs &a, const Row &row, int n,
                                             int g) {
#pragma unroll
  for (int r = 0; r < RT; r++) {
#pragma unroll
    for (int c = 0; c < D / 32; c++) {
      uint4 raw = make_uint4(0, 0, 0, 0);
      if (16 * r + n < row.heads)
        raw = *reinterpret_cast<const uint4 *>(a.q + (row.q0 + 16 * r + n) * D + 64 * (c >> 1) + 16 * g + 8 * (c & 1));
      qf[r][c] = as_bf16x8(raw.x, raw.y, raw.z, raw.w);
    }
  }
}

template <int D, int RT>
__device__ __forceinline__ void clear_state(State<D> (&st)[RT]) {
#pragma unroll
  for (int r = 0; r < RT; r++) {
    st[r].m = -INFINITY;
    st[r].l = 0.f;
#pragma unroll
    for (int i = 0; i < D / 16; i++) st[r].o[i] = v4f{0.f, 0.f, 0.f, 0.f};
  }
}

// The cache line of `token` of sequence b (which must be below max_len).
__device__ __forceinline__ int64_t line_of(const DecodeArgs &a, int b, int kvh, int token) {
  const int p = (int)((uint32_t)token / (uint32_t)a.page_size);
  const int page = min(max(a.block_table[(int64_t)b * a.max_pages + p], 0), a.pages - 1);
  return ((int64_t)page * a.Hkv + kvh) * a.page_size + (token - p * a.page_size);
}

__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int from_lane(int x, int lane) { return __builtin_amdgcn_readlane(x, lane); }
__device__ __forceinline__ int64_t from_lane(int64_t x, int lane) {
  return (int64_t)(uint32_t)from_lane((int)x, lane) | (int64_t)from_lane((int)(x >> 32), lane) << 32;
}

// Quotient of a unit's place among a sequence's units by the units of a row.
__device__ __forceinline__ int row_of(int64_t inside, int units) {
  return inside >> 31 ? (int)(inside / units) : (int)((uint32_t)inside / (uint32_t)units);
}

__device__ __forceinline__ Place find_unit(const DecodeArgs &a, int rows, int lane, int64_t at, int64_t before,
                                           int64_t upto) {
  const int per = (a.B + 63) / 64, b0 = lane * per, b1 = min(a.B, b0 + per);
  int b = 0, band = 0, tile = 0, len = 0;
  const bool mine = at >= before && at < upto;
  if (mine) {
    b = b0;
    len = length_of(a, b);
    int64_t inside = at - before;
    for (int64_t n; b + 1 < b1 && inside >= (n = (int64_t)(tiles_of(a, len) + 1) * rows); inside -= n) len = length_of(a, ++b);
    const int units = tiles_of(a, len) + 1;
    band = row_of(inside, units);
    tile = (int)(inside - (int64_t)band * units);
  }
  const int src = __ffsll((unsigned long long)__ballot(mine)) - 1;
  return Place{from_lane(b, src), from_lane(band, src), from_lane(tile, src), from_lane(len, src)};
}

template <int D, bool FP8, int RT>
__global__ __launch_bounds__(kThreads, D <= 128 ? (RT == 1 ? 3 : 2) : 2) void decode_kernel(DecodeArgs a, DecodePlan plan, float *part,
                                                                           Cut *cuts) {
  const int lane = threadIdx.x & 63, n = lane & 15, g = lane >> 4;
  const int self = uniform((int)blockIdx.x * kWaves + (int)(threadIdx.x >> 6));
  if (self >= plan.owners) return;
  const int group = a.Hq / a.Hkv, bands = (group + 16 * RT - 1) / (16 * RT), rows = a.Hkv * bands;

  Place at;      // the next tile to list
  int64_t left;  // units of the share that are not listed yet
  int64_t total = 0, position = 0;  // units of the batch, and where the share starts in them
  int64_t before, upto;
  total = batch_units(a, rows, lane, before, upto);
  position = share_start(self, total, plan.log2_parts);
  left = share_start(self + 1, total, plan.log2_parts) - position;
  if (!plan.by_row && lane == 0) cuts[self].slot = -1;
  if (left <= 0) return;  // there are more waves than units
  at = find_unit(a, rows, lane, position, before, upto);
  auto next_row = [&] {
    at.tile = 0;
    if (++at.band == rows) {
      at.band = 0;
      at.b++;
      at.len = uniform(length_of(a, at.b));
    }
  };
  if (at.tile == tiles_of(a, at.len)) {  // a row's end alone: nothing is left to do for it
    if (--left == 0) return;
    position++;
    next_row();
  }
  bool started = true;        // whether this is the share's first row
  int row_begin = at.tile;    // first tile of the present row that is in the share
  int64_t row_position = position - at.tile;  // of the present row's first tile

  v8bf qf[RT][D / 32];
  State<D> st[RT];
  bool fresh = true;  // whether the next tile begins a row (here)

  while (left > 0) {
    // list the next units: lane x finds unit x and its cache lines
    const int count = (int)min(left, (int64_t)kListed);
    int rb = at.b, rband = at.band, rtile = at.tile + lane, rlen = at.len;
    if (count > tiles_of(a, at.len) + 1 - at.tile) {  // they reach past the present row
      const int len = length_of(a, at.b + lane), units = tiles_of(a, len) + 1;
      // units of sequence at.b + lane from here on (more than 1024 are as good), and their running sum
      const int64_t all = (int64_t)units * rows - (lane == 0 ? (int64_t)at.band * units + at.tile : 0);
      int mine = at.b + lane < a.B ? (int)min(all, (int64_t)1024) : 0, upto = mine;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int x = __shfl_up(upto, off, 64);
        if (lane >= off) upto += x;
      }
      int s = 0;  // first sequence whose running sum passes the lane's number
#pragma unroll
      for (int step = 32; step; step >>= 1)
        if (__shfl(upto, s + step - 1, 64) <= lane) s += step;
      const int before = __shfl(upto - mine, s, 64);
      const int sunits = __shfl(units, s, 64);
      rlen = __shfl(len, s, 64);
      rb = at.b + s;
      const int64_t inside = lane - before + (s == 0 ? (int64_t)at.band * sunits + at.tile : 0);
      rband = row_of(inside, sunits);
      rtile = (int)(inside - (int64_t)rband * sunits);
    }
    const int rtoken = first_token(rlen, a.window) + rtile * kTile;
    int64_t rline[2] = {0, 0};  // of tokens past the end, which count for nothing: any line will do
    const int rkvh = rband / bands;
#pragma unroll
    for (int hh = 0; hh < 2; hh++) {
      const int token = rtoken + 16 * hh;
      if (lane < count && token < rlen) rline[hh] = line_of(a, rb, rkvh, token);
    }
    // where the next list begins: one unit after the last of this one
    at = Place{from_lane(rb, count - 1), from_lane(rband, count - 1), from_lane(rtile, count - 1) + 1,
               from_lane(rlen, count - 1)};
    left -= count;
    if (left > 0 && at.tile > tiles_of(a, at.len)) next_row();
    auto load = [&](Tile<D, FP8> &t, int i) {
      const int64_t line[2] = {from_lane(rline[0], i), from_lane(rline[1], i)};
      load_tile<D, FP8>(t, a, line, n, g);
    };
    for (int i = 0; i < count; i++) {
      const int token = from_lane(rtoken, i), len = from_lane(rlen, i), tiles = tiles_of(a, len);
      if (from_lane(rtile, i) == tiles) continue;  // a row's end
      if (fresh) {
        load_queries<D, FP8, RT>(qf, a, Row(a, from_lane(rb, i), from_lane(rband, i), RT), n, g);
        clear_state(st);
        fresh = false;
      }
      Tile<D, FP8> now;
      load(now, i);
      use_tile<D, FP8, RT>(now, a, qf, st, token, a.window > 0 ? max(0, len - a.window) : 0, len, g);
      const bool row_ends = token + kTile >= len, share_ends = i + 1 == count && left == 0;
      if (row_ends || share_ends) {
        const int b = from_lane(rb, i), band = from_lane(rband, i);
        const bool whole = row_begin == 0 && row_ends;
        const int slot = 2 * self + (started ? 0 : 1);
        const Row row(a, b, band, RT);
#pragma unroll
        for (int r = 0; r < RT; r++) {
          const int head = 16 * r + n;
          float l = st[r].l;
          l += __shfl_xor(l, 16, 64);
          l += __shfl_xor(l, 32, 64);
          if (head >= row.heads) continue;
          // this lane holds values D / 4 g .. + D / 4 - 1 of its head
          if (whole) {
            const float inv = l == 0.f ? 0.f : 1.f / l;
            uint16_t *dst = a.o + (row.q0 + head) * D + D / 4 * g;
#pragma unroll
            for (int e = 0; e < D / 4; e += 8) {
              float v[8];
#pragma unroll
              for (int k = 0; k < 8; k++) v[k] = st[r].o[(e + k) % (D / 16)][(e + k) / (D / 16)] * inv;
              *reinterpret_cast<uint4 *>(dst + e) = pack8(v);
            }
            if (a.lse && g == 0) a.lse[row.q0 + head] = l == 0.f ? -INFINITY : kLn2 * (st[r].m + log2f(l));
          } else {
            float *base = part + slot * part_floats(D, RT), *dst = base + head * D + D / 4 * g;
#pragma unroll
            for (int e = 0; e < D / 4; e += 4) {
              float v[4];
#pragma unroll
              for (int k = 0; k < 4; k++) v[k] = st[r].o[(e + k) % (D / 16)][(e + k) / (D / 16)];
              *reinterpret_cast<float4 *>(dst + e) = make_float4(v[0], v[1], v[2], v[3]);
            }
            if (g == 0) {
              base[16 * RT * D + head] = st[r].m;
              base[16 * RT * (D + 1) + head] = l;
            }
          }
        }
        if (lane == 0 && row_begin == 0 && (plan.by_row || !whole)) {
          cuts[plan.by_row ? (int64_t)b * rows + band : (int64_t)self] =
              Cut{total, row_position + tiles, b, band, whole ? -1 : slot, 0, self, 0};
        }
        fresh = true;
        started = false;
        row_begin = 0;
        row_position += tiles + 1;
      }
    }
  }
}

// A row's tiles divided by the grid: workgroup `split` of a row takes tiles per split
// .. per split + per - 1, its waves every WAVES-th of them, and the waves' states
// are added through LDS, in a fixed order.
template <int D, bool FP8, int RT, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void row_kernel(DecodeArgs a, DecodePlan plan, float *part, Cut *cuts) {
  constexpr int kPad = RowBoxOf<D>::kHead;
  extern __shared__ __align__(16) float lds[];
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6), n = lane & 15, g = lane >> 4;
  const int group = a.Hq / a.Hkv, rows = a.Hkv * ((group + 16 * RT - 1) / (16 * RT));
  int row_at = (int)blockIdx.x / plan.splits;
  const int split = (int)blockIdx.x - row_at * plan.splits;
  row_at += plan.first_row;
  const int b = row_at / rows, band = row_at - b * rows;
  const Row row(a, b, band, RT);
  const RowBox box = RowBoxOf<D>::at(WAVES, row.heads);
  float *box_o = lds + box.o, *box_m = lds + box.m, *box_l = lds + box.l;
  v8bf qf[RT][D / 32];
  load_queries<D, FP8, RT>(qf, a, row, n, g);
  // Lane x looks up half tile x % 2 of the wave's tile x / 2; without a window
  // before the length is known (which takes as long).
  const int64_t begin = split * plan.per;
  const int64_t mine = kTile * (begin + wave + WAVES * (lane >> 1)) + 16 * (lane & 1);
  int64_t found = 0;
  if (a.window == 0 && mine < a.max_len) found = line_of(a, b, row.kvh, (int)mine);
  const int len = uniform(length_of(a, b)), first = first_token(len, a.window), tiles = tiles_of(a, len);
  if (begin >= tiles) return;
  const int end = (int)min((int64_t)tiles, begin + plan.per);
  if (a.window > 0 && first + mine < len) found = line_of(a, b, row.kvh, (int)(first + mine));
  State<D> st[RT];
  clear_state(st);
  for (int i = (int)begin + wave, x = 0; i < end && len > 0; i += WAVES, x++) {
    const int token = first + kTile * i;
    if (x == 32) {  // the next 32 tiles
      x = 0;
      const int ahead = token + kTile * WAVES * (lane >> 1) + 16 * (lane & 1);
      found = ahead < len ? line_of(a, b, row.kvh, ahead) : 0;
    }
    // a half tile past the end counts for nothing: any line will do
    const int64_t line[2] = {from_lane(found, 2 * x), token + 16 < len ? from_lane(found, 2 * x + 1) : 0};
    Tile<D, FP8> t;
    load_tile<D, FP8>(t, a, line, n, g);
    use_tile<D, FP8, RT>(t, a, qf, st, token, a.window > 0 ? max(0, len - a.window) : 0, len, g);
  }
#pragma unroll
  for (int r = 0; r < RT; r++) {
    const int head = 16 * r + n;
    float l = st[r].l;
    l += __shfl_xor(l, 16, 64);
    l += __shfl_xor(l, 32, 64);
    if (head >= row.heads) continue;
    float *dst = box_o + (wave * row.heads + head) * kPad + D / 4 * g;
#pragma unroll
    for (int e = 0; e < D / 4; e += 4) {
      float v[4];
#pragma unroll
      for (int k = 0; k < 4; k++) v[k] = st[r].o[(e + k) % (D / 16)][(e + k) / (D / 16)];
      *reinterpret_cast<float4 *>(dst + e) = make_float4(v[0], v[1], v[2], v[3]);
    }
    if (g == 0) {
      box_m[wave * row.heads + head] = st[r].m;
      box_l[wave * row.heads + head] = l;
    }
  }
  __syncthreads();
  const bool whole = begin == 0 && end == tiles;
  float *base = part + 2 * (size_t)blockIdx.x * part_floats(D, RT);
  for (int c = threadIdx.x; c < row.heads * (D / 4); c += 64 * WAVES) {
    const int head = c / (D / 4), d = c % (D / 4) * 4;
    float top = -INFINITY, l = 0.f, o[4] = {};
#pragma unroll
    for (int w = 0; w < WAVES; w++) top = fmaxf(top, box_m[w * row.heads + head]);
#pragma unroll
    for (int w = 0; w < WAVES; w++) {
      const float m = box_m[w * row.heads + head], f = m == top ? 1.f : __builtin_amdgcn_exp2f(m - top);
      const float4 x = *reinterpret_cast<const float4 *>(box_o + (w * row.heads + head) * kPad + d);
      l += box_l[w * row.heads + head] * f;
      o[0] += x.x * f;
      o[1] += x.y * f;
      o[2] += x.z * f;
      o[3] += x.w * f;
    }
    if (whole) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
      *reinterpret_cast<uint2 *>(a.o + (row.q0 + head) * D + d) =
          make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
      if (a.lse && d == 0) a.lse[row.q0 + head] = l == 0.f ? -INFINITY : kLn2 * (top + log2f(l));
    } else {
      *reinterpret_cast<float4 *>(base + head * D + d) = make_float4(o[0], o[1], o[2], o[3]);
      if (d == 0) {
        base[16 * RT * D + head] = top;
        base[16 * RT * (D + 1) + head] = l;
      }
    }
  }
  if (plan.splits > 1 && split == 0 && threadIdx.x == 0)
    cuts[row_at] = Cut{0, 0, b, band, whole ? -1 : 2 * (int)blockIdx.x, (int)((tiles + plan.per - 1) / plan.per),
                       (int)blockIdx.x, 0};
}

// Joins the parts of divided rows, in a fixed order.  Workgroup (i, y) takes row i
// of the list and HEADS of its query heads.  Where the row has few parts each wave
// joins one head alone, else all waves share the parts of one head after the
// other, through LDS.  Eight parts are in flight at a time, under a running
// maximum; a part weighs 2^(m - top).
template <int D, int RT, int WAVES, int HEADS>
__global__ __launch_bounds__(64 * WAVES) void join_kernel(DecodeArgs a, int log2_parts, const float *part,
                                                          const Cut *cuts) {
  constexpr int E = D / 64;
  __shared__ float wave_top[WAVES], wave_l[WAVES], wave_o[WAVES][D];
  const Cut cut = cuts[blockIdx.x];
  if (cut.slot < 0) return;
  const int lane = threadIdx.x & 63, wave = uniform(threadIdx.x >> 6);
  const int group = a.Hq / a.Hkv, bands = (group + 16 * RT - 1) / (16 * RT);
  const int kvh = cut.band / bands, band_head = (cut.band - kvh * bands) * 16 * RT;
  const int heads = min(group - band_head, 16 * RT);
  int parts = cut.parts;
  if (parts == 0) {
    // shares from the owner's on that start before the row's end
    int low = 1, high = (1 << log2_parts) - cut.owner;
    while (low < high) {
      const int mid = (low + high) / 2;
      if (share_start((int64_t)cut.owner + mid, cut.total, log2_parts) < cut.row_end)
        low = mid + 1;
      else
        high = mid;
    }
    parts = low;
  }
  const bool alone = HEADS > 1 && parts <= 24;
  const int step = alone ? 1 : WAVES, head_end = min(heads, (int)(blockIdx.y + 1) * HEADS);
  for (int head = blockIdx.y * HEADS + (alone ? wave : 0); head < head_end; head += alone ? WAVES : 1) {
    float top = -INFINITY, l = 0.f, o[E] = {};
    for (int k0 = alone ? 0 : wave; k0 < parts; k0 += 8 * step) {
      float m[8], lp[8], op[8][E];
#pragma unroll
      for (int u = 0; u < 8; u++) {
        const int k = min(k0 + step * u, parts - 1);
        const float *p = part + (size_t)(k == 0 ? cut.slot : 2 * (cut.owner + k)) * part_floats(D, RT);
        m[u] = p[16 * RT * D + head];
        lp[u] = p[16 * RT * (D + 1) + head];
#pragma unroll
        for (int e = 0; e < E; e++) op[u][e] = p[head * D + E * lane + e];
      }
      float high = top;
#pragma unroll
      for (int u = 0; u < 8; u++) high = fmaxf(high, m[u]);
      const float shrink = top == high ? 1.f : __builtin_amdgcn_exp2f(top - high);
      top = high;
      l *= shrink;
#pragma unroll
      for (int e = 0; e < E; e++) o[e] *= shrink;
#pragma unroll
      for (int u = 0; u < 8; u++) {
        if (k0 + step * u < parts) {
          const float f = m[u] == top ? 1.f : __builtin_amdgcn_exp2f(m[u] - top);
          l += lp[u] * f;
#pragma unroll
          for (int e = 0; e < E; e++) o[e] += op[u][e] * f;
        }
      }
    }
    const int64_t at = (int64_t)cut.b * a.Hq + kvh * group + band_head + head;
    if (alone) {
      const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
      for (int e = 0; e < E; e++) a.o[at * D + E * lane + e] = (uint16_t)f32_to_bf16_rne(o[e] * inv);
      if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : kLn2 * (top + log2f(l));
      continue;
    }
    __syncthreads();  // the boxes are free
    if (lane == 0) {
      wave_top[wave] = top;
      wave_l[wave] = l;
    }
#pragma unroll
    for (int e = 0; e < E; e++) wave_o[wave][E * lane + e] = o[e];
    __syncthreads();
    for (int d = threadIdx.x; d < D; d += 64 * WAVES) {
      float high = -INFINITY, sum = 0.f, weight = 0.f;
#pragma unroll
      for (int w = 0; w < WAVES; w++) high = fmaxf(high, wave_top[w]);
#pragma unroll
      for (int w = 0; w < WAVES; w++) {
        const float f = wave_top[w] == high ? 1.f : __builtin_amdgcn_exp2f(wave_top[w] - high);
        weight += wave_l[w] * f;
        sum += wave_o[w][d] * f;
      }
      a.o[at * D + d] = (uint16_t)f32_to_bf16_rne(weight == 0.f ? 0.f : sum / weight);
      if (a.lse && d == 0) a.lse[at] = weight == 0.f ? -INFINITY : kLn2 * (high + log2f(weight));
    }
  }
}

template <int D, bool FP8, int RT, int WAVES>
hipError_t launch_row(const DecodeArgs &a, const DecodePlan &p, float *part, Cut *cuts, hipStream_t stream) {
  const int group = a.Hq / a.Hkv, heads = group < 16 * RT ? group : 16 * RT;
  const size_t lds = (size_t)RowBoxOf<D>::at(WAVES, heads).floats * sizeof(float);
  auto *kernel = row_kernel<D, FP8, RT, WAVES>;
  if (lds > 65536) {
    const hipError_t e = hipFuncSetAttribute(reinterpret_cast<const void *>(kernel),
                                             hipFuncAttributeMaxDynamicSharedMemorySize, (int)lds);
    if (e != hipSuccess) return e;
  }
  DecodePlan q = p;  // more rows than a grid takes (never divided ones) go in several launches
  for (; p.owners - q.first_row > kRowGrid; q.first_row += kRowGrid)
    hipLaunchKernelGGL(kernel, dim3((unsigned)kRowGrid), dim3(64 * WAVES), lds, stream, a, q, part, cuts);
  hipLaunchKernelGGL(kernel, dim3((unsigned)(p.owners - q.first_row)), dim3(64 * WAVES), lds, stream, a, q, part, cuts);
  return hipSuccess;
}

template <int D, bool FP8, int RT>
hipError_t launch_decode(const DecodeArgs &a, const DecodePlan &p, float *part, hipStream_t stream) {
  Cut *cuts = reinterpret_cast<Cut *>(part + 2 * (size_t)p.owners * part_floats(D, RT));
  hipError_t e = hipErrorInvalidValue;  // a form that is not built
  if (p.row_waves == 0) {
    hipLaunchKernelGGL((decode_kernel<D, FP8, RT>), dim3((unsigned)((p.owners + kWaves - 1) / kWaves)), dim3(kThreads),
                       0, stream, a, p, part, cuts);
    e = hipSuccess;
  }
  if constexpr (has_row_form(D, RT, 1)) {
    if (p.row_waves == 1) e = launch_row<D, FP8, RT, 1>(a, p, part, cuts, stream);
  }
  if (p.row_waves == 2) e = launch_row<D, FP8, RT, 2>(a, p, part, cuts, stream);
  if (p.row_waves == 4) e = launch_row<D, FP8, RT, 4>(a, p, part, cuts, stream);
  if constexpr (has_row_form(D, RT, 8)) {
    if (p.row_waves == 8) e = launch_row<D, FP8, RT, 8>(a, p, part, cuts, stream);
  }
  if (e != hipSuccess) return e;
  if (!p.row_waves || p.splits > 1) {
    const int group = a.Hq / a.Hkv, heads = group < 16 * RT ? group : 16 * RT;
    const unsigned listed = (unsigned)(p.by_row ? p.rows : p.owners);
    // many (row, head) pairs: four heads a workgroup (2048 pairs of 5 parts: 8.1 us with a workgroup for each, 5.1
    // so); few: one, with more waves where a row has many parts (32 pairs of 25 parts: 8.3 us with four, 3.6 so)
    if (p.rows * heads > 1024)
      hipLaunchKernelGGL((join_kernel<D, RT, 4, 4>), dim3(listed, (unsigned)((heads + 3) / 4)), dim3(256), 0, stream, a,
                         p.log2_parts, (const float *)part, (const Cut *)cuts);
    else if (p.rows * 64 > p.owners)
      hipLaunchKernelGGL((join_kernel<D, RT, 4, 1>), dim3(listed, (unsigned)heads), dim3(256), 0, stream, a,
                         p.log2_parts, (const float *)part, (const Cut *)cuts);
    else
      hipLaunchKernelGGL((join_kernel<D, RT, 16, 1>), dim3(listed, (unsigned)heads), dim3(1024), 0, stream, a,
                         p.log2_parts, (const float *)part, (const Cut *)cuts);
  }
  return hipGetLastError();
}

template <int D, bool FP8>
hipError_t launch_rows(const DecodeArgs &a, const DecodePlan &p, float *part, hipStream_t stream) {
  if constexpr (D < 256) {
    if (row_tiles(a) == 2) return launch_decode<D, FP8, 2>(a, p, part, stream);
  }
  return launch_decode<D, FP8, 1>(a, p, part, stream);
}

template <int D>
hipError_t launch_dim(const DecodeArgs &a, const DecodePlan &p, float *part, hipStream_t stream) {
  return a.k_scale ? launch_rows<D, true>(a, p, part, stream) : launch_rows<D, false>(a, p, part, stream);
}

}  // namespace

size_t paged_decode_partial_bytes(const DecodeArgs &a, int cus) {
  const DecodePlan p = plan_decode(a, cus);
  if (p.row_waves && p.splits == 1) return 0;
  return 2 * (size_t)p.owners * part_floats(a.D, row_tiles(a)) * sizeof(float) +
         (size_t)(p.by_row ? p.rows : p.owners) * sizeof(Cut);
}

hipError_t launch_paged_decode(const DecodeArgs &a, float *part, hipStream_t stream) {
  const DecodePlan p = plan_decode(a, device_cu_count());
  if (a.D == 64) return launch_dim<64>(a, p, part, stream);
  if (a.D == 128) return launch_dim<128>(a, p, part, stream);
  return launch_dim<256>(a, p, part, stream);
}

}  // namespace fp8lin
