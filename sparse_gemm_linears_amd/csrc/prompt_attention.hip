// Attention of several tokens of each sequence: of packed prompts over their own keys, or
// of the last tokens of each sequence over a paged key-value cache.
//
// For query head n of a token at place p of its sequence, over the keys t that it sees
// (t <= p where causal, the last `window` of them, or all): score_t = scale q.k_t, capped as
// c tanh(score / c) when a cap is given, o = sum_t softmax(score)_t v_t and
// lse = log sum_t exp(score_t), in one pass with a running maximum and sum.
//
// Bound: the matrix rate for long chunks (4 D flops for each query head and key against
// 4 D bytes for each key head and key of a whole block of rows), the cache's bytes for
// chunks of a few tokens.  The query heads of a key head share its keys: a row is a token
// and one of these heads (row = token * group + head), so that a block of rows reads each
// key once for all of them and a short chunk still fills a wave's rows.
//
// A workgroup of four waves takes a block of up to 128 rows of one sequence and key head and goes
// over the keys that some row of it sees, in tiles of 64 (32 for D = 256) that are copied to LDS
// past the registers while the tile before is used, two buffers each.  How the waves share a
// tile depends on the block's rows:
//   more than 64   a wave holds 32 rows and takes all keys of a tile;
//   33 to 64       two waves hold the same 32 rows and take half of a tile's keys each;
//   at most 32 (a short sequence over a cache)   as many waves as LDS has tiles for (four over e4m3
//                  heads of 64 and 128, two over bf16 ones and e4m3 heads of 256) hold the rows, and
//                  each goes over tiles of 32 keys of its own without a barrier, codes
//                  converted as they are read: such blocks wait for the cache alone.  The other
//                  waves have no work.
// 256-wide heads know the first form, and over e4m3 the last: of up to 32 rows over a bf16 cache one wave
// computes and all four copy.
// Waves with the same rows add their states up through LDS at the end.
//
// Layouts (v_mfma_f32_32x32x16_bf16: lane l, n = l % 32, h = l / 32):
//   scores   A = K: row n is key n, B = Q: column n is a row; lane half h holds values
//            16 s + 8 h .. + 7 of step s;
//   weights  the scores come out with column n = row and register i = key
//            8 (i / 4) + 4 h + i % 4: a row's maximum and sum stay in two lanes, and registers
//            8 s .. 8 s + 7 are the B operand of the second product's step s if its 16
//            keys are counted in that order;
//   values   A = V transposed, read from LDS by ds_read_b64_tr_b16 (16 lanes take 4 keys
//            of 16 values; lane i gets value i of the four).
// The weights enter the second product as one bf16 each (2^-8 of a weight at most): for values of
// either sign that adds about as much to o as its own rounding does, over few keys or many.
// Sums of weights are of the fp32 values.  A second product for the low halves takes a third of
// the matrix rate of large blocks; small ones have the rate, but not the time for the halves
// (in us, as it is and with them: 32 sequences of 5 to 8192 tokens, 4 new ones each, e4m3, 56.1
// and 58.7, heads of 64 41.1 and 44.0, of 256 156 and 165; 256 single tokens 200 and 217).
// paged_decode_attention has them.  The reference of a row's exponents moves only when a score passes
// it by 2^8, so that most tiles need no exchange between lanes and no correction of o.
//
// LDS rows are whole lines of a head; 16-byte chunks of a row are permuted by key_swizzle
// and value_swizzle so that 16 rows of one column of K, and 8 rows of four columns
// of V, lie in different banks (no conflict counted over 8192 tokens).
//
// Measured (32 / 8 heads of 128): a prompt of 8192 tokens 537 to 567 us, 1.0 PFLOP/s, as the clock
// allows (one bf16 product of 8192^3 reaches 1.25 to 1.36); 2048 tokens over 32768 1040 to
// 1100 us, 1.0 PFLOP/s (e4m3 1594 us, 0.67).  The matrix units are busy half of the time there, the
// vector units 0.47 of it (exponentials, maxima, packing), two workgroups to a compute unit so that one's exponentials
// overlap the other's products.  Level or slower at the long prompt: the next tile's scores
// between the exponentials of this one (583 us against 537), three waves a SIMD with tiles of 32 keys (578 against
// 565), blocks of 64 rows (676 against 566), blocks of 256 whose two halves take turns at products and
// exponentials (580 against 569), wave priorities.  Few rows: 32 sequences of 5 to
// 8192 tokens, 4 new ones each, e4m3, 190 MB in 55 to 58 us: 3.4 TB/s, the start of a part (5 us) and the
// join (7 us) included.  Heads of 256 reach 0.94 to 1.0 PFLOP/s over 8192 tokens, of 64 0.75 to 0.87: half
// the products for as many exponentials.
//
// Registers: the forms of 256-wide heads have all 256 in use and spill, 66 to 71 vector registers over an
// e4m3 cache (124 to 152 bytes a lane), 2 to 4 over a bf16 one and for capped rows.  The e4m3 forms of
// 64 and 128 keep 183 to 205 scalar registers in lanes of vector ones.
#include <cmath>
#include <type_traits>

#include "device_common.hpp"
#include "gemm_common.hpp"
#include "launch.hpp"
#include "launch_layer.hpp"
#include "prompt_plan.hpp"

namespace fp8lin {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kLarge = 0x1p26f;  // of exponents, see weigh

typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef uint32_t v4u __attribute__((ext_vector_type(4)));
typedef short v4s __attribute__((ext_vector_type(4)));
typedef int v2i __attribute__((ext_vector_type(2)));
typedef __attribute__((address_space(3))) v4s lds_v4s;
typedef __attribute__((address_space(3))) v2i lds_v2i;

__device__ __forceinline__ v8bf as_bf16x8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  return __builtin_bit_cast(v8bf, (v4u{a, b, c, d}));
}
__device__ __forceinline__ int uniform(int x) { return __builtin_amdgcn_readfirstlane(x); }
__device__ __forceinline__ int from_lane(int x, int lane) { return __builtin_amdgcn_readlane(x, lane); }
__device__ __forceinline__ int64_t from_lane(int64_t x, int lane) {
  return (int64_t)(uint32_t)from_lane((int)x, lane) | (int64_t)from_lane((int)(x >> 32), lane) << 32;
}

#define FP8LIN_INLINE __attribute__((always_inline))

// The same address, which stays on the scalar side: lanes add 32-bit offsets to it.
__device__ __forceinline__ const char *scalar(const char *p) {
  uint64_t x = reinterpret_cast<uint64_t>(p);
  asm volatile("" : "+s"(x));
  return reinterpret_cast<const char *>(x);
}

// The same value, of which the compiler knows nothing: what is computed from it in a path that is
// rarely taken is not computed ahead of the loop, where it would hold registers.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// a * b, rounded by itself.
__device__ __forceinline__ float product(float a, float b) {
#pragma clang fp contract(off)
  return a * b;
}

// Neither loads nor anything else is moved past this place.
__device__ __forceinline__ void step_ends() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_sched_barrier(0);
}

// A barrier for LDS alone: unlike __syncthreads it does not wait for the copies under way.
__device__ __forceinline__ void lds_barrier() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); }

// Two e4m3 codes (the low or the high half of w) as packed bf16, exactly.
template <bool HIGH>
__device__ __forceinline__ uint32_t e4m3x2_to_bf16(uint32_t w) {
  return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HIGH));
}

enum class Source { kRows, kCache, kCodes };  // strided bf16 rows, a bf16 cache, an e4m3 cache

// Position of 16-byte chunk c of row r in an LDS row of D values.
template <int D>
__device__ __forceinline__ int key_swizzle(int r, int c) {
  return c ^ (D == 64 ? (r >> 1) & 7 : r & 15);
}
template <int D>
__device__ __forceinline__ int value_swizzle(int r, int c) {
  return c ^ (D == 64 ? (r >> 1 & 1) << 2 : (r & 3) << 2);
}

// A block of rows: rows row0 .. row0 + block rows - 1 of the `rows` of sequence b, whose
// first token is `start`; tokens first .. last of it.
struct Block {
  int b, start, tokens, keys, row0, rows;
  int begin, end;  // keys that some row of the block sees (begin rounded down to 16)
  int lowest;      // the first of them
  int place0;      // place of the sequence's first token among the keys
  int tiles;
};

__device__ __forceinline__ int start_of(const PromptArgs &a, int b) { return min(max(a.starts[b], 0), a.T); }

// The rest of block k, whose sequence is known.
__device__ __forceinline__ void fill_block(const PromptArgs &a, int row0, int tile, Block &k) {
  const int group = a.Hq / a.Hkv;
  k.row0 = uniform(row0);
  k.rows = k.tokens * group;
  const int first = k.row0 / group, last = min(k.row0 + kBlockRows, k.rows) - 1;
  k.place0 = k.keys - k.tokens;
  k.end = a.causal ? max(0, k.place0 + last / group + 1) : k.keys;
  k.lowest = a.window > 0 ? max(0, k.place0 + first - a.window + 1) : 0;
  k.begin = k.lowest & ~15;
  k.tiles = (max(0, k.end - k.begin) + tile - 1) / tile;
}

// Of two bf16 values, the top bit of each that is an infinity or a NaN.
__device__ __forceinline__ uint32_t not_finite(uint32_t w) {
  return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u;
}

// Finds block `number` of the batch; false if the number is not used.
__device__ __forceinline__ bool find_block(const PromptArgs &a, int64_t number, int tile, Block &k) {
  const int lane = threadIdx.x & 63, group = a.Hq / a.Hkv;
  // The last sequence whose numbers start at `number` or before, 64 candidates at a time; each
  // lane reads all that its candidate needs at once, so that one read follows the other only
  // where there are more than 64 sequences.
  int low = 0, high = a.B;
  for (;;) {
    const int step = (high - low + 63) / 64, b = low + lane * step, at = min(b, a.B - 1);
    const int start = start_of(a, at), next = start_of(a, at + 1);
    const int length = a.block_table ? min(max(a.seq_lens[at], 0), a.max_len) : 0;
    const int count = __popcll(__ballot(b < high && first_block(start, b, group) <= number));
    if (count == 0) return false;
    if (step == 1) {
      k.b = uniform(low + count - 1);
      k.start = from_lane(start, count - 1);
      k.tokens = from_lane(next, count - 1) - k.start;
      k.keys = a.block_table ? from_lane(length, count - 1) : k.tokens;
      break;
    }
    low = uniform(low + (count - 1) * step);
    high = min(high, low + step);
  }
  const int64_t row0 = (number - first_block(k.start, k.b, group)) * kBlockRows;
  if (k.tokens <= 0 || row0 < 0 || row0 >= (int64_t)k.tokens * group) return false;
  fill_block(a, (int)row0, tile, k);
  return true;
}

// Sum over the wave's 64 lanes, in every lane.
__device__ __forceinline__ int wave_sum(int v) {
  v += __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, false);   // quad_perm 1,0,3,2
  v += __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, false);   // quad_perm 2,3,0,1
  v += __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, false);  // half mirror
  v += __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, false);  // mirror
  return from_lane(v, 0) + from_lane(v, 16) + from_lane(v, 32) + from_lane(v, 48);
}

// Largest over the wave's 64 lanes of values that are not negative, in every lane.
__device__ __forceinline__ int wave_max(int v) {
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0xB1, 0xF, 0xF, false));   // quad_perm 1,0,3,2
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x4E, 0xF, 0xF, false));   // quad_perm 2,3,0,1
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x141, 0xF, 0xF, false));  // half mirror
  v = max(v, __builtin_amdgcn_update_dpp(0, v, 0x140, 0xF, 0xF, false));  // mirror
  return max(max(from_lane(v, 0), from_lane(v, 16)), max(from_lane(v, 32), from_lane(v, 48)));
}

// The block at `rank` of up to 64 prompts' blocks in falling order of their place in their
// prompt: the ones with the most keys begin first, and the short ones fill the end.  (Seven
// prompts of 131 to 1357 tokens of 28 heads of 64: 36 us with one prompt after the
// other, 34 so; of 32 heads of 128 63 and 59.)
__device__ __forceinline__ bool find_ranked(const PromptArgs &a, int rank, int tile, Block &k) {
  const int lane = threadIdx.x & 63, group = a.Hq / a.Hkv, at = min(lane, a.B - 1);
  const int start = start_of(a, at), tokens = start_of(a, at + 1) - start;
  const int blocks = lane < a.B && tokens > 0 ? (int)(((int64_t)tokens * group + kBlockRows - 1) / kBlockRows) : 0;
  const int total = wave_sum(blocks);
  if (rank >= total) return false;
  int place = 0;  // the largest with more than `rank` blocks at it or behind it
  for (int bit = 1 << (31 - __builtin_clz(total)); bit > 0; bit >>= 1)
    if (wave_sum(max(blocks - (place + bit), 0)) > rank) place += bit;
  const int which = rank - wave_sum(max(blocks - (place + 1), 0));  // of the sequences that have it
  const uint64_t have = __ballot(blocks > place);
  const int before = __popcll(have & ((1ull << lane) - 1));
  const int from = __ffsll((unsigned long long)__ballot(blocks > place && before == which)) - 1;
  k.b = from;
  k.start = from_lane(start, from);
  k.tokens = k.keys = from_lane(tokens, from);
  fill_block(a, place * kBlockRows, tile, k);
  return true;
}

// A workgroup's part of a block.
struct Part {
  int per;       // tiles of a part of its block
  int split;     // which one it is
  int splits;    // the most that there are
  int64_t slot;  // place of the block's first part among the partials, and steps to the next one
  int step;
};

// The part at `rank` of a key head's, where long sequences are divided most: into as many
// parts as keep every one's cost below the least bound for which all parts are at most
// plan.shares.  A tile of a block of at most 32 rows counts as two thirds of another one in e4m3
// (which waits for the cache), and one and a half times as much in bf16 (measured with heads of 128).
template <bool CODES>
__device__ __forceinline__ bool find_share(const PromptArgs &a, const PromptPlan &plan, int rank, int kvh, int tile,
                                           Block &k, Part &part) {
  constexpr int kEach = kShareBatch / 64, kMost = 4096;  // (a valid batch has fewer blocks and parts)
  const int lane = threadIdx.x & 63, group = a.Hq / a.Hkv, each = (a.B + 63) / 64;
  int start[kEach], tokens[kEach], keys[kEach], blocks[kEach], cost[kEach];
#pragma unroll
  for (int j = 0; j < kEach; j++) {
    const int b = lane * each + j, at = min(b, a.B - 1);
    start[j] = tokens[j] = keys[j] = blocks[j] = cost[j] = 0;
    if (j >= each) continue;
    start[j] = start_of(a, at);
    tokens[j] = start_of(a, at + 1) - start[j];
    keys[j] = min(max(a.seq_lens[at], 0), a.max_len);
    if (b >= a.B || tokens[j] <= 0) continue;
    const int64_t rows = (int64_t)tokens[j] * group;
    blocks[j] = (int)((rows + kBlockRows - 1) / kBlockRows);
    const int seen = a.window > 0 ? min(keys[j], a.window + (kBlockRows + group - 1) / group + 15) : keys[j];
    cost[j] = (seen + tile - 1) / tile * ((rows <= kWaveRows) == CODES ? 2 : 3);
  }
  auto parts_of = [&](int j, float inverse) FP8LIN_INLINE {
    return min(max((int)__builtin_ceilf((float)cost[j] * inverse), 1), kMost);
  };
  auto count_of = [&](int j, float inverse) FP8LIN_INLINE {
    return min(min(blocks[j], kMost) * parts_of(j, inverse), 1 << 20);
  };
  auto large = [&](int j) FP8LIN_INLINE { return tokens[j] * (int64_t)group > kWaveRows; };
  auto mine_of = [&](float inverse, bool larges, bool others) FP8LIN_INLINE {
    int mine = 0;
#pragma unroll
    for (int j = 0; j < kEach; j++)
      if (j < each && (large(j) ? larges : others)) mine += count_of(j, inverse);
    return mine;
  };
  int most = 0;
#pragma unroll
  for (int j = 0; j < kEach; j++) most = max(most, cost[j]);
  most = wave_max(most);
  // Two tiles at least, and as much as makes joining the longest sequence's parts (0.25 us each)
  // cost no more than going over them does.
  int bound = max(6, (int)__builtin_amdgcn_sqrtf((float)most)) - 1;  // the largest that is too small, or is not tried
  auto too_many = [&](int x) FP8LIN_INLINE {
    return wave_sum(mine_of(__builtin_amdgcn_rcpf((float)x), true, true)) > plan.shares;
  };
  if (too_many(bound + 1)) {
    for (int bit = 1 << (31 - __builtin_clz(most | 1)); bit > 0; bit >>= 1)
      if (too_many(bound + bit)) bound += bit;
  }
  const float inverse = __builtin_amdgcn_rcpf((float)(bound + 1));
  const int mine_large = mine_of(inverse, true, false), all_large = wave_sum(mine_large);
  const bool takes_large = rank < all_large;  // the blocks that take longest begin first
  const int mine = takes_large ? mine_large : mine_of(inverse, false, true);
  int before = mine;  // and of the lanes below
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int other = __shfl_up(before, d, 64);
    if (lane >= d) before += other;
  }
  const int place = takes_large ? rank : rank - all_large;
  const uint64_t behind = __ballot(before > place);
  if (behind == 0) return false;
  const int from = __ffsll((unsigned long long)behind) - 1;
  int index = place - (from_lane(before, from) - from_lane(mine, from)), splits = 0, all = 0;
#pragma unroll
  for (int j = 0; j < kEach; j++) {
    const int count = from_lane(large(j) == takes_large ? count_of(j, inverse) : 0, from);
    if (j < each && splits == 0) {
      if (index < count) {
        k.b = from * each + j;
        k.start = from_lane(start[j], from);
        k.tokens = from_lane(tokens[j], from);
        k.keys = from_lane(keys[j], from);
        splits = from_lane(parts_of(j, inverse), from);
        all = from_lane(blocks[j], from);
      } else {
        index -= count;
      }
    }
  }
  const int behind_it = index / splits;  // blocks of the sequence: the last ones see the most keys
  if (behind_it >= all) return false;
  fill_block(a, (all - 1 - behind_it) * kBlockRows, tile, k);
  part.split = index - behind_it * splits;
  part.splits = splits;
  part.per = max(1, (k.tiles + splits - 1) / splits);
  part.slot = (int64_t)(rank - part.split) * a.Hkv + kvh;
  part.step = a.Hkv;
  // The block's parts have slots rank - split .. rank - split + splits - 1 (split <= index <= rank): all of
  // them lie in the partials' memory.  (Starts that are out of order may make more.)
  return rank - part.split + splits <= plan.shares;
}

// tanh of each value.  tanh z = 1 - 2 / (1 + exp 2z), but below 1/4, where that would lose a
// small score's low bits, its power series (2^-26 of it is left out).
template <int N>
__device__ __forceinline__ void tanh_each(float (&z)[N]) {
  float most = 0.f;
#pragma unroll
  for (int j = 0; j < N; j++) most = fmaxf(most, fabsf(z[j]));
  // (a NaN stays one on either way)
  if (__any(most >= 0.25f)) {
#pragma unroll
    for (int j = 0; j < N; j++) {
      const float w = fabsf(z[j]), u = z[j] * z[j], e = __builtin_amdgcn_exp2f(2.f * kLog2e * w);
      float t = __builtin_fmaf(u, 62.f / 2835.f, -17.f / 315.f);
      t = __builtin_fmaf(u, t, 2.f / 15.f);
      t = __builtin_fmaf(u, t, -1.f / 3.f);
      t = __builtin_fmaf(z[j] * u, t, z[j]);
      z[j] = w >= 0.25f ? copysignf(1.f - 2.f * __builtin_amdgcn_rcpf(1.f + e), z[j]) : t;
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; j++) {
      const float u = z[j] * z[j];
      float t = __builtin_fmaf(u, 62.f / 2835.f, -17.f / 315.f);
      t = __builtin_fmaf(u, t, 2.f / 15.f);
      t = __builtin_fmaf(u, t, -1.f / 3.f);
      z[j] = __builtin_fmaf(z[j] * u, t, z[j]);
    }
  }
}

template <int D, Source SRC, bool CAP>
__global__ __launch_bounds__(64 * kBlockWaves, 2) void prompt_kernel(PromptArgs a, PromptPlan plan, float *part) {
  constexpr bool kPaged = SRC != Source::kRows, kFp8 = SRC == Source::kCodes;
  constexpr int KT = tile_keys(D), WAVES = kBlockWaves, kRow = 2 * D;  // bytes of an LDS row
  __shared__ __align__(1024) uint8_t lds_k0[KT * kRow], lds_k1[KT * kRow], lds_v0[KT * kRow], lds_v1[KT * kRow];
  constexpr int kBytes = kFp8 ? 1 : 2, kLine = D * kBytes;  // of a value and a cache line in memory
  // waves of a block of at most 32 rows that work, each on tiles of 32 keys of its own
  constexpr int kFewTile = 32 * kLine, kFewWaves = KT * kRow / kFewTile < WAVES ? KT * kRow / kFewTile : WAVES;
  __shared__ __align__(16) float lds_s0[kFp8 ? 64 * WAVES : 1], lds_s1[kFp8 ? 64 * WAVES : 1];
  constexpr int kOddKeys = 32 * kFewWaves > KT ? 32 * kFewWaves : KT;
  // of a chunk of eight values, two bits for each; at the end 512 bytes of up to three waves
  __shared__ __align__(16) uint16_t lds_odd[kOddKeys * D / 8 > 768 ? kOddKeys * D / 8 : 768];
  __shared__ int lds_any[2];
  // Of 256-wide heads the last query fragments stay in LDS: the registers would not hold them, and a
  // reload from scratch memory waits for the copies under way.
  constexpr int kHeld = D == 256 ? D / 16 - (kFp8 ? 2 : 3) : D / 16;  // fragments in registers
  __shared__ __align__(16) uint4 lds_q[kHeld < D / 16 ? (D / 16 - kHeld) * 64 * WAVES : 1];
  const int lane = threadIdx.x & 63, wave = uniform((int)(threadIdx.x >> 6)), n = lane & 31, h = lane >> 5;
  const int group = a.Hq / a.Hkv;
  const uint32_t self = (uint32_t)plan.first + blockIdx.x, rest = self / (uint32_t)a.Hkv;
  const int kvh = (int)(self - rest * (uint32_t)a.Hkv);
  Block blk;
  Part mine_part{};
  if (kPaged && plan.shares > 0) {
    if (!find_share<kFp8>(a, plan, (int)rest, kvh, KT, blk, mine_part)) return;
  } else {
    const int64_t number = plan.blocks - 1 - (int)(rest / (uint32_t)plan.splits);  // a sequence's longest rows first
    const bool ranked = !kPaged && a.causal && a.window == 0 && a.B > 1 && a.B <= 64 && plan.splits == 1;
    if (!(ranked ? find_ranked(a, (int)rest, KT, blk) : find_block(a, number, KT, blk))) return;
    mine_part = Part{plan.per, (int)(rest % (uint32_t)plan.splits), plan.splits,
                     (number * a.Hkv + kvh) * plan.splits, 1};
  }
  const int split = mine_part.split, tile0 = split * mine_part.per, tile_end = min(blk.tiles, tile0 + mine_part.per);
  if (split > 0 && tile0 >= blk.tiles) return;

  // Blocks of more than 64 rows: a wave takes 32 of them and all keys of a tile.  Of 33 to 64: two
  // waves share 32 rows and take 32 keys of a tile each.  Smaller ones: the waves share all
  // rows, and each goes over tiles of 32 keys of its own.
  const int filled = min(kBlockRows, blk.rows - blk.row0);
  // (not the last rows of more: their keys would wait for fewer waves)
  const bool few = kPaged && kFewWaves > 1 && blk.rows <= kWaveRows;
  const bool shared = KT == 64 && !few && filled <= 2 * kWaveRows;
  const int half = shared ? wave & 1 : 0;  // of the tile's keys
  // the wave's rows; rows past the last one repeat it and are not stored
  const int wave_row = blk.row0 + (few ? 0 : shared ? wave >> 1 : wave) * kWaveRows;
  const bool working = few ? wave < kFewWaves : wave_row < blk.rows;
  const int row = min(wave_row + n, blk.rows - 1), token = row / group;
  auto low_of = [&](int place) { return a.window > 0 ? place - a.window + 1 : 0; };
  const int place = blk.place0 + token;
  const int seen_end = a.causal ? place + 1 : blk.end, seen_low = low_of(place);
  // of the wave's first and last row
  const int first_place = blk.place0 + min(wave_row, blk.rows - 1) / group;
  const int last_place = blk.place0 + (min(wave_row + kWaveRows, blk.rows) - 1) / group;
  const int all_end = a.causal ? first_place + 1 : blk.end;                    // keys before it are seen by all rows
  const int all_low = low_of(last_place);
  const int any_end = a.causal ? last_place + 1 : blk.end, any_low = low_of(first_place);

  // keys from block_low to block_end - 1 are seen by all rows of the block
  const int block_end = a.causal ? blk.place0 + blk.row0 / group + 1 : blk.end;
  const int block_low = low_of(blk.place0 + (min(blk.row0 + kBlockRows, blk.rows) - 1) / group);
  if (threadIdx.x < 2) lds_any[threadIdx.x] = 0;  // (before the first barrier)

  v8bf qf[kHeld];
  auto load_queries = [&]() FP8LIN_INLINE {
    const uint16_t *src =
        a.q + (int64_t)(blk.start + token) * a.q_token + (int64_t)(kvh * group + row % group) * a.q_head;
    // the order of few_tiles' raw codes, or key_frag's
    const int first = kFp8 && few ? 16 * h : 8 * h, odd_step = kFp8 && few ? 8 : 16;
    // the weights' exponents grow with the scores: a negative scale turns the queries over
    const uint32_t sign = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
    for (int s = 0; s < D / 16; s++) {
      const uint4 raw = *reinterpret_cast<const uint4 *>(src + first + 32 * (s >> 1) + odd_step * (s & 1));
      const v8bf f = as_bf16x8(raw.x ^ sign, raw.y ^ sign, raw.z ^ sign, raw.w ^ sign);
      if (s < kHeld)
        qf[s] = f;
      else
        lds_q[((s - kHeld) * WAVES + wave) * 64 + lane] = __builtin_bit_cast(uint4, f);
    }
  };
  auto query = [&](int s) FP8LIN_INLINE {
    return s < kHeld ? qf[s] : __builtin_bit_cast(v8bf, lds_q[((s - kHeld) * WAVES + wave) * 64 + lane]);
  };
  v16f o[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; i++)
#pragma unroll
    for (int j = 0; j < 16; j++) o[i][j] = 0.f;
  float m = -INFINITY, l = 0.f;
  const float scale = fabsf(a.scale), to_tanh = CAP ? scale / a.softcap : 0.f;

  // Copies.  Keys are taken in runs of 16 (which lie in one page): a wave's copy of 64 x 16
  // bytes covers a few rows of one run, at an address that the wave shares and offsets of
  // the lanes that repeat with the runs.
  int64_t found = 0;   // of a cache: lane x holds the line of run x of the next 64 runs
  int found_from = 0;  // key of run 0
  auto look_up = [&](int key0) FP8LIN_INLINE {
    found_from = key0;
    const int key = key0 + 16 * lane;
    if (key < blk.end) {
      const int p = (int)((uint32_t)key / (uint32_t)a.page_size);
      const int page = min(max(a.block_table[(int64_t)blk.b * a.max_pages + p], 0), a.pages - 1);
      found = ((int64_t)page * a.Hkv + kvh) * a.page_size + (key - p * a.page_size);
    }
  };
  // line in the cache of the first key of run `run` of the tile at key0
  auto run_line = [&](int key0, int run) FP8LIN_INLINE { return from_lane(found, (key0 - found_from) / 16 + run); };
  const int64_t k_line = kPaged ? D * kBytes : a.k_token * 2, v_line = kPaged ? D * kBytes : a.v_token * 2;
  const char *k_base = static_cast<const char *>(a.k) + (kPaged ? 0 : (int64_t)kvh * a.k_head * 2);
  const char *v_base = static_cast<const char *>(a.v) + (kPaged ? 0 : (int64_t)kvh * a.v_head * 2);
  // Rows of a tile that no row of the block sees may hold anything: such rows repeat the nearest
  // key that is seen.  Row r of the tile at key0 is then row near(r).
  auto near = [&](int key0, int r) FP8LIN_INLINE { return max(min(r, blk.end - 1 - key0), blk.lowest - key0); };
  auto whole = [&](int key0) FP8LIN_INLINE { return key0 >= blk.lowest && key0 + KT <= blk.end; };

  constexpr int kCopyRows = 1024 / (D * kBytes);  // rows of a wave's copy
  constexpr int kLanes = 64 / kCopyRows;          // lanes of a row
  constexpr int kCopies = KT / kCopyRows, kCopiesPer = (kCopies + WAVES - 1) / WAVES;
  // copy i of a wave covers rows copy_row(i) on; rows are alike modulo 16, so a few offsets serve all
  constexpr int kStep = kCopyRows * WAVES;
  constexpr int kKinds = kStep % 16 == 0 ? 1 : 16 / kStep < kCopiesPer ? 16 / kStep : kCopiesPer;
  auto copy_row = [&](int i) FP8LIN_INLINE { return i * kStep + wave * kCopyRows; };
  auto copy_run = [&](int i) FP8LIN_INLINE { return i * kStep / 16 + (kStep > 16 ? wave * kCopyRows / 16 : 0); };
  uint32_t k_off[kKinds], v_off[kKinds];
  auto offsets = [&](int r, int c, int src, uint32_t &ko, uint32_t &vo) FP8LIN_INLINE {
    ko = (uint32_t)((src & 15) * (int)k_line + 16 * (kFp8 ? c : key_swizzle<D>(r, c)));
    vo = (uint32_t)((src & 15) * (int)v_line + 16 * (kFp8 ? c : value_swizzle<D>(r, c)));
  };
#pragma unroll
  for (int i = 0; i < kKinds; i++) {
    const int r = copy_row(i) + lane / kLanes;
    offsets(r, lane % kLanes, r, k_off[i], v_off[i]);
  }
  // e4m3 codes go through registers: 16 codes of a lane become 32 bytes of bf16
  uint4 raw_k[kFp8 ? kCopiesPer : 1], raw_v[kFp8 ? kCopiesPer : 1];
  float raw_s[2];
  // kt, vt: the lines of the first row's run
  auto copy_rows = [&](int i, const char *kt, const char *vt, uint32_t ko, uint32_t vo, uint8_t *lk,
                       uint8_t *lv) FP8LIN_INLINE {
    const char *kp = scalar(kt) + ko, *vp = scalar(vt) + vo;
    if constexpr (kFp8) {
      raw_k[i] = *reinterpret_cast<const uint4 *>(kp);
      raw_v[i] = *reinterpret_cast<const uint4 *>(vp);
    } else {
      copy16_global_to_lds(kp, lk + copy_row(i) * kRow);
      copy16_global_to_lds(vp, lv + copy_row(i) * kRow);
    }
  };
  auto fetch = [&](int t, uint8_t *lk, uint8_t *lv) FP8LIN_INLINE {
    const int key0 = blk.begin + t * KT;
    if constexpr (kPaged) {
      if (t == tile0 || key0 + KT > found_from + 1024) look_up(key0);
    }
    const char *kt = k_base, *vt = v_base;  // the tile's lines, of rows
    const int64_t k_run16 = 16 * k_line, v_run16 = 16 * v_line;
    if constexpr (!kPaged) {
      kt += (int64_t)(blk.start + key0) * k_line;
      vt += (int64_t)(blk.start + key0) * v_line;
    }
    auto k_run = [&](int run) FP8LIN_INLINE { return kt + (kPaged ? run_line(key0, run) * kLine : run * k_run16); };
    auto v_run = [&](int run) FP8LIN_INLINE { return vt + (kPaged ? run_line(key0, run) * kLine : run * v_run16); };
    if (whole(key0)) {
#pragma unroll
      for (int i = 0; i < kCopiesPer; i++) {
        if (kCopies % WAVES != 0 && copy_row(i) >= KT) break;
        uint32_t ko = k_off[i % kKinds], vo = v_off[i % kKinds];
        if constexpr (D == 256) {  // no registers to keep them
          const int self = opaque(lane), r = copy_row(i) + self / kLanes;
          offsets(r, self % kLanes, r, ko, vo);
        }
        const int run = copy_run(i);
        copy_rows(i, k_run(run), v_run(run), ko, vo, lk, lv);
      }
    } else {
#pragma unroll
      for (int i = 0; i < kCopiesPer; i++) {
        if (kCopies % WAVES != 0 && copy_row(i) >= KT) break;
        const int self = opaque(lane), r = copy_row(i) + self / kLanes;
        uint32_t ko, vo;
        offsets(r, self % kLanes, near(key0, r), ko, vo);
        const int run = uniform(near(key0, copy_row(i))) >> 4;
        copy_rows(i, k_run(run), v_run(run), ko, vo, lk, lv);
      }
    }
    if constexpr (kFp8) {  // the scales: the first wave those of the keys, the last those of the values
      if (wave == 0 || wave == WAVES - 1) {
        const int src = near(key0, lane & (KT - 1));
        const int64_t at = __shfl(found, (key0 - found_from) / 16 + (src >> 4), 64) + (src & 15);
        if (wave == 0) raw_s[0] = a.k_scale[at];
        if (wave == WAVES - 1) raw_s[1] = a.v_scale[at];
      }
    }
  };
  auto store_codes = [&](uint8_t *lk, uint8_t *lv, float *ls) FP8LIN_INLINE {
    auto put = [&](const uint4 &raw, uint8_t *row_at, int c0, int c1) FP8LIN_INLINE {
      const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
      uint32_t b[8];
#pragma unroll
      for (int j = 0; j < 4; j++) {
        b[2 * j] = e4m3x2_to_bf16<false>(w[j]);
        b[2 * j + 1] = e4m3x2_to_bf16<true>(w[j]);
      }
      *reinterpret_cast<uint4 *>(row_at + 16 * c0) = make_uint4(b[0], b[1], b[2], b[3]);
      *reinterpret_cast<uint4 *>(row_at + 16 * c1) = make_uint4(b[4], b[5], b[6], b[7]);
    };
    const int self = opaque(lane);
#pragma unroll
    for (int i = 0; i < kCopiesPer; i++) {
      if (kCopies % WAVES != 0 && copy_row(i) >= KT) break;
      const int r = copy_row(i) + self / kLanes, c = 2 * (self % kLanes);
      put(raw_k[i], lk + r * kRow, key_swizzle<D>(r, c), key_swizzle<D>(r, c + 1));
      put(raw_v[i], lv + r * kRow, value_swizzle<D>(r, c), value_swizzle<D>(r, c + 1));
    }
    if (wave == 0 && lane < KT) ls[lane] = raw_s[0];
    if (wave == WAVES - 1 && lane < KT) ls[KT + lane] = raw_s[1];
  };

  // Reads of a tile's fragments, from the lane's place in it: steps and value blocks change bits
  // of the place that nothing else has.
  const int key_at = (32 * half + n) * kRow + 16 * key_swizzle<D>(n, h);
  const int value_r = 4 * h + (lane & 15) / 4;
  const int value_at = (32 * half + value_r) * kRow + 8 * (lane & 1) +
                       16 * value_swizzle<D>(value_r, 2 * (lane >> 4 & 1) + (lane & 3) / 2);
  auto key_frag = [&](const uint8_t *lk, int at, int sub, int s) FP8LIN_INLINE {
    const uint4 raw = *reinterpret_cast<const uint4 *>(lk + (at ^ 32 * s) + 32 * sub * kRow);
    return as_bf16x8(raw.x, raw.y, raw.z, raw.w);
  };
  auto value_frag = [&](uint8_t *lv, int at, int db, int step) FP8LIN_INLINE {  // values 32 db .. of keys 16 step ..
    uint8_t *p = lv + (at ^ 64 * db) + 16 * step * kRow;
    const v4s lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)p);
    const v4s hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_v4s *)(p + 8 * kRow));
    typedef short v8s __attribute__((ext_vector_type(8)));
    return __builtin_bit_cast(v8bf, (v8s{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]}));
  };

  // The rows that see a value that was taken out of a tile get what a sum with it is.  (keys: of
  // the tile at key0; at: of the first one in lds_odd)
  auto put_odd = [&](int key0, int keys, int at) FP8LIN_INLINE {
    uint32_t flags[D / 16] = {};  // of the values of the keys that the row sees
#pragma unroll 1
    for (int key = max(0, seen_low - key0); key < min(keys, seen_end - key0); key++) {
      const uint4 *from = reinterpret_cast<const uint4 *>(lds_odd + (key + at) * (D / 8));
#pragma unroll
      for (int w = 0; w < D / 64; w++) {
        const uint4 f = from[w];
        flags[4 * w] |= f.x;
        flags[4 * w + 1] |= f.y;
        flags[4 * w + 2] |= f.z;
        flags[4 * w + 3] |= f.w;
      }
    }
#pragma unroll
    for (int i = 0; i < D / 8; i++) {
      const uint32_t f = flags[i / 2] >> (16 * (i & 1) + 8 * h);
#pragma unroll
      for (int j = 0; j < 4; j++)
        o[i / 4][4 * (i % 4) + j] += (f >> 2 * j & 1 ? INFINITY : 0.f) - (f >> 2 * j & 2 ? INFINITY : 0.f);
    }
  };
  // Weights of the scores sc of 32 S keys from key0 on.  before: what is done between the
  // maximum and the exponentials.  edge: some row of the wave does not see some of the keys.
  auto weigh = [&](auto subs, const v16f(&sc)[decltype(subs)::value], v8bf(&p)[2 * decltype(subs)::value], int key0,
                   const float *ks, const float *vs, bool edge, auto before) FP8LIN_INLINE {
    constexpr int S = decltype(subs)::value;
    float x[16 * S];
#pragma unroll
    for (int j = 0; j < 16 * S; j++) x[j] = sc[j / 16][j % 16];
    if constexpr (kFp8) {
#pragma unroll
      for (int j = 0; j < 4 * S; j++) {
        if (j % 4 == 0) __builtin_amdgcn_sched_barrier(0);
        const float4 g = *reinterpret_cast<const float4 *>(ks + 8 * j + 4 * h);
        x[4 * j] *= g.x;
        x[4 * j + 1] *= g.y;
        x[4 * j + 2] *= g.z;
        x[4 * j + 3] *= g.w;
      }
    }
    if constexpr (CAP) {
#pragma unroll
      for (int j = 0; j < 16 * S; j++) x[j] *= to_tanh;
      tanh_each(x);
    }
    const float rate = (CAP ? a.softcap : scale) * kLog2e;  // of the exponents in units of x
    const int live_end = seen_end - key0 - 4 * h, live_low = seen_low - key0 - 4 * h;
    auto live = [&](int j) { return 8 * (j >> 2) + (j & 3) < live_end && 8 * (j >> 2) + (j & 3) >= live_low; };
    if (edge) {
#pragma unroll
      for (int j = 0; j < 16 * S; j++) x[j] = live(j) ? x[j] : -INFINITY;
    }
    float top = x[0];
#pragma unroll
    for (int j = 1; j < 16 * S; j++) top = fmaxf(top, x[j]);
    top = product(top, rate);
    // The reference of the exponents follows the maximum only when some score passes it by
    // 2^8: weights stay below 2^8 and sums far below overflow, and most tiles need no
    // exchange between the lane halves and no product with the factor.  The reference is a rounded
    // product: from 2^26 on an exact one may lie far from it (all weights would be 0, or infinite), and
    // the products are rounded as it was.
    float factor = rate;
    bool rounded = false;
    if (__any(top > (fabsf(m) < kLarge ? m + 8.f : -INFINITY))) {
      top = fmaxf(fmaxf(top, __shfl_xor(top, 32, 64)), m);
      const float shrink = top == m ? 1.f : __builtin_amdgcn_exp2f(m - top);
      m = top;
      l *= shrink;
#pragma unroll
      for (int i = 0; i < D / 32; i++) o[i] *= shrink;
      const float large = m == -INFINITY ? 0.f : m;
      rounded = __any(fabsf(large) >= kLarge);
      if (__builtin_expect(rounded, 0)) {
        factor = 1.f;
#pragma unroll
        for (int j = 0; j < 16 * S; j++) x[j] = product(x[j], rate) - large;
      }
    }
    before();
    const float base = rounded || m == -INFINITY ? 0.f : m;
#pragma unroll
    for (int j = 0; j < 16 * S; j++) x[j] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[j], factor, -base));
    {
      float sum[4] = {};
#pragma unroll
      for (int j = 0; j < 16 * S; j++) sum[j & 3] += x[j];
      l += (sum[0] + sum[1]) + (sum[2] + sum[3]);
    }
    if constexpr (kFp8) {
#pragma unroll
      for (int j = 0; j < 4 * S; j++) {
        if (j % 4 == 0) __builtin_amdgcn_sched_barrier(0);
        const float4 g = *reinterpret_cast<const float4 *>(vs + 8 * j + 4 * h);
        x[4 * j] *= g.x;
        x[4 * j + 1] *= g.y;
        x[4 * j + 2] *= g.z;
        x[4 * j + 3] *= g.w;
      }
      if (edge) {  // a scale that is not finite belongs to no row that does not see its key
#pragma unroll
        for (int j = 0; j < 16 * S; j++) x[j] = live(j) ? x[j] : 0.f;
      }
    }
#pragma unroll
    for (int s = 0; s < 2 * S; s++)
      p[s] = as_bf16x8(pack_bf16x2(x[8 * s], x[8 * s + 1]), pack_bf16x2(x[8 * s + 2], x[8 * s + 3]),
                       pack_bf16x2(x[8 * s + 4], x[8 * s + 5]), pack_bf16x2(x[8 * s + 6], x[8 * s + 7]));
  };

  // One tile; odd: lds_odd has values
  // that were taken out of the tile.
  auto use_tile = [&](auto subs, int key0, uint8_t *lk, uint8_t *lv, const float *ks, const float *vs,
                      bool edge, bool odd) FP8LIN_INLINE {
    constexpr int S = decltype(subs)::value;
    // Fragments are read a few steps ahead of the products that take them, and no earlier: the
    // compiler would fill the registers with them.
    constexpr int kKeyRing = S == 2 ? 3 : D == 256 ? 2 : 4, kSteps = D / 16;
    const int ka = opaque(key_at);
    v16f sc[S];
    v8bf kf[kKeyRing][S];
    auto read_keys = [&](int s) FP8LIN_INLINE {
#pragma unroll
      for (int sub = 0; sub < S; sub++) kf[s % kKeyRing][sub] = key_frag(lk, ka, sub, s);
    };
#pragma unroll
    for (int s = 0; s + 1 < kKeyRing; s++) read_keys(s);
#pragma unroll
    for (int sub = 0; sub < S; sub++)
#pragma unroll
      for (int j = 0; j < 16; j++) sc[sub][j] = 0.f;
#pragma unroll
    for (int s = 0; s < kSteps; s++) {
      if (s + kKeyRing - 1 < kSteps) read_keys(s + kKeyRing - 1);
      step_ends();
#pragma unroll
      for (int sub = 0; sub < S; sub++)
        sc[sub] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[s % kKeyRing][sub], query(s), sc[sub], 0, 0, 0);
      step_ends();
    }
    constexpr int kDb = D / 32, kProducts = kDb * 2 * S, kValueRing = D == 256 ? 2 : 4;
    const int va = opaque(value_at);
    v8bf vf[kValueRing];
    auto read_values = [&](int i) FP8LIN_INLINE { vf[i % kValueRing] = value_frag(lv, va, i % kDb, i / kDb); };
    v8bf p[2 * S];
    weigh(subs, sc, p, key0, ks, vs, edge, [&]() FP8LIN_INLINE {
#pragma unroll
      for (int i = 0; i + 1 < kValueRing; i++) read_values(i);
      step_ends();
    });
#pragma unroll
    for (int i = 0; i < kProducts; i++) {
      if (i + kValueRing - 1 < kProducts) read_values(i + kValueRing - 1);
      step_ends();
      o[i % kDb] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[i % kValueRing], p[i / kDb], o[i % kDb], 0, 0, 0);
      step_ends();
    }
    if (__builtin_expect(odd, 0)) put_odd(key0, 32 * S, 32 * half);
  };
  // 0 times an infinity or a NaN is a NaN, and such a value must not reach rows that do not see
  // its key: they are taken out of a tile of values and noted in lds_odd.
  auto take_odd = [&](uint8_t *lv, int parity) FP8LIN_INLINE -> bool {
    bool mine = false;
    const int self = opaque(threadIdx.x);
    for (int i = self; i < KT * D / 8; i += 64 * WAVES) {
      const uint4 x = *reinterpret_cast<const uint4 *>(lv + 16 * i);
      mine |= (not_finite(x.x) | not_finite(x.y) | not_finite(x.z) | not_finite(x.w)) != 0;
    }
    if (mine) lds_any[parity] = 1;
    lds_barrier();
    const bool any = uniform(lds_any[parity]) != 0;
    if (__builtin_expect(!any, 1)) return false;
    for (int i = self; i < KT * D / 8; i += 64 * WAVES) {
      uint4 *at = reinterpret_cast<uint4 *>(lv + 16 * i);
      const uint4 x = *at;
      const uint32_t w[4] = {x.x, x.y, x.z, x.w};
      uint32_t kept[4], flags = 0;
#pragma unroll
      for (int j = 0; j < 4; j++) {
        kept[j] = w[j];
#pragma unroll
        for (int e = 0; e < 2; e++) {
          const uint32_t v = w[j] >> 16 * e & 0xFFFFu;
          if ((v & 0x7F80u) != 0x7F80u) continue;
          kept[j] &= ~(0xFFFFu << 16 * e);
          flags |= (v & 0x7Fu ? 3u : v >> 15 ? 2u : 1u) << (4 * j + 2 * e);
        }
      }
      const int r = i / (D / 8), c = i % (D / 8);  // position c holds chunk value_swizzle(r, c): it is its own inverse
      lds_odd[r * (D / 8) + value_swizzle<D>(r, c)] = (uint16_t)flags;
      *at = make_uint4(kept[0], kept[1], kept[2], kept[3]);
    }
    lds_barrier();
    if (threadIdx.x == 0) lds_any[parity] = 0;
    return true;
  };

  // subs: sets of 32 keys of a tile that the wave takes
  auto all_tiles = [&](auto subs) FP8LIN_INLINE {
    constexpr int kMine = 32 * decltype(subs)::value;
    auto step = [&](int t, auto stage) FP8LIN_INLINE {
      constexpr bool kOdd = decltype(stage)::value;
      uint8_t *lk = kOdd ? lds_k1 : lds_k0, *lv = kOdd ? lds_v1 : lds_v0;
      float *ls = kOdd ? lds_s1 : lds_s0;
      if constexpr (kFp8)
        store_codes(lk, lv, ls);
      else
        wait_global_loads();
      __syncthreads();
      if (t + 1 < tile_end) fetch(t + 1, kOdd ? lds_k0 : lds_k1, kOdd ? lds_v0 : lds_v1);
      const int key0 = blk.begin + t * KT, mine = key0 + 32 * half;
      bool odd = false;
      if (key0 + KT > block_end || key0 < block_low) odd = take_odd(lv, kOdd);
      const bool edge = mine + kMine > all_end || mine < all_low;
      if (working && mine < any_end && mine + kMine > any_low)
        use_tile(subs, mine, lk, lv, ls + 32 * half, ls + KT + 32 * half, edge, odd);
    };
    if (tile0 < tile_end) {
      fetch(tile0, lds_k0, lds_v0);
      load_queries();
    }
    for (int t = tile0; t < tile_end; t += 2) {
      step(t, std::false_type{});
      if (t + 1 < tile_end) step(t + 1, std::true_type{});
    }
  };
  // Blocks of at most 32 rows, over a cache.  A wave's tile of 32 keys lies in LDS as it lies in memory (codes
  // become bf16 when they are read: no other wave reads them); the copies of the next
  // tile are under way while one is used, and no wave waits for another.
  auto raw_swizzle = [&](int r, int c) FP8LIN_INLINE {
    return c ^ (D == 64 ? r >> 2 & 3 : D == 128 ? r >> 1 & 7 : r & 15);
  };
  auto few_tiles = [&]() FP8LIN_INLINE {
    constexpr int kFewCopies = 32 / kCopyRows, kLoads = 2 * kFewCopies + (kFp8 ? 1 : 0);
    const int key_begin = blk.begin + tile0 * KT, key_end = min(blk.end, blk.begin + tile_end * KT);
    const int tiles = (key_end - key_begin + 31) / 32;
    auto key_of = [&](int i) FP8LIN_INLINE { return key_begin + 32 * (wave + kFewWaves * i); };  // of the wave's tile i
    const int rl = lane / kLanes, cl = lane % kLanes;
    auto place = [&](auto keys, int r, int c) FP8LIN_INLINE {  // source chunk of position c of row r
      constexpr bool kKeys = decltype(keys)::value;
      return kFp8 ? raw_swizzle(r, c) : kKeys ? key_swizzle<D>(r, c) : value_swizzle<D>(r, c);
    };
    int64_t runs = 0;  // lane x holds the line of run x % 2 of the wave's tile 32 j + x / 2
    auto fetch = [&](int i, uint8_t *lk, uint8_t *lv, float *ls) FP8LIN_INLINE {
      const int key0 = key_of(i);
      if (i % 32 == 0) {
        const int key = key_of(i + (lane >> 1)) + 16 * (lane & 1);
        if (key < blk.end) {
          const int p = (int)((uint32_t)key / (uint32_t)a.page_size);
          const int page = min(max(a.block_table[(int64_t)blk.b * a.max_pages + p], 0), a.pages - 1);
          runs = ((int64_t)page * a.Hkv + kvh) * a.page_size + (key - p * a.page_size);
        }
      }
      const bool full = key0 >= blk.lowest && key0 + 32 <= blk.end;
      auto line_of = [&](int run) FP8LIN_INLINE { return from_lane(runs, 2 * (i % 32) + run); };
      auto copy = [&](auto keys, int j, const char *base, int64_t line, uint8_t *to) FP8LIN_INLINE {
        const int r0 = j * kCopyRows;  // and rl: a copy's rows differ from the first one's by whole bits
        const int flip = place(keys, r0, 0);
        int run = r0 >> 4;
        uint32_t at;
        if (full) {
          at = (uint32_t)(((r0 & 15) + rl) * (int)line + 16 * (place(keys, rl, cl) ^ flip));
        } else {
          const int src = near(key0, r0 + opaque(rl));
          run = uniform(near(key0, r0)) >> 4;
          at = (uint32_t)((src & 15) * (int)line + 16 * (place(keys, rl, cl) ^ flip));
        }
        copy16_global_to_lds(scalar(base + line_of(run) * line) + at, to + wave * kFewTile + r0 * kLine);
      };
#pragma unroll
      for (int j = 0; j < kFewCopies; j++) copy(std::true_type{}, j, k_base, k_line, lk);
#pragma unroll
      for (int j = 0; j < kFewCopies; j++) copy(std::false_type{}, j, v_base, v_line, lv);
      if constexpr (kFp8) {  // lanes 0 .. 31 the keys' scales, the others the values'
        const int src = near(key0, n);
        const int64_t at = (src >> 4 ? line_of(1) : line_of(0)) + (src & 15);
        __builtin_amdgcn_global_load_lds((glb_void *)const_cast<float *>((h ? a.v_scale : a.k_scale) + at),
                                         (lds_void *)(ls + 64 * wave), 4, 0, 0);
      }
      step_ends();
    };
    const int few_key = kFp8 ? wave * kFewTile + n * kLine + 16 * raw_swizzle(n, h)
                             : wave * kFewTile + n * kLine + 16 * key_swizzle<D>(n, h);
    const int vr = kFp8 ? 4 * h + (lane >> 1 & 3) + 8 * (lane >> 3 & 1) : value_r, dh = lane >> 4 & 1;
    const int few_value = wave * kFewTile + vr * kLine + 8 * (lane & 1) +
                          16 * (kFp8 ? raw_swizzle(vr, dh) : value_swizzle<D>(vr, 2 * dh + (lane & 3) / 2));
    auto bf16_of = [&](uint32_t w0, uint32_t w1) FP8LIN_INLINE {
      return as_bf16x8(e4m3x2_to_bf16<false>(w0), e4m3x2_to_bf16<true>(w0), e4m3x2_to_bf16<false>(w1),
                       e4m3x2_to_bf16<true>(w1));
    };
    auto few_value_frag = [&](uint8_t *lv, int at, int db, int step) FP8LIN_INLINE {
      if constexpr (!kFp8) {
        return value_frag(lv, at, db, step);
      } else {
        const v2i raw = __builtin_amdgcn_ds_read_tr8_b64_v2i32((lds_v2i *)(lv + (at ^ 32 * db) + 16 * step * kLine));
        return bf16_of((uint32_t)raw[0], (uint32_t)raw[1]);
      }
    };
    // Values that are not finite, as in take_odd, in the wave's own tile.
    auto take_few_odd = [&](uint8_t *lv, float *vs) FP8LIN_INLINE -> bool {
      constexpr int kParts = kFewTile / 16;
      const int self = opaque(lane);
      uint8_t *const mine = lv + wave * kFewTile;
      auto finite = [](float x) { return (__float_as_uint(x) & 0x7F800000u) != 0x7F800000u; };
      bool found_one = false;
      if (kFp8 && self < 32) found_one = !finite(vs[self]);
      for (int i = self; i < kParts; i += 64) {
        const uint4 x = *reinterpret_cast<const uint4 *>(mine + 16 * i);
        const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
        for (int j = 0; j < 4; j++)
          found_one |= (kFp8 ? ((w[j] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u : not_finite(w[j])) != 0;
      }
      if (__builtin_expect(!__any(found_one), 1)) return false;
#pragma unroll 1
      for (int i = self; i < kParts; i += 64) {
        constexpr int kChunks = kLine / 16, kEach = 16 / kBytes;
        uint32_t *at = reinterpret_cast<uint32_t *>(mine + 16 * i);
        const int r = i / kChunks, c = place(std::false_type{}, r, i % kChunks);
        uint32_t flags = 0;
#pragma unroll 1
        for (int j = 0; j < kEach; j++) {
          const int word = j * kBytes / 4, shift = 8 * (j * kBytes % 4);
          const uint32_t bits = at[word] >> shift & (kFp8 ? 0xFFu : 0xFFFFu);
          float v = bf16_to_f32(bits);
          if constexpr (kFp8) v = bf16_to_f32(e4m3x2_to_bf16<false>(bits) & 0xFFFFu) * vs[r];
          if (finite(v)) continue;
          at[word] &= ~((kFp8 ? 0xFFu : 0xFFFFu) << shift);
          flags |= (v != v ? 3u : v < 0.f ? 2u : 1u) << 2 * j;
        }
        uint16_t *to = lds_odd + (32 * wave + r) * (D / 8) + c * kEach / 8;
        to[0] = (uint16_t)flags;
        if constexpr (kFp8) to[1] = (uint16_t)(flags >> 16);
      }
      step_ends();
      if (kFp8 && self < 32 && !finite(vs[self])) vs[self] = 0.f;
      step_ends();
      return true;
    };
    auto step = [&](int i, auto stage) FP8LIN_INLINE {
      constexpr bool kOdd = decltype(stage)::value;
      uint8_t *lk = kOdd ? lds_k1 : lds_k0, *lv = kOdd ? lds_v1 : lds_v0;
      float *ls = (kOdd ? lds_s1 : lds_s0) + 64 * wave * (kFp8 ? 1 : 0);
      if (wave + kFewWaves * (i + 1) < tiles) {
        fetch(i + 1, kOdd ? lds_k0 : lds_k1, kOdd ? lds_v0 : lds_v1, kOdd ? lds_s0 : lds_s1);
        __builtin_amdgcn_s_waitcnt(0x0F70 | (kLoads & 15) | (kLoads >> 4) << 14);  // all but the copies just begun
      } else {
        wait_global_loads();
      }
      step_ends();
      const int key0 = key_of(i);
      const bool edge = key0 + 32 > all_end || key0 < all_low;
      const bool odd = edge && take_few_odd(lv, ls + 32);
      v16f sc[1];
#pragma unroll
      for (int j = 0; j < 16; j++) sc[0][j] = 0.f;
      const int ka = opaque(few_key), va = opaque(few_value);
      if constexpr (kFp8) {
#pragma unroll
        for (int c = 0; c < D / 32; c++) {
          const uint4 raw = *reinterpret_cast<const uint4 *>(lk + (ka ^ 32 * c));
          sc[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf16_of(raw.x, raw.y), query(2 * c), sc[0], 0, 0, 0);
          sc[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(bf16_of(raw.z, raw.w), query(2 * c + 1), sc[0], 0, 0, 0);
          if (c % 4 == 3) step_ends();
        }
      } else {
#pragma unroll
        for (int s = 0; s < D / 16; s++) {
          sc[0] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(key_frag(lk, ka, 0, s), query(s), sc[0], 0, 0, 0);
          if (s % 4 == 3) step_ends();
        }
      }
      v8bf p[2];
      weigh(std::integral_constant<int, 1>{}, sc, p, key0, ls, ls + 32, edge, [] {});
#pragma unroll
      for (int j = 0; j < 2 * (D / 32); j++) {
        const int db = j % (D / 32), s = j / (D / 32);
        o[db] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(few_value_frag(lv, va, db, s), p[s], o[db], 0, 0, 0);
        if (j % 4 == 3) step_ends();
      }
      if (__builtin_expect(odd, 0)) put_odd(key0, 32, 32 * wave);
    };
    if (wave >= tiles) return;
    fetch(0, lds_k0, lds_v0, lds_s0);
    load_queries();
    for (int i = 0; wave + kFewWaves * i < tiles; i += 2) {
      step(i, std::false_type{});
      if (wave + kFewWaves * (i + 1) < tiles) step(i + 1, std::true_type{});
    }
  };
  if (few) {
    if constexpr (kPaged && kFewWaves > 1) {
      if (working) few_tiles();
    }
  } else if constexpr (KT == 64) {
    if (shared)
      all_tiles(std::integral_constant<int, 1>{});
    else
      all_tiles(std::integral_constant<int, 2>{});
  } else {
    all_tiles(std::integral_constant<int, 1>{});
  }

  if (few || shared) {
    // The other waves of the rows hand their states to the first, lane by lane: each has a box
    // for o, and 512 bytes for m and l.
    auto box = [&](int slot, int i) FP8LIN_INLINE {
      const int part = D == 256 ? 2 * slot + i / 16 : slot, at = D == 256 ? i % 16 : i;
      uint8_t *base = part == 0 ? lds_k0 : part == 1 ? lds_k1 : part == 2 ? lds_v0 : lds_v1;
      return reinterpret_cast<float4 *>(base) + 64 * at + lane;
    };
    float *ml = reinterpret_cast<float *>(lds_odd);
    const int slot = few ? wave - 1 : wave >> 1;
    const bool gives = working && (few ? wave > 0 : half == 1);
    __syncthreads();
    if (gives) {
#pragma unroll
      for (int i = 0; i < D / 8; i++)
        *box(slot, i) = make_float4(o[i / 4][4 * (i % 4)], o[i / 4][4 * (i % 4) + 1], o[i / 4][4 * (i % 4) + 2],
                                    o[i / 4][4 * (i % 4) + 3]);
      ml[128 * slot + lane] = m;
      ml[128 * slot + 64 + lane] = l;
    }
    __syncthreads();
    if (gives || (few && wave > 0)) return;
    const int end = few ? kFewWaves - 1 : slot + 1;
    if (!working) return;
    for (int from = few ? 0 : slot; from < end; from++) {
      const float m2 = ml[128 * from + lane], top = fmaxf(m, m2);
      const float f1 = m == top ? 1.f : __builtin_amdgcn_exp2f(m - top);
      const float f2 = m2 == top ? 1.f : __builtin_amdgcn_exp2f(m2 - top);
      m = top;
      l = l * f1 + ml[128 * from + 64 + lane] * f2;
#pragma unroll
      for (int i = 0; i < D / 8; i++) {
        const float4 x = *box(from, i);
        float *mine = reinterpret_cast<float *>(&o[i / 4]) + 4 * (i % 4);
        mine[0] = mine[0] * f1 + x.x * f2;
        mine[1] = mine[1] * f1 + x.y * f2;
        mine[2] = mine[2] * f1 + x.z * f2;
        mine[3] = mine[3] * f1 + x.w * f2;
      }
    }
  }
  if (!working) return;
  l += __shfl_xor(l, 32, 64);
  const int mine = wave_row + opaque(n);
  if (mine >= blk.rows) return;
  const int64_t out = (int64_t)(blk.start + mine / group) * a.Hq + kvh * group + mine % group;
  if (blk.tiles <= mine_part.per) {
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t *dst = a.o + out * D + 4 * h;
#pragma unroll
    for (int i = 0; i < D / 8; i++) {
      const v16f &v = o[i / 4];
      const int j = 4 * (i % 4);
      *reinterpret_cast<uint2 *>(dst + 8 * i) =
          make_uint2(pack_bf16x2(v[j] * inv, v[j + 1] * inv), pack_bf16x2(v[j + 2] * inv, v[j + 3] * inv));
    }
    if (a.lse && h == 0) a.lse[out] = l == 0.f ? -INFINITY : kLn2 * (m + log2f(l));
  } else {
    float *base = part + (mine_part.slot + split * mine_part.step) * (int64_t)prompt_part_floats(D);
    const int r = mine - blk.row0;
#pragma unroll
    for (int i = 0; i < D / 8; i++) {
      const v16f &v = o[i / 4];
      const int j = 4 * (i % 4);
      *reinterpret_cast<float4 *>(base + r * D + 8 * i + 4 * h) = make_float4(v[j], v[j + 1], v[j + 2], v[j + 3]);
    }
    if (h == 0) {
      base[kBlockRows * D + r] = m;
      base[kBlockRows * (D + 1) + r] = l;
    }
  }
}

// Joins the parts of divided blocks, in order: D / 4 lanes take a row, kJoinRows rows a
// workgroup.
template <int D>
constexpr int kJoinRows = 256 / (D / 4);
template <int D>
__global__ __launch_bounds__(256) void prompt_join_kernel(PromptArgs a, PromptPlan plan, const float *part) {
  const int group = a.Hq / a.Hkv;
  const int64_t number = blockIdx.x / (unsigned)a.Hkv;  // few blocks are divided: one launch
  const int kvh = (int)(blockIdx.x % (unsigned)a.Hkv);
  const int d = (int)(threadIdx.x % (D / 4)) * 4;
  Block blk;
  Part from{};
  // of shares the block's parts' workgroups take its rows in turn
  int first = (int)blockIdx.y, stride = (int)gridDim.y;
  if (plan.shares > 0) {
    if (!(a.k_scale ? find_share<true>(a, plan, (int)number, kvh, tile_keys(D), blk, from)
                    : find_share<false>(a, plan, (int)number, kvh, tile_keys(D), blk, from)))
      return;
    first = from.split * stride + first;
    stride *= from.splits;
  } else {
    if (!find_block(a, number, tile_keys(D), blk)) return;
    from = Part{plan.per, 0, plan.splits, (number * a.Hkv + kvh) * plan.splits, 1};
  }
  if (blk.tiles <= from.per) return;
  const int parts = (blk.tiles + from.per - 1) / from.per;
  const int64_t floats = (int64_t)from.step * prompt_part_floats(D);
  const float *base = part + from.slot * prompt_part_floats(D);
  const int filled = min(kBlockRows, blk.rows - blk.row0);
  for (int r = first * kJoinRows<D> + (int)threadIdx.x / (D / 4); r < filled; r += stride * kJoinRows<D>) {
    float top = -INFINITY, l = 0.f, o[4] = {};
    for (int k0 = 0; k0 < parts; k0 += 4) {  // four parts in flight
      float mp[4], lp[4];
      float4 op[4];
#pragma unroll
      for (int u = 0; u < 4; u++) {
        const float *p = base + (int64_t)min(k0 + u, parts - 1) * floats;
        mp[u] = p[kBlockRows * D + r];
        lp[u] = p[kBlockRows * (D + 1) + r];
        op[u] = *reinterpret_cast<const float4 *>(p + r * D + d);
      }
      const float high = fmaxf(fmaxf(fmaxf(mp[0], mp[1]), fmaxf(mp[2], mp[3])), top);
      const float shrink = top == high ? 1.f : __builtin_amdgcn_exp2f(top - high);
      top = high;
      l *= shrink;
#pragma unroll
      for (int e = 0; e < 4; e++) o[e] *= shrink;
#pragma unroll
      for (int u = 0; u < 4; u++) {
        if (k0 + u < parts) {
          const float f = mp[u] == top ? 1.f : __builtin_amdgcn_exp2f(mp[u] - top);
          l += lp[u] * f;
          o[0] += op[u].x * f;
          o[1] += op[u].y * f;
          o[2] += op[u].z * f;
          o[3] += op[u].w * f;
        }
      }
    }
    const int row = blk.row0 + r;
    const int64_t out = (int64_t)(blk.start + row / group) * a.Hq + kvh * group + row % group;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    *reinterpret_cast<uint2 *>(a.o + out * D + d) =
        make_uint2(pack_bf16x2(o[0] * inv, o[1] * inv), pack_bf16x2(o[2] * inv, o[3] * inv));
    if (a.lse && d == 0) a.lse[out] = l == 0.f ? -INFINITY : kLn2 * (top + log2f(l));
  }
}

template <int D, Source SRC, bool CAP>
hipError_t launch(const PromptArgs &a, const PromptPlan &p, float *part, hipStream_t stream) {
  const int64_t all = prompt_parts(p, a.Hkv);
  PromptPlan q = p;
  for (int64_t first = 0; first < all; first += kPromptGrid) {
    q.first = (int)first;
    const dim3 grid((unsigned)(all - first < kPromptGrid ? all - first : kPromptGrid));
    hipLaunchKernelGGL((prompt_kernel<D, SRC, CAP>), grid, dim3(64 * kBlockWaves), 0, stream, a, q, part);
  }
  if (prompt_joins(p)) {
    // four passes each where there are many: workgroups that only look their block up take longer than they save
    const int rows = kJoinRows<D> * ((int64_t)p.blocks * a.Hkv * p.filled > 1024 * kJoinRows<D> ? 4 : 1);
    const unsigned x = p.shares > 0 ? (unsigned)all : (unsigned)p.blocks * (unsigned)a.Hkv;
    const unsigned y = p.shares > 0 ? (p.filled > kWaveRows ? 2 : 1) : (unsigned)((p.filled + rows - 1) / rows);
    hipLaunchKernelGGL((prompt_join_kernel<D>), dim3(x, y), dim3(256), 0, stream, a, p, (const float *)part);
  }
  return hipGetLastError();
}

template <int D>
hipError_t launch_dim(const PromptArgs &a, const PromptPlan &p, float *part, hipStream_t stream) {
  auto with = [&](auto source) {
    constexpr Source kSrc = decltype(source)::value;
    return a.softcap > 0.f ? launch<D, kSrc, true>(a, p, part, stream) : launch<D, kSrc, false>(a, p, part, stream);
  };
  if (!a.block_table) return with(std::integral_constant<Source, Source::kRows>{});
  return a.k_scale ? with(std::integral_constant<Source, Source::kCodes>{})
                   : with(std::integral_constant<Source, Source::kCache>{});
}

}  // namespace

size_t prompt_partial_bytes(const PromptArgs &a, int cus) {
  const PromptPlan p = plan_prompt(a, cus);
  return prompt_joins(p) ? (size_t)prompt_parts(p, a.Hkv) * prompt_part_floats(a.D) * sizeof(float) : 0;
}

hipError_t launch_prompt_attention(const PromptArgs &a, float *part, hipStream_t stream) {
  const PromptPlan p = plan_prompt(a, device_cu_count());
  if (a.D == 64) return launch_dim<64>(a, p, part, stream);
  if (a.D == 128) return launch_dim<128>(a, p, part, stream);
  return launch_dim<256>(a, p, part, stream);
}

}  // namespace fp8lin
