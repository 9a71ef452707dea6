// How the attention of prompt_attention.hip divides a batch: the launch plan, which the
// host makes from sizes alone.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "launch_layer.hpp"

namespace fp8lin {

constexpr int kWaveRows = 32;    // rows of a wave; a row is a token and a query head of one key head
constexpr int kBlockWaves = 4;   // waves of a workgroup
constexpr int kBlockRows = kBlockWaves * kWaveRows;
constexpr int tile_keys(int D) { return D == 256 ? 32 : 64; }

// A block of kBlockRows rows of one sequence and key head is a workgroup, or `splits` of
// them that take `per` key tiles each and leave partials.  Blocks are numbered through the
// batch: sequence b has numbers first_block(b) .. first_block(b + 1) - 1, some unused.
// With shares the blocks of the longest sequences are divided most: the kernel finds
// from the lengths how, so that a key head has at most `shares` parts (`per` is then the number
// of tiles that no block has more of).
struct PromptPlan {
  int splits, per, shares;
  int blocks;
  int filled;  // rows of a block, on average
  int first;  // workgroup of the whole grid that a launch begins at
};

// Sequences of a batch that shares are made for: four a lane.
constexpr int kShareBatch = 256;

// Most bytes of partials that a division leaves.
constexpr int64_t kMostPartialBytes = 300000000;

// Workgroups of one launch: a grid counts its threads in 32 bits.
constexpr int kPromptGrid = 1 << 22;

// Number of the first block of a sequence whose first token is `start`: at least as many
// numbers lie between two sequences' as the first one's rows need.
__host__ __device__ inline int64_t first_block(int64_t start, int64_t b, int group) {
  return start * group / kBlockRows + b;
}

// Partials of one part of a block: o [kBlockRows][D], then m and l [kBlockRows] each.
__host__ __device__ constexpr int prompt_part_floats(int D) { return kBlockRows * (D + 2); }

// Workgroups of the attention, each of which may leave partials.
inline int64_t prompt_parts(const PromptPlan &p, int Hkv) {
  return (int64_t)Hkv * (p.shares > 0 ? p.shares : (int64_t)p.blocks * p.splits);
}
inline bool prompt_joins(const PromptPlan &p) { return p.splits > 1 || p.shares > 0; }

inline PromptPlan plan_prompt(const PromptArgs &a, int cus) {
  const int group = a.Hq / a.Hkv;
  const int64_t rows = (int64_t)a.T * group;  // of a key head
  PromptPlan p{};
  p.blocks = (int)first_block(a.T, a.B, group);
  int64_t keys = a.max_len;  // that a block sees, from the run of 16 on that holds the first one
  const int64_t seen = (int64_t)a.window + (kBlockRows + group - 1) / group + 15;
  if (a.window > 0 && keys > seen) keys = seen;
  const int tile = tile_keys(a.D);
  const int64_t tiles = keys <= tile ? 1 : (keys + tile - 1) / tile;
  const int64_t found = (int64_t)p.blocks * a.Hkv;
  p.filled = rows <= p.blocks ? 1 : (int)(rows / p.blocks);
  int64_t splits = 1;
  // Workgroups whose partials kMostPartialBytes holds, and the most that an even division makes: eight a
  // compute unit.
  const int64_t held = kMostPartialBytes / (prompt_part_floats(a.D) * (int64_t)sizeof(float));
  const int64_t most = 8 * cus < held ? 8 * cus : held;
  if (a.block_table && a.B > 1 && a.B <= kShareBatch && found <= most && tiles > 4) {
    // As many parts as run at once, or a multiple of it where there are more blocks: a few more than run
    // at once take longest.  (32 sequences of 5 to 8192 tokens, 16 rows each, e4m3, 8 key
    // heads: 64 parts a head 58 us, 72 70, 128 66, 192 75; of equal lengths 52 with 64, and 67 in 8 parts
    // each.)  Where some blocks are large they come first, and small ones fill the end.  (512 tokens over 4096
    // beside 23 single ones over 300 to 4096: 64 parts a head 113 us, 80 99, 96 108.)
    // Larger batches fill the device whole: of lengths that spread they lose nothing, but one long sequence among
    // short ones is then a single workgroup's for each key head.  (4 tokens each, e4m3, 8 key heads: 228
    // sequences of 300 to 4096 210 us divided, 229 188 whole; with one of 32768 among at most 300 93 and 483.  256
    // sequences on 2 key heads, one long: 58 us, 257: 917.)
    const int64_t round = 2 * cus, rounds = (found + found / 4 + round - 1) / round;
    // (up to 12.5 workgroups a compute unit; fewer of 256-wide heads, by their partials' bytes)
    const int64_t all = rounds * round * (p.filled > kWaveRows ? 5 : 4) / 4;
    p.shares = (int)((all < held ? all : held) / a.Hkv);
    p.splits = 1;
    p.per = (int)tiles;
    return p;
  }
  if (p.filled <= 64) {
    // Small blocks: a part takes its start and 1.3 us for each tile, or 1.7 for two of an e4m3 cache
    // (whose tiles four waves hold at once, not two), and a division the second kernel and 0.25 us for
    // each part that it joins.  (In us, 1 new token, 32 / 8 heads of 128 in bf16: over 777 in 7 parts 10.7; over
    // 1500 in 12 12.2, in 5 14.4; over 8000 in 14, 42 and 63 20.9, 22.3 and 25.0; over 256 whole 10.3, in 2
    // 10.1; over 384 13.0 and 10.2; in e4m3 over 448 whole 12.8, in 4 10.6.)  The rates are of heads of
    // 128, and serve the others: of 1 to 64 parts for 1 and 12 new tokens over 384 to 8000, in both types,
    // the choice is within 10 % of the best for heads of 64 (384 keys in 6 parts 10.1, whole 9.3), 6 % for 128,
    // and 13 % for 256 (12 tokens over 8000 in bf16 in 36 parts 33.7, in 32 29.9).
    const int64_t each = a.k_scale && p.filled <= kWaveRows ? 2 : 1;
    const double step = a.k_scale ? 1.7 : 1.3;
    double best = 0;
    for (int64_t s = 1; s == 1 || (s <= 64 && s <= tiles && s * found <= most); s++) {
      const int64_t per = (tiles + s - 1) / s, parts = found * s;
      const int64_t rounds = (parts + 2 * cus - 1) / (2 * cus);
      double us = rounds * (5 + (per + each - 1) / each * step);
      if (s > 1) us += 2.5 + s * 0.25;
      if (s == 1 || us < best) {
        best = us;
        splits = s;
      }
    }
  } else {
    // Large blocks: a tile takes a workgroup that has its compute unit alone about 0.7 of the time
    // that it takes two that share one; a part costs its start and its partials, and any division
    // the second kernel.  (In us, 32 / 8 heads of 128: 512 tokens over 4096 70 whole, 56 in 4 parts;
    // prompts of 500 and of 1000 tokens 22 and 36 in 4 and 2 parts, 18 and 30 whole; 20 tokens over 512
    // 16.9 whole, 11.4 in 4.)
    const int64_t real = a.B == 1 ? (rows + kBlockRows - 1) / kBlockRows : rows / kBlockRows + (a.B + 1) / 2;
    const double codes = a.k_scale ? 1.5 : 1.0;
    const double alone = codes * (a.D == 64 ? 0.9 : 1.5), pair = codes * (a.D == 64 ? 1.4 : a.D == 128 ? 2.1 : 2.3);
    // (of packed prompts only the sum of their lengths is known: twice the mean stands for the longest)
    const int64_t mean = 2 * (int64_t)a.T / a.B / tile + 1, usual = a.block_table || tiles < mean ? tiles : mean;
    double best = 0;
    for (int64_t s = 1; s == 1 || (s <= 64 && s <= tiles && s * found <= most); s++) {
      const int64_t per = (usual + s - 1) / s, parts = real * a.Hkv * s;
      const int64_t rounds = parts <= cus ? 1 : (parts + 2 * cus - 1) / (2 * cus);
      double us = rounds * (5 + per * (parts <= cus ? alone : pair));
      if (s > 1) us += 4 + s * 0.25 + parts * p.filled * (a.D + 2) * 8 / 8e6;
      if (s == 1 || us < best) {
        best = us;
        splits = s;
      }
    }
  }
  p.per = (int)((tiles + splits - 1) / splits);
  p.splits = (int)((tiles + p.per - 1) / p.per);
  return p;
}

}  // namespace fp8lin
