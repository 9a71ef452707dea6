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
struct PromptPlan {
  int splits, per;
  int blocks;
  int first;  // workgroup of the whole grid that a launch begins at
};

// Workgroups of one launch: a grid counts its threads in 32 bits.
constexpr int kPromptGrid = 1 << 22;

// Number of the first block of a sequence whose first token is `start`: at least as many
// numbers lie between two sequences' as the first one's rows need.
__host__ __device__ inline int64_t first_block(int64_t start, int64_t b, int group) {
  return start * group / kBlockRows + b;
}

// Partials of one part of a block: o [kBlockRows][D], then m and l [kBlockRows] each.
__host__ __device__ constexpr size_t prompt_part_floats(int D) { return (size_t)kBlockRows * (D + 2); }

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
  const int64_t resident = (int64_t)cus * 2, found = (int64_t)p.blocks * a.Hkv;
  const int64_t filled = rows / p.blocks;  // rows of a block
  const int64_t parts = resident * (filled <= 32 ? 4 : filled <= 64 ? 2 : 1);
  int64_t splits = 4 * found > 3 * parts ? 1 : (parts + found - 1) / found;
  if (splits > tiles / 2) splits = tiles / 2;
  if (splits < 1) splits = 1;
  p.per = (int)((tiles + splits - 1) / splits);
  p.splits = (int)((tiles + p.per - 1) / p.per);
  return p;
}

}  // namespace fp8lin
