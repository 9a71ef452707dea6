// How the attention of prompt_attention.hip divides a batch: the launch plan, which the
// host makes from sizes alone.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "launch_layer.hpp"

namespace fp8lin {

constexpr int kWaveRows = 32;  // rows of a wave; a row is a token and a query head of one key head

// Keys of a tile.
constexpr int prompt_tile_keys(int D) { return D == 256 ? 32 : 64; }

// A block of 32 `waves` rows of one sequence and key head is a workgroup, or `splits` of
// them that take `per` key tiles each and leave partials.  Blocks are numbered through the
// batch: sequence b has numbers first_block(b) .. first_block(b + 1) - 1, some unused.
struct PromptPlan {
  int waves, splits, per;
  int blocks;
  int first;  // workgroup of the whole grid that a launch begins at
};

// Workgroups of one launch: a grid counts its threads in 32 bits.
constexpr int kPromptGrid = 1 << 22;

// Number of the first block of a sequence whose first token is `start`: at least as many
// numbers lie between two sequences' as the first one's rows need.
__host__ __device__ inline int64_t first_block(int64_t start, int64_t b, int group, int block_rows) {
  return start * group / block_rows + b;
}

constexpr size_t prompt_part_floats(int D, int waves) { return (size_t)waves * kWaveRows * (D + 2); }

inline PromptPlan plan_prompt(const PromptArgs &a, int cus) {
  const int group = a.Hq / a.Hkv;
  const int64_t rows = (int64_t)a.T * group;  // of a key head
  PromptPlan p{};
  p.waves = 1;
  while (p.waves < 4 && rows > (int64_t)a.B * p.waves * kWaveRows) p.waves *= 2;
  p.blocks = (int)first_block(a.T, a.B, group, p.waves * kWaveRows);
  int64_t keys = a.max_len;
  const int64_t seen = (int64_t)a.window + (p.waves * kWaveRows + group - 1) / group + 15;
  if (a.window > 0 && keys > seen) keys = seen;
  const int tile = prompt_tile_keys(a.D);
  const int64_t tiles = keys <= tile ? 1 : (keys + tile - 1) / tile;
  const int64_t resident = (int64_t)cus * 8 / p.waves, found = (int64_t)p.blocks * a.Hkv;
  int64_t splits = found >= resident ? 1 : resident / found;
  if (splits > tiles / 2) splits = tiles / 2 < 1 ? 1 : tiles / 2;
  p.per = (int)((tiles + splits - 1) / splits);
  p.splits = (int)((tiles + p.per - 1) / p.per);
  return p;
}

}  // namespace fp8lin
