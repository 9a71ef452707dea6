// How the attention of paged_decode.hip divides a batch: the launch plan, which the
// host makes from sizes alone, and the layouts that the plan and the kernels share.
// Times are of one call of a replayed graph over three sets of inputs in turn, or of the
// kernel alone in a trace where that is said.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "launch_layer.hpp"

namespace fp8lin {

constexpr int kTile = 32;  // tokens of a wave's tile

__host__ __device__ inline int first_token(int len, int window) {
  const int lo = window > 0 && len > window ? len - window : 0;
  return lo & ~15;  // a half tile lies in one page
}

// How work is divided.  row_waves > 0: by the grid, `splits` workgroups of so
// many waves for each row, `per` tiles each (row_kernel).  Else in even shares: the
// rows of a sequence follow each other (bands of query heads within a key head),
// and wave i of 2^log2_parts takes units share_start(i) .. share_start(i + 1) - 1 of
// all.  A unit is a tile, and one more for the end of each row, which costs about as
// much (shares of equal tiles took the kernel 77 us on 64 sequences of 1 to 8192 tokens
// where sequences of equal length took 63).
struct DecodePlan {
  int row_waves, splits;
  int first_row;  // of a launch (splits == 1)
  int64_t per;
  int log2_parts;
  int owners;    // workgroups (row_kernel) or waves (shares): each has two slots for partials
  int64_t rows;  // of the batch
  bool by_row;   // whether the list of divided rows is indexed by row, or by share
};

__host__ __device__ inline int64_t share_start(int64_t i, int64_t total, int log2_parts) {
  const int64_t parts = (int64_t)1 << log2_parts;
  return total <= parts ? (i < total ? i : total) : i * total >> log2_parts;
}

// Partials of one part of a row: o [16 RT][D], then m and l [16 RT] each.
__host__ __device__ constexpr size_t part_floats(int D, int RT) { return (size_t)16 * RT * (D + 2); }

// LDS of a row_kernel workgroup, offsets in floats: o of each wave's heads, kHead floats
// each, then m and l.  o comes first because it is read and written 16 bytes at a time:
// behind the 8 n bytes of m and l it would start off 16 bytes for an odd n.
struct RowBox {
  int o, m, l, floats;
};
template <int D>
struct RowBoxOf {
  static constexpr int kHead = D + 4;  // off the bank period, whole 16 bytes
  static __host__ __device__ constexpr RowBox at(int waves, int heads) {
    const int n = waves * heads;
    return RowBox{0, n * kHead, n * kHead + n, n * (kHead + 2)};
  }
};

// Sets of 16 query heads that a row holds: two where a key head has more than 16,
// so that its lines are read once for up to 32 (not for D = 256, whose state of
// two sets leaves no registers for the tiles).
inline int row_tiles(const DecodeArgs &a) { return a.Hq / a.Hkv <= 16 || a.D == 256 ? 1 : 2; }

// Whether row_kernel exists for this many waves of a workgroup (a plan asks for no other).
constexpr bool has_row_form(int D, int RT, int waves) {
  return (waves == 1 && RT == 1) || waves == 2 || waves == 4 || (waves == 8 && D <= 128 && RT == 1);
}

// Workgroups of one row_kernel launch: a grid counts its threads in 32 bits.
constexpr int kRowGrid = 1 << 22;

inline DecodePlan plan_decode(const DecodeArgs &a, int cus) {
  int64_t tokens = a.max_len;  // live tokens of a sequence, from the tile that holds the first one
  if (a.window > 0 && tokens > (int64_t)a.window + 15) tokens = (int64_t)a.window + 15;
  const int64_t tiles = tokens <= kTile ? 1 : (tokens + kTile - 1) / kTile;
  const int wide = 16 * row_tiles(a);
  DecodePlan p{};
  p.rows = (int64_t)a.B * a.Hkv * ((a.Hq / a.Hkv + wide - 1) / wide);
  // Waves that are resident together; fewer where a wave's tiles would be few
  // beside the partials that it leaves (32 query heads on one key head of 128, 16
  // sequences of 4000 to 8000 tokens: 2048 waves 36 us, 1024 27 us).
  const int heads = a.Hq / a.Hkv < wide ? a.Hq / a.Hkv : wide;
  const int64_t resident = (a.D <= 128 ? 8 : 4) * cus, fed = p.rows * tiles * 8 / heads;
  const int64_t parts = resident < fed ? resident : fed > 512 ? fed : 512;
  // Short sequences: a workgroup for each row and no second kernel, while the longest
  // row takes one compute unit less time than dividing it costs; that is more when rows
  // fill the device.  A tile costs its bytes and as much as 4 KiB beside them.  Whole / divided
  // in us, by the longest row's tiles (32 query and 8 key heads; lengths from 1 on,
  // crowding at the short ones, so that a whole row of the longest stands out):
  //   of 128, bf16:  32 rows  8: 6.4 / 8.3, 16: 8.4 / 8.3, 24: 10.5 / 8.8
  //                 128 rows 16: 9.3 / 11.3, 24: 12.6 / 13.8, 32: 15.7 / 13.7
  //                 512 rows 24: 20.1 / 22.9, 32: 25.1 / 26.7, 48: 35.1 / 32.1
  //   of 64, e4m3:   32 rows 24: 6.6 / 7.3, 32: 7.4 / 7.5, 48: 9.2 / 7.9
  //                 256 rows 32: 8.8 / 12, 64: 12.9 / 16.4
  //   of 256, bf16:  32 rows  8: 9.4 / 10.2, 16: 14.4 / 11.1
  //                 256 rows 16: 20.3 / 20.2, 24: 27.4 / 24.5
  const int tile_kb = 2 * kTile * a.D * (a.k_scale ? 1 : 2) / 1024;
  const bool small = tiles * (tile_kb + 4) <= (p.rows < 64            ? 256
                                               : p.rows < cus / 2     ? 336
                                               : p.rows < cus / 4 * 3 ? 448
                                                                      : 640);
  // The grid divides rows as if all were as long as the longest: no search, and one
  // join of parts of a workgroup.  That is faster while a wave has a few tiles, and
  // for windows, which make rows alike; ragged batches of more take even shares.
  // (bf16, up to 2000 tokens: 8 equal sequences 17.0 us by the grid, 20.4 by shares,
  // 8 of 100 on 13.9 / 16.5; up to 8000: 4 equal 26.4 / 31.1, 4 of 500 on 20.6 /
  // 22.0, 8 of 500 on 32 / 28; a window of 1024 in 37 of 5 to 6000 22.6 / 26.7, of
  // 4096 in 32 of 4000 to 9000 84 / 100, of 100 to 9000 65 / 64.)
  const bool alike = a.window > 0 && a.window < a.max_len;
  if (small || a.B == 1 || p.rows * tiles <= (alike ? 32 : 4) * parts) {
    // more waves of a workgroup join through LDS where rows have work for them: 4000
    // tokens of one sequence 9.8 us with four and 11.0 with eight, 131072 89.3 / 88.1
    // (short: 512 rows of 8 to 48 tiles 9.8 to 33.8 us with eight, 8.9 to 33.0 with four; but windows
    // of 1024 in 592 rows of 64 22.4 / 25.6, in 1024 rows of 128 75.6 / 78.1).
    const bool few = small && (!alike || tiles <= 16);
    p.row_waves = a.D <= 128 && wide == 16 && (few ? p.rows <= cus : p.rows * tiles > parts) ? 8 : 4;
    // no waves without a tile: 200 sequences of up to 30 tokens 11.2 us with four, 8.1 with one;
    // but for three tiles four in few rows (8 rows 4.7 / 5.0 with two, 256 5.5 / 6.1, 1024 of 256
    // 21.3 / 19.4), and two that write 32 heads (16 rows of 18 tokens 7.4, with one 8.2)
    while (p.row_waves > (p.rows <= cus ? 2 * tiles - 1 : tiles) * (wide / 16)) p.row_waves /= 2;
    p.per = small ? tiles : p.row_waves * ((p.rows * tiles + parts - 1) / parts);
    p.splits = (int)((tiles + p.per - 1) / p.per);
    p.owners = (int)(p.rows * p.splits);
    p.by_row = p.splits > 1;
    return p;
  }
  while ((int64_t)3 << p.log2_parts <= 2 * parts) p.log2_parts++;  // the nearest power of two
  p.owners = 1 << p.log2_parts;
  p.by_row = p.rows <= p.owners;
  return p;
}

}  // namespace fp8lin
