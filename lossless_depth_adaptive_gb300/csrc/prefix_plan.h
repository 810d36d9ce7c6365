// What a shared-prefix attention call launches and where its parts lie in the workspace: from sizes alone, on the
// host (no device code, so that a test can compile it by itself).
#pragma once

#include <stddef.h>
#include <stdint.h>

#include "kernels.h"

#ifdef __CUDACC__
#define DEX_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define DEX_HOST_DEVICE inline
#endif

namespace dex {

constexpr int kRowsTile = 64;     // keys of a tile of rows_kernel
constexpr int kRowsUnit = 16;     // its query rows come in m16 tiles
constexpr int kRowsMax = 32;      // and at most this many
constexpr int kRowsSlotRows = 64; // rows of the segments posted ahead
constexpr int kRowsPerSm = 2;     // resident CTAs
constexpr int kSms = 152;         // of the sm_103 part: workspace sizes and grids, whatever device is current
constexpr int kTileRows = 256;    // query rows of a segment of tile_kernel (two tiles of 128)
constexpr int kQueueBytes = 16;   // state of a queue of ranges
constexpr int kRowsQueue = 2;     // ranges per CTA of rows_kernel where it takes several

// Parts of a row that a segment's entry (first and last range) stands for, none where it is not one that the kernel
// of `ranges` ranges can have written: a kernel that gave up waiting leaves entries that hold anything, and the
// workspace has room for the parts of those ranges alone.
DEX_HOST_DEVICE int parts_in(int first, int last, int ranges) {
  return first >= 0 && first <= last && last < ranges ? last - first + 1 : 0;
}

struct Plan {
  bool share, prefix_tile, own_tile;   // prefix / own segments on tile_kernel
  int rows_mt;                         // row tiles of rows_kernel: 1 or 2 (0: it has nothing to do)
  int slots;
  bool queue() const { return prefix_tile && !own_tile; }   // rows_kernel behind tile_kernel
  int rows_per_cta() const { return queue() || (share && !prefix_tile) ? kRowsQueue : 1; }
  int rows_ranges() const { return rows_per_cta() * kRowsPerSm * kSms; }
  size_t o_queue, o_rows_part, o_rows_ml, o_tile_part, o_tile_ml, o_pre, o_pre_ml, o_own, o_own_ml, o_pre_info, o_own_info, total;
  int own_rt() const { return own_tile ? kTileRows : rows_mt * kRowsUnit; }
  int pre_rt() const { return prefix_tile ? kTileRows : rows_mt * kRowsUnit; }
  int own_ranges() const { return own_tile ? kSms : rows_ranges(); }
  int pre_ranges() const { return prefix_tile ? kSms : rows_ranges(); }
};

// Which kernel computes what.  Segments of at most 32 rows go to rows_kernel, unless tile_kernel runs for the prefix
// and there are few of them: a launch less (14 sequences of 8 K/V heads behind 27032 positions 46.5 -> 41.7 us; for
// 36 of 8 behind 938 it would be 22.0 -> 28.3).  They are counted by the table's slots, used or not: 14 sequences in 64
// slots 53.2 us, with own_tile 51.7; 16 in 128 slots behind 4096 25.6, with own_tile 27.5.  With 16 rows as the limit, 8 x 8 segments of 32 prefix rows take
// 23.4 us instead of 14.9, 32 of 32 rows 48.9 instead of 41.8.
// Sharing costs a join of two parts of every row and mostly a launch, and saves reading the prefix for each sequence.
// So it is shared when more than one sequence can have queries (n_tokens > max_q) and reading it for all of
// them would give every CTA of rows_kernel three key tiles: at 624 tiles in all (13 sequences of 4 heads behind 777
// positions) it takes 13.2 us shared and 12.2 not, at 1188 (9 of 4 behind 2158) 10.4 and 12.6, at 2048 (8 of 8
// behind 2048) 13.1 and 16.3.  A prefix below two tiles is not shared (73 positions, 202 sequences of 8 heads: 83 us
// shared, 70 not).  A sequence whose own rows fill a 128-row tile gains nothing from sharing, and the longest run
// decides for the batch: where its rows can fill one, nothing is shared.  That is right for batches of such runs and
// costs batches with one of them what sharing would have saved for the others (63 single tokens of 32 / 8 heads and a
// run of 31 behind 8192 positions 83 us, and a run of 32 294; the single tokens alone 49, the run 19).
inline Plan make_plan(const PrefixAttnArgs& a) {
  Plan p = {};
  const int64_t own_rows = static_cast<int64_t>(a.max_q) * a.G, all_rows = static_cast<int64_t>(a.n_tokens) * a.G;
  const int64_t readers = a.n_tokens < a.kv.batch ? a.n_tokens : a.kv.batch;
  p.share = a.prefix_len >= 2 * kRowsTile && a.n_tokens > a.max_q && own_rows < 128 &&
            readers * a.kv.KVH * (a.prefix_len / kRowsTile) >= 3 * kRowsPerSm * kSms;
  p.prefix_tile = p.share && all_rows > kRowsMax;
  p.own_tile = own_rows > kRowsMax || (p.prefix_tile && a.kv.batch * a.kv.KVH <= kSms);
  const int64_t most = p.share && !p.prefix_tile ? all_rows : p.own_tile ? 0 : own_rows;   // rows of a rows_kernel segment
  p.rows_mt = most == 0 ? 0 : most <= kRowsUnit ? 1 : kRowsMax / kRowsUnit;
  p.slots = most == 0 ? 1 : static_cast<int>(kRowsSlotRows / ((most + kRowsUnit - 1) / kRowsUnit * kRowsUnit));
  auto up = [](size_t x) { return (x + 255) & ~size_t(255); };
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = up(at + bytes);
    return o;
  };
  const size_t hd4 = static_cast<size_t>(a.kv.hd) * 4;
  if (p.rows_mt) {
    if (p.queue()) p.o_queue = take(kQueueBytes);
    p.o_rows_part = take(size_t(2) * p.rows_ranges() * p.rows_mt * kRowsUnit * hd4);
    p.o_rows_ml = take(size_t(2) * p.rows_ranges() * p.rows_mt * kRowsUnit * 8);
  }
  if (p.own_tile || p.prefix_tile) {
    p.o_tile_part = take(size_t(2) * kSms * kTileRows * hd4);
    p.o_tile_ml = take(size_t(2) * kSms * kTileRows * 8);
  }
  const size_t all = static_cast<size_t>(a.n_tokens) * a.H;
  if (p.share) {
    p.o_pre = take(all * hd4);
    p.o_pre_ml = take(all * 8);
    p.o_own = take(all * hd4);
    p.o_own_ml = take(all * 8);
    p.o_pre_info = take((all_rows / p.pre_rt() + 1) * a.kv.KVH * 8);
  }
  p.o_own_info = take((all_rows / p.own_rt() + own_rows / p.own_rt() + a.kv.batch + 2) * a.kv.KVH * 8);
  p.total = at;
  return p;
}

}  // namespace dex
