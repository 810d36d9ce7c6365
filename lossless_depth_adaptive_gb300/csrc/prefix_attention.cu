// Attention of a ragged batch of queries over a paged K/V cache whose sequences share a prefix.
//
//   o_i = sum_j softmax_j(scale q_i . k_j) v_j        over the keys j that query i sees
//
// The softmax over a set of keys is carried as (m, l, O): the largest score, the sum of
// exp2(c (s - m)) and the sum of exp2(c (s - m)) v, with scores s before the scale and c = scale log2(e), taken
// positive (a negative scale turns the scores' sign).  Two disjoint key sets join as m = max(m1, m2),
// x = x1 2^(c (m1-m)) + x2 2^(c (m2-m)), so any split of a query's keys over CTAs gives the same result.  The
// scale comes after the difference because the difference of near scores is exact, whatever their size; rounded
// products s c are off by half the distance of fp32 neighbours, from 2^27 on by powers of 2^8.
//
// A *segment* is a set of query rows of one K/V head that reads the same keys:
//  * prefix segment: rows of all sequences (token-major, the G query heads of the K/V head
//    next to each other) against the shared positions [0, prefix_len) -- each key is read once
//    for up to 256 rows;
//  * own segment: rows of one sequence against its positions from prefix_len on (from 0 when
//    nothing is shared).
// Key tiles of all segments are laid end to end, each segment behind a few units that stand for what it
// costs beside its tiles, and cut into equal contiguous ranges, one per CTA of a persistent grid (or two, from a
// queue), so lengths need no plan on the host and any mix of lengths balances.
// A segment that lies in one range is finished there; one that is cut leaves a partial (m, l, O) per
// range, and combine_kernel joins the parts of each row in a fixed order (no atomics: the same
// lengths give the same bits).
//
// Two kernels compute segments:
//  * rows_kernel (at most 32 rows: single tokens, a few lattice nodes): the keys are the work, so it is a
//    stream of K and V through a TMA ring into m16n8k16 MMAs on register fragments;
//  * tile_kernel (up to 256 rows): 5th-generation tensor cores, two 128-row tiles per CTA that
//    share every K and V tile.
#include <math.h>

#include <atomic>
#include <type_traits>

#include "../../include/dex.h"
#include "common.cuh"
#include "kernels.h"
#include "prefix_plan.h"

namespace dex {

namespace {

constexpr int kRowsWarps = 4;     // compute warps
constexpr int kRowsThreads = 32 * (kRowsWarps + 1);
constexpr int kTileKeys = 128;    // keys of a tile of tile_kernel
// What a segment costs a CTA beside its key tiles, in tiles (queries, start and end of its pipeline, result);
// kTileHalfCost where the teams of tile_kernel share its rows.  With no cost 64 sequences behind 8192 positions take
// 60 us instead of 46 (some CTAs get seven segments of one tile), 32 of 32 heads 45.5 instead of 42; with two tiles
// in rows_kernel the latter 46; with two instead of four in tile_kernel 256 sequences behind 32768 162 instead of
// 158; with four for half segments too 16 lattices behind 4096 31.1 instead of 28.6, with one 34.7.
constexpr int kRowsSegCost = 1, kTileSegCost = 4, kTileHalfCost = 2;
// Units (tiles and these costs) of a range, at least.  Few long ranges leave SMs idle: 8 tokens behind 2048 positions
// take 12.9 us with two units, 14.3 with three; 13 sequences behind 777 on tile_kernel 13.2 with one, 15.0 with
// three.  Two units of rows_kernel hold a tile.
constexpr int kRowsMinUnits = kRowsSegCost + 1, kTileMinUnits = 1;
// Where tile_kernel computes the prefix and rows_kernel the rest, they run side by side: tile_kernel takes SMs in
// proportion to the work, a unit of it counted as kTileWeight of rows_kernel's, and rows_kernel's CTAs, those on
// the other SMs from the start and those that follow on its SMs, take kRowsQueue ranges each on average from a
// queue.  64 sequences behind 8192 positions and 256 behind 32768: 37.7 and 144.8 us; weight 4 41.5 and 149.7, 6
// 39.2 and 146.9; with a fixed range per CTA and all SMs for tile_kernel first 44.7 and 151.9; four ranges per CTA
// 40.9 and 145.3, one (at weight 6) 40.6 and 156.
// Where rows_kernel computes both, its CTAs take two ranges in turn, so that each has prefix segments, whose tiles
// cost more, and own ones: 32 sequences of 32 heads behind 4096 positions 40.2 us, with one range 42.2, with three
// 41.9.  Below kRowsTwo units per CTA it is one range (3 sequences of 4 heads behind 12815, three units per CTA:
// 10.9 us, with two 12.5).
constexpr float kTileWeight = 5.0f;
constexpr uint32_t kRowsTwo = 8;
constexpr int kMaxBatch = 1024;
static_assert(kRowsPerSm * kSms <= 0x3ff, "CTAs in the gate of a queue");

// Division by a number fixed for the call: n / d for 0 <= n < 2^31 (multiply, add, shift).
struct FastDiv {
  uint32_t d, mul, shift;
  FastDiv() = default;
  explicit FastDiv(uint32_t div) : d(div), shift(0) {
    while ((uint64_t(1) << shift) < d) ++shift;
    mul = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << shift) - d)) / d + 1);
  }
  __device__ __forceinline__ int div(int n) const {
    return static_cast<int>((__umulhi(static_cast<uint32_t>(n), mul) + static_cast<uint32_t>(n)) >> shift);
  }
};

// Ranges of a rows_kernel behind tile_kernel, which opens the queue for it.
struct RangeQueue {
  uint32_t next;   // next range to take
  uint32_t pad;
  uint64_t gate;   // kGate + CTAs of rows_kernel that start beside tile_kernel; anything else: not open (yet)
};
static_assert(sizeof(RangeQueue) == kQueueBytes, "workspace of the queue");
// rows_kernel can run before tile_kernel ends, so no kernel boundary makes `next` visible to it.  It takes the gate's
// word by an acquiring load, tile_kernel stores it by a releasing one, and the join, which runs when both have ended,
// takes it back for the next call.  A workspace's first bytes before its first call hold it once in 2^54.
constexpr uint64_t kGate = 0x5bd1e9a74c36f800ull, kGateCtas = 0x3ffull;
__device__ __forceinline__ uint64_t load_acquire(const uint64_t* p) {
  uint64_t v;
  asm volatile("ld.acquire.gpu.global.u64 %0, [%1];" : "=l"(v) : "l"(p) : "memory");
  return v;
}
__device__ __forceinline__ void store_release(uint64_t* p, uint64_t v) {
  asm volatile("st.release.gpu.global.u64 [%0], %1;" ::"l"(p), "l"(v) : "memory");
}

// What one of the two kernels has to do in a call.
struct SegWork {
  PrefixAttnArgs a;
  FastDiv by_g, by_kvh; // query heads per K/V head, K/V heads
  int32_t first;        // 1: the call's first kernel (it waits for what precedes the call)
  int32_t share;        // 1: positions below prefix_len belong to prefix segments
  int32_t do_prefix;    // this kernel computes the prefix segments
  int32_t do_own;       // this kernel computes the own segments
  int32_t joined;       // 1: rows have prefix and own parts, so a finished segment is not yet the output
  int32_t slots;        // rows_kernel: segments posted ahead
  int32_t per_cta;      // rows_kernel: ranges per CTA, at most
  int32_t behind_rt;    // tile_kernel: rows per segment of the rows_kernel behind it (it computes the own segments), or 0
  RangeQueue* queue;    // rows_kernel behind tile_kernel, or null: CTA i takes range i
  float* part_o;        // parts of cut segments, two per range: [2 * ranges][hd / 4][rows][4]
  float2* part_ml;      // [2 * ranges][rows] (m, l)
  float* pre_o;         // finished prefix segments (joined): [KVH][hd / 4][n_tokens * G][4]
  float2* pre_ml;       // [KVH][n_tokens * G]
  float* own_o;         // the same of own segments
  float2* own_ml;
  int2* pre_info;       // [prefix segments] first and last range
  int2* own_info;       // [own segments]
};

template <typename T> struct Half2Of;
template <> struct Half2Of<__nv_bfloat16> { using type = __nv_bfloat162; };
template <> struct Half2Of<__half> { using type = __half2; };

template <typename T>
__device__ __forceinline__ uint32_t pack2(float x, float y) {   // x in the low half
  typename Half2Of<T>::type v;
  if constexpr (std::is_same<T, __half>::value) v = __floats2half2_rn(x, y);
  else v = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// Probabilities go to the tensor cores in 16 bits, one number each: off by half a step, 2^-8 in bf16 and 2^-11 in
// fp16, which is chosen over a pair of numbers (2^-16 and less) because that takes twice the products with V: against
// 64 bits results are off by 0.0021-0.0024 (bf16) and 0.00027-0.00029 (fp16) of their size, of which their own
// rounding is 0.0017 and 0.00021.  In fp16 half a step is 2^-11 of a number down to 2^-14 only.  So fp16
// probabilities are exp2(c (s - m) + kUp), a factor that O and l share, and m, otherwise the largest score so far,
// comes down to that of a key tile which stays kDrop and more below it: the weights of a tile are rounded relative to
// the tile's own, not to one key's far above (with values near zero there, what an attention sink is, the others' sum
// is the result).  kDeep bounds the way down, so that fp32 holds what the far key's weight is then.  In rows_kernel
// that takes 42.0 us instead of 41.0 for 32 sequences of 32 heads behind 4096 positions, in tile_kernel nothing that
// shows.
template <typename T> constexpr bool kIsHalf = std::is_same<T, __half>::value;
template <typename T> constexpr float kUp = kIsHalf<T> ? 7.0f : 0.0f;
constexpr float kDrop = 10.0f, kDeep = 60.0f;
// lse of a row: log of the sum that (m, l) stand for
template <typename T>
__device__ __forceinline__ float log_sum(float m, float l, float c) {
  return isnan(l) ? l : l > 0.0f ? (m * c + (log2f(l) - kUp<T>)) * 0.6931471805599453f : -INFINITY;
}
// c of the scores; a zero scale zeroes them instead.
__device__ __forceinline__ float score_scale(const PrefixAttnArgs& a) {
  return a.scale_log2 == 0.0f ? 1.0f : fabsf(a.scale_log2);
}
__device__ __forceinline__ float quiet_nan() { return __int_as_float(0x7fffffff); }

// Where the (m, l, O) of one row of a part lies: four head dims at o, the next four `step` floats on.
struct PartRef {
  float* o;
  int64_t step;
  float2* ml;
};
template <int HD>
__device__ __forceinline__ PartRef slot_part(float* part_o, float2* part_ml, int slot, int rows, int r) {
  return PartRef{part_o + (static_cast<int64_t>(slot) * (HD / 4) * rows + r) * 4, static_cast<int64_t>(rows) * 4,
                 part_ml + static_cast<int64_t>(slot) * rows + r};
}
template <int HD>
__device__ __forceinline__ PartRef joined_part(float* o, float2* ml, int kvh, int rows_all, int rg) {
  return PartRef{o + (static_cast<int64_t>(kvh) * (HD / 4) * rows_all + rg) * 4, static_cast<int64_t>(rows_all) * 4,
                 ml + static_cast<int64_t>(kvh) * rows_all + rg};
}

// ---- segments ------------------------------------------------------------------------------
struct SeqRef {
  int q0, n, len;
  bool valid;   // has queries, and they are in range
  bool bad;     // length out of range: rows are poisoned
};
// Lengths and tables are read by plain loads: a kernel here can be resident before the kernel that writes them
// ends (programmatic launches), so they are not read-only for its lifetime.
__device__ __forceinline__ SeqRef seq_ref(const PrefixAttnArgs& a, int b, bool* report = nullptr) {
  SeqRef s;
  s.q0 = a.q_start[b];
  const int q1 = a.q_start[b + 1];
  s.len = a.seq_len[b];
  const bool range = s.q0 >= 0 && q1 >= s.q0 && q1 <= a.n_tokens && q1 - s.q0 <= a.max_q;
  s.n = range ? q1 - s.q0 : 0;
  s.valid = s.n > 0;
  s.bad = s.len < 0 || s.len > (a.kv.table_width << a.kv.page_shift);
  if (report) *report = !range || s.bad;
  if (s.bad) s.len = 0;
  return s;
}

// Keys [lo, hi) of a sequence's own segment of rows [r0, r1) and its tiles.
struct KeyRange {
  int lo, hi, t0, nt;
};
template <int TILE>
__device__ __forceinline__ KeyRange own_range(const SegWork& w, const SeqRef& s, int r1) {
  KeyRange k;
  k.lo = w.share ? w.a.prefix_len : 0;
  const int last = s.len - s.n + w.by_g.div(r1 - 1);   // position of the last query
  k.hi = s.bad ? 0 : w.a.tree ? s.len : min(max(0, last + 1), s.len);
  k.t0 = k.lo / TILE;
  k.nt = k.hi > k.lo ? (k.hi + TILE - 1) / TILE - k.t0 : 0;
  if (k.nt == 0) {
    k.hi = k.lo;
    // someone has to write the row: an empty tile, unless the prefix part covers it
    if (!w.share || s.bad) k.nt = 1;
  }
  return k;
}

// Index of an own segment's entry in own_info: distinct for the row tiles of sequences in order.
__device__ __forceinline__ int own_info_of(const PrefixAttnArgs& a, int RT, int q0, int b, int rt, int kvh) {
  return (static_cast<int>(static_cast<uint32_t>(q0 * a.G) / static_cast<uint32_t>(RT)) + b + rt) * a.kv.KVH + kvh;
}

// The part of a segment that a CTA's range of units covers.
struct Piece {
  int tile, cnt;      // first key tile, number of tiles (none where the range ends before the first)
  uint32_t units;
  bool starts, ends;  // it holds the segment's first, last tile
};

// The segment that holds a unit, and the walk to the next one.  A segment is its cost (COST units, fewer where its rows
// are half a tile_kernel's) followed by its key tiles.  Lengths that change under a call (a caller's mistake) make
// its results wrong, but no loop endless and no index leave its array: each read of a sequence is checked, and the
// walk ends within the batch.
template <int RT, int TILE, int COST>
struct Walker {
  const SegWork& w;
  int n_pre, pre_nt, pre_cost;   // prefix segments of this kernel, their tiles and cost
  // current segment
  bool prefix;
  int seg, b, rt, kvh, rows, r0, cost;   // seg: prefix segment index; r0: first row within the sequence / batch
  SeqRef s;
  KeyRange k;

  __device__ __forceinline__ explicit Walker(const SegWork& work) : w(work) {
    const int pre_rows = w.a.n_tokens * w.a.G;
    n_pre = w.do_prefix ? (pre_rows + RT - 1) / RT * w.a.kv.KVH : 0;
    pre_nt = (w.a.prefix_len + TILE - 1) / TILE;
    pre_cost = cost_of(pre_rows);
  }
  __device__ __forceinline__ static int cost_of(int rows) { return RT == kTileRows && rows <= kTileRows / 2 ? kTileHalfCost : COST; }
  __device__ __forceinline__ static uint32_t units(int nt, int cost) { return nt > 0 ? static_cast<uint32_t>(nt + cost) : 0u; }
  __device__ __forceinline__ uint32_t units() const { return units(k.nt, cost); }
  __device__ __forceinline__ uint32_t pre_units() const { return static_cast<uint32_t>(n_pre) * units(pre_nt, pre_cost); }
  // units of one K/V head over the row tiles of sequence b
  __device__ __forceinline__ uint32_t seq_units(const SeqRef& q) const {
    if (!q.valid) return 0;
    uint32_t n = 0;
    for (int r = 0; r < q.n * w.a.G; r += RT) {
      const int end = min(r + RT, q.n * w.a.G);
      n += units(own_range<TILE>(w, q, end).nt, cost_of(end - r));
    }
    return n;
  }
  // The part of the segment from unit `off` on that `left` more units cover.
  __device__ __forceinline__ Piece piece(int off, uint32_t left) const {
    Piece p;
    p.units = min(units() - static_cast<uint32_t>(off), left);
    p.tile = max(off - cost, 0);
    p.cnt = max(off + static_cast<int>(p.units) - cost, 0) - p.tile;
    p.starts = p.tile == 0;
    p.ends = p.tile + p.cnt == k.nt;
    return p;
  }
  __device__ __forceinline__ void set_prefix(int index) {
    prefix = true;
    seg = index;
    rt = w.by_kvh.div(index);
    kvh = index - rt * w.a.kv.KVH;
    r0 = rt * RT;
    rows = min(RT, w.a.n_tokens * w.a.G - r0);
    k = KeyRange{0, w.a.prefix_len, 0, pre_nt};
    cost = pre_cost;
  }
  __device__ __forceinline__ void set_own() {
    prefix = false;
    r0 = rt * RT;
    rows = min(RT, s.n * w.a.G - r0);
    k = own_range<TILE>(w, s, max(r0 + rows, 1));
    cost = cost_of(rows);
  }
  // Segment of unit g (cum[b]: own units of all K/V heads before sequence b); returns the unit within it.
  __device__ __forceinline__ int find(uint32_t g, const uint32_t* cum) {
    if (g < pre_units()) {
      set_prefix(static_cast<int>(g / units(pre_nt, pre_cost)));
      return static_cast<int>(g % units());
    }
    g -= pre_units();
    int lo = 0, hi = w.a.kv.batch - 1;
    while (lo < hi) {   // last b with cum[b] <= g: a sequence with units, since the total is beyond g
      const int mid = (lo + hi + 1) >> 1;
      if (cum[mid] <= g) lo = mid;
      else hi = mid - 1;
    }
    b = lo;
    g -= cum[lo];
    s = seq_ref(w.a, b);
    for (rt = 0;; ++rt) {
      set_own();
      const uint32_t cnt = units() * static_cast<uint32_t>(w.a.kv.KVH);
      if (g < cnt || (rt + 1) * RT >= s.n * w.a.G) break;
      g -= cnt;
    }
    const uint32_t each = max(units(), 1u);
    kvh = min(static_cast<int>(g / each), w.a.kv.KVH - 1);
    return static_cast<int>(g % each);
  }
  // The next segment that has tiles (the caller knows that there is one).
  __device__ __forceinline__ void next() {
    if (prefix) {
      if (seg + 1 < n_pre) {
        set_prefix(seg + 1);
        return;
      }
      b = -1;
    } else {
      if (++kvh < w.a.kv.KVH) return;
      kvh = 0;
      while ((rt + 1) * RT < s.n * w.a.G) {
        ++rt;
        set_own();
        if (k.nt > 0) return;
      }
    }
    kvh = 0;
    while (++b < w.a.kv.batch) {
      s = seq_ref(w.a, b);
      if (!s.valid) continue;
      for (rt = 0; rt * RT < s.n * w.a.G; ++rt) {
        set_own();
        if (k.nt > 0) return;
      }
    }
    b = w.a.kv.batch - 1;
  }
  // Token and query head of row r of the segment.
  __device__ __forceinline__ void row_of(int r, int& t, int& h) const {
    const int i = w.by_g.div(r0 + r);
    t = (prefix ? 0 : s.q0) + i;
    h = kvh * w.a.G + r0 + r - i * w.a.G;
  }
  __device__ __forceinline__ int own_info_index() const { return own_info_of(w.a, RT, s.q0, b, rt, kvh); }
};

// The sequence whose queries can hold token t: the last b with q_start[b] <= t.
__device__ __forceinline__ int seq_of_token(const PrefixAttnArgs& a, int t) {
  int lo = 0, hi = a.kv.batch - 1;
  // with one query per sequence it is t itself: two loads instead of a chain of them
  if (t <= hi && a.q_start[t] <= t && (t == hi || a.q_start[t + 1] > t)) return t;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (a.q_start[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Which keys a row sees: j in [lo, hi), and j <= last or (tree) bit j - first of the word.
struct RowView {
  int last;        // causal: the row's position; tree: the last key before the queries' own
  int first;       // tree: position of the first query
  uint64_t word;
  bool owned;      // the row belongs to a sequence (its result is written)
};
__device__ __forceinline__ RowView row_view(const PrefixAttnArgs& a, const SeqRef& s, int t) {
  RowView v;
  v.owned = s.valid && t >= s.q0 && t < s.q0 + s.n;
  v.first = s.len - s.n;
  // bits from the sequence's number of queries on name nothing: in a prefix segment, which ends behind a shorter
  // sequence, they would be positions that it does not have
  v.word = a.tree && v.owned ? a.tree[t] & (~0ull >> (64 - min(s.n, 64))) : 0ull;
  v.last = a.tree ? v.first - 1 : v.first + (t - s.q0);
  if (s.bad) v.last = -1, v.word = 0;
  if (!v.owned) v.last = 0x7fffffff;   // its result is not used: no reason to mask
  return v;
}

// Which of the 32 keys from `at` on a row sees, within [lo, hi).
__device__ __forceinline__ uint32_t range_bits(int from, int to) {   // bits from .. to - 1 of a word
  from = max(from, 0);
  to = min(to, 32);
  if (to <= from) return 0u;
  return (0xffffffffu >> (32 - (to - from))) << from;
}
__device__ __forceinline__ uint32_t seen_bits(const RowView& v, int lo, int hi, int at) {
  uint32_t bits = range_bits(0, v.last >= at + 31 ? 32 : v.last - at + 1);
  if (v.word) {
    const int sh = v.first - at;   // column of the first query's position
    if (sh >= 0) bits |= sh < 32 ? static_cast<uint32_t>(v.word << sh) : 0u;
    else if (sh > -64) bits |= static_cast<uint32_t>(v.word >> -sh);
  }
  return bits & range_bits(lo - at, hi - at);
}

// Whether a row sees one of the keys [lo, hi) whose page in the table has an id out of range.  Asked only where a
// segment has met such a page: its keys and values are zeros there, so the rows that do not see it are right.
__device__ __forceinline__ bool sees_bad_page(const PagedKv& kv, const int32_t* table, RowView v, int lo, int hi) {
  for (int entry = lo >> kv.page_shift; (entry << kv.page_shift) < hi; ++entry) {
    const int id = table[entry];
    if (id >= 0 && id < kv.n_pages) continue;
    const int begin = max(lo, entry << kv.page_shift), end = min(hi, (entry + 1) << kv.page_shift);
    for (int at = begin; at < end; at += 32)
      if (seen_bits(v, begin, end, at)) return true;
  }
  return false;
}

// Own units of every sequence, as running totals in cum[0 .. batch]; the block's threads together.
// scratch: a word per warp.  token_seq (at most 64 tokens, or null) receives each token's sequence.
// Returns the total number of units of the kernel.
template <int THREADS, typename W>
__device__ __forceinline__ uint32_t count_units(const W& wk, uint32_t* cum, uint32_t* scratch,
                                                int* token_seq = nullptr) {
  const SegWork& w = wk.w;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, B = w.do_own ? w.a.kv.batch : 0;
  uint32_t base = 0;
  for (int b0 = 0; b0 < B; b0 += THREADS) {
    const int b = b0 + tid;
    uint32_t n = 0;
    if (b < B) {
      bool report;
      const SeqRef s = seq_ref(w.a, b, &report);
      n = wk.seq_units(s) * static_cast<uint32_t>(w.a.kv.KVH);
      if (token_seq)
        for (int i = 0; i < s.n; ++i) token_seq[s.q0 + i] = b;
      if (report && blockIdx.x == 0 && w.a.status) atomicOr(w.a.status, DEX_ATTN_BAD_RANGE);
    }
    uint32_t x = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) scratch[warp] = x;
    __syncthreads();
    uint32_t before = base;
    for (int i = 0; i < THREADS / 32; ++i) {
      if (i < warp) before += scratch[i];
      base += scratch[i];
    }
    if (b < B) cum[b] = before + x - n;
    __syncthreads();
  }
  return wk.pre_units() + base;
}

// Units of the rows_kernel behind a tile_kernel (about: a causal segment may end a tile earlier); the block's threads
// together.  scratch: a word per warp.
template <int THREADS>
__device__ __forceinline__ uint32_t units_behind(const SegWork& w, uint32_t* scratch) {
  uint32_t n = 0;
  for (int b = threadIdx.x; b < w.a.kv.batch; b += THREADS) {
    const SeqRef s = seq_ref(w.a, b);
    if (s.valid && s.len > w.a.prefix_len)
      n += static_cast<uint32_t>((s.n * w.a.G + w.behind_rt - 1) / w.behind_rt *
                                 ((s.len - w.a.prefix_len + kRowsTile - 1) / kRowsTile + kRowsSegCost));
  }
  n = __reduce_add_sync(0xffffffffu, n);
  if (threadIdx.x % 32 == 0) scratch[threadIdx.x / 32] = n;
  __syncthreads();
  n = 0;
  for (int i = 0; i < THREADS / 32; ++i) n += scratch[i];
  return n * static_cast<uint32_t>(w.a.kv.KVH);
}

// Shares of `total` units in at most `grid` ranges (of a CTA each, mostly): contiguous, equal within one, none below
// `least` (but in a call that has no more); range c is [begin(c), begin(c + 1)).
struct Share {
  uint32_t ctas, each, more;   // the first `more` CTAs take each + 1 units
  __device__ __forceinline__ Share(uint32_t total, uint32_t grid, uint32_t least) {
    ctas = min(grid, total > least ? total / least : min(total, 1u));
    each = ctas ? total / ctas : 0;
    more = total - each * ctas;
  }
  __device__ __forceinline__ uint32_t begin(uint32_t c) const { return c * each + min(c, more); }
  __device__ __forceinline__ int owner(uint32_t g) const {   // the CTA that holds unit g
    const uint32_t head = more * (each + 1);
    return static_cast<int>(g < head ? g / (each + 1) : more + (g - head) / each);
  }
};

// Barrier `id` of n threads; whether ok holds on all of them.
__device__ __forceinline__ bool named_bar_and(int id, int n, bool ok) {
  int r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.s32 p, %3, 0;\n\t"
      "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
      "selp.s32 %0, 1, 0, q;\n\t}"
      : "=r"(r)
      : "r"(id), "r"(n), "r"(static_cast<int>(ok))
      : "memory");
  return r != 0;
}

// mbar_wait without the clock on the way of a short wait: it is first read after 1024 tries.
__device__ __forceinline__ bool pipe_wait(uint64_t* bar, uint32_t parity) {
  uint64_t t0 = 0;
  for (uint32_t it = 1; !mbar_try_wait(bar, parity); ++it) {
    if ((it & 1023u) == 0) {
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kWaitLimitNs) return false;
    }
  }
  return true;
}

// ---- device primitives beyond common.cuh ------------------------------------------------------
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}
__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(addr) : "memory");
}
template <typename T>
__device__ __forceinline__ void mma_16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (std::is_same<T, __half>::value)
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Loads key tiles (TILE positions) of a segment: K and V boxes of the pages that hold a key of [lo, hi),
// one box per lane; the whole warp takes part.  ids holds the page ids of table entries id0 + lane.
template <int HD, int TILE>
struct PageLoader {
  const CUtensorMap* map;
  const PagedKv* kv;
  const int32_t* tab = nullptr;
  int id0, ids, lane;
  int id_end = 0;   // entries below this one are in use
  __device__ __forceinline__ void start(const int32_t* table, int key_end) {
    const int end = (key_end + (1 << kv->page_shift) - 1) >> kv->page_shift;
    if (table == tab && end <= id_end) return;   // the entries at hand are good for this segment too
    tab = table;
    id0 = -(1 << 30);
    id_end = end;
  }
  __device__ __forceinline__ int boxes(int key0, int lo, int hi, int& first) const {   // pages of the tile in use
    const int a = max(key0, lo), b = min(key0 + TILE, hi);
    if (b <= a) return 0;
    first = a >> kv->page_shift;
    return ((b - 1) >> kv->page_shift) - first + 1;
  }
  // rows of one box: a page, or the whole tile when pages are larger
  __device__ __forceinline__ int box_rows() const { return min(1 << kv->page_shift, TILE); }
  __device__ __forceinline__ void prefetch(int first, int n) {
    if (n > 0 && (first < id0 || first + n > id0 + 32)) {
      id0 = first;
      ids = first + lane < id_end ? tab[first + lane] : -1;
    }
  }
  // Whether a page of the tile has an id out of range.
  __device__ __forceinline__ bool bad_page(int first, int n) const {
    const int page = __shfl_sync(0xffffffffu, ids, (first - id0 + lane) & 31);
    return __any_sync(0xffffffffu, lane < n && (page < 0 || page >= kv->n_pages));
  }
  // One box per lane: the tile's pages in use x the 64-dim halves, into dst [HD/64][TILE rows][128 B];
  // which: 0 K, 1 V.
  __device__ __forceinline__ void load(uint8_t* dst, uint64_t* bar, int which, int kvh, int key0, int first, int n) const {
    const int i = lane / (HD / 64), h = lane % (HD / 64);
    const int page = page_at(first + i);
    if (i < n) box(dst, bar, which, kvh, key0, first + i, page, h);
  }
  // K and V of a tile likewise: lanes of K, then of V.
  __device__ __forceinline__ void load_kv(uint8_t* k, uint64_t* k_bar, uint8_t* v, uint64_t* v_bar, int kvh, int key0, int first,
                                          int n) const {
    const int i = lane / (HD / 32), h = lane % (HD / 64), which = lane / (HD / 64) % 2;
    const int page = page_at(first + i);
    if (i < n) box(which ? v : k, which ? v_bar : k_bar, which, kvh, key0, first + i, page, h);
  }
  // The same in boxes of 16 rows, n16 of them from row 16 first16 on: what a tile at the end of a segment needs of
  // its 64 rows (a sixth of the bytes of a batch of short sequences are beyond their ends otherwise).
  __device__ __forceinline__ void load_kv16(const CUtensorMap* map16, uint8_t* k, uint64_t* k_bar, uint8_t* v, uint64_t* v_bar,
                                            int kvh, int key0, int first16, int n16) const {
    const int i = lane / (HD / 32), h = lane % (HD / 64), which = lane / (HD / 64) % 2;
    const int at = (first16 + i) * 16, page = page_at(at >> kv->page_shift);
    if (i < n16)
      tma_load_4d((which ? v : k) + h * TILE * 128 + (at - key0) * 128, map16, which ? v_bar : k_bar, h * 64,
                  at & ((1 << kv->page_shift) - 1), which * kv->KVH + kvh, page);
  }
  // The page of a table entry at hand, n_pages (beyond the tensor: the copy fills zeros) for a bad id.
  __device__ __forceinline__ int page_at(int entry) const {
    const int page = __shfl_sync(0xffffffffu, ids, (entry - id0) & 31);
    return page < 0 || page >= kv->n_pages ? kv->n_pages : page;
  }
  __device__ __forceinline__ void box(uint8_t* dst, uint64_t* bar, int which, int kvh, int key0, int entry, int page, int h) const {
    const int row = entry - (key0 >> kv->page_shift);    // page within the tile
    const int y = key0 & ((1 << kv->page_shift) - 1);    // tile within the page (pages larger than a tile)
    tma_load_4d(dst + h * TILE * 128 + (row << kv->page_shift) * 128, map, bar, h * 64, y, which * kv->KVH + kvh, page);
  }
};

}  // namespace

// ============================================================================================
// At most 16 MT rows per segment (MT m16 tiles).  Four compute warps share every 64-key tile:
//   S = Q K^T      warp w takes keys 16 w .. 16 w + 15 of the tile and all row tiles
//   m, P           the row maxima meet in shared memory, so all warps keep the same running m
//   O += P V       warp w takes head dims w HD/4 .. and all keys, P read back from shared memory
// so K and V leave shared memory once, O needs no join and a segment ends with its l alone.  A fifth
// warp does everything with a memory latency: it walks the segments, streams their pages by TMA
// (128-byte swizzle: the ldmatrix reads are free of bank conflicts) and posts each segment's
// description and query rows ahead of its tiles.
// ============================================================================================
struct alignas(16) SegDesc {
  int32_t rows, mt, lo, hi;
  int32_t key0, cnt, kvh, flags;            // key0: first tile's first position; flags: kSeg* bits
  int32_t info, range, last_range, seq;     // entry of pre_info / own_info, the range, that of the last tile (first
                                            // part only), the sequence (own segments)
};
constexpr int kSegPrefix = 1, kSegStarts = 2, kSegEnds = 4, kSegBad = 8, kSegLast = 16;
struct alignas(16) RowDesc {
  int32_t last, first, token, head;
  uint64_t word, pad;
};

template <int HD, int MT>
struct RowsSmem {
  static constexpr int kRows = kRowsUnit * MT;                   // rows of a segment
  static constexpr int kStages = HD == 128 ? 5 : 10;             // K or V tiles in the ring
  static constexpr int kSlots = 4;                               // segments posted ahead, at most
  static constexpr uint32_t kBuf = kRowsTile * HD * 2;
  static constexpr uint32_t kQRow = HD * 2 + 16;                 // padded: ldmatrix without bank conflicts
  static constexpr int kQRows = kRowsSlotRows;                   // rows of all slots together
  static constexpr uint32_t oP = kStages * kBuf;                 // [MT][16][64] probabilities, swizzled
  static constexpr uint32_t oQ = oP + kRows * kRowsTile * 2;
  static constexpr uint32_t oRow = oQ + kQRows * kQRow;          // RowDesc [64]
  static constexpr uint32_t oMax = oRow + kQRows * sizeof(RowDesc);   // float [4][kRows]
  static constexpr uint32_t oSum = oMax + kRowsWarps * kRows * 4;     // float [4][kRows]
  static constexpr uint32_t oSeg = oSum + kRowsWarps * kRows * 4;     // SegDesc [kSlots]
  static constexpr uint32_t oBar = oSeg + kSlots * sizeof(SegDesc);   // full, empty, seg_full, seg_empty
  static constexpr uint32_t oMisc = oBar + (2 * kStages + 2 * kSlots) * 8;   // bad flags, scratch [32], sequence of a token [64]
  static constexpr uint32_t oCum = oMisc + (kStages + 32 + 64) * 4;   // own units before each sequence
  static constexpr uint32_t kTotal = oCum + kMaxBatch * 4 + 1024;
  static_assert(kRowsPerSm * (kTotal + 1024) <= 228 * 1024, "resident CTAs");
};

template <typename T, int HD, int MT>
__global__ void __launch_bounds__(kRowsThreads, kRowsPerSm)
    rows_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ CUtensorMap tm16, const __grid_constant__ SegWork w) {
  using SM = RowsSmem<HD, MT>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::oBar);
  uint64_t* empty = full + SM::kStages;
  uint64_t* seg_full = empty + SM::kStages;
  uint64_t* seg_empty = seg_full + SM::kSlots;
  volatile int* bad_stage = reinterpret_cast<volatile int*>(smem + SM::oMisc);
  uint32_t* scratch = reinterpret_cast<uint32_t*>(smem + SM::oMisc) + SM::kStages;
  int* token_seq = reinterpret_cast<int*>(scratch + 32);
  uint32_t* cum = reinterpret_cast<uint32_t*>(smem + SM::oCum);
  const PrefixAttnArgs& a = w.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < SM::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], kRowsWarps);
    }
    for (int s = 0; s < SM::kSlots; ++s) {
      mbar_init(&seg_full[s], 1);
      mbar_init(&seg_empty[s], kRowsWarps);
    }
    fence_mbar_init();
    tma_prefetch(&tm);
  }
  if (tid < 64) token_seq[tid] = -1;
  // A CTA that starts when tile_kernel's are done leaves if those that started with them have at most one range each
  // to go: its own start takes longer (64 sequences behind 8192 positions: 39.5 us, 37.7 so).  Those never leave,
  // so every range is taken whatever `taken`, which is read ahead of the gate, says.
  if (w.queue && tid == 0) {
    const uint32_t taken = __ldcg(&w.queue->next);
    uint64_t gate = load_acquire(&w.queue->gate), t0 = 0;
    while ((gate & ~kGateCtas) != kGate) {   // stored before this kernel could start: a matter of its becoming visible
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > kWaitLimitNs) break;
      gate = load_acquire(&w.queue->gate);
    }
    const bool open = (gate & ~kGateCtas) == kGate;
    if (!open && a.status) atomicOr(a.status, DEX_ATTN_TIMEOUT);
    const uint32_t early = static_cast<uint32_t>(gate & kGateCtas);
    scratch[30] = open;
    scratch[31] = blockIdx.x >= early && early > 0 ? taken + early : 0;
  }
  __syncthreads();
  if (w.queue && !scratch[30]) {
    griddep_wait();
    return;
  }
  if (w.first) griddep_wait();
  const uint32_t enough = w.queue ? scratch[31] : 0;   // the counts use the first words
  Walker<SM::kRows, kRowsTile, kRowsSegCost> wk(w);
  const uint32_t total = count_units<kRowsThreads>(wk, cum, scratch, w.do_prefix ? token_seq : nullptr);
  const uint32_t per_cta = w.queue || total >= kRowsTwo * gridDim.x ? static_cast<uint32_t>(w.per_cta) : 1u;
  const Share sh(total, per_cta * gridDim.x, kRowsMinUnits);
  if (w.queue && enough >= sh.ctas) {
    griddep_wait();
    return;
  }
  __syncthreads();
  griddep_launch_dependents();
  const int n_slots = w.slots;   // 64 / (rows of the call's largest segment), at most kSlots

  if (warp == kRowsWarps) {
    // ---------------- producer ----------------
    PageLoader<HD, kRowsTile> ld;
    ld.map = &tm;
    ld.kv = &a.kv;
    ld.lane = lane;
    uint32_t n_ld = 0, n_seg = 0, phase = 0;
    int st = 0;
    bool ok = true;
    uint32_t g = 0, g1 = 0, range = 0;
    auto claim = [&] {   // the next range
      if (!w.queue) return range + gridDim.x;
      uint32_t r = 0;
      if (lane == 0) r = atomicAdd(&w.queue->next, 1u);
      return __shfl_sync(0xffffffffu, r, 0);
    };
    auto slot_free = [&](int slot) {
      if (n_seg >= static_cast<uint32_t>(n_slots) && !pipe_wait(&seg_empty[slot], (n_seg / n_slots - 1) & 1u)) ok = false;
      ok = __all_sync(0xffffffffu, ok);
      return ok;
    };
    int off = 0;
    auto start_range = [&](uint32_t r) {
      range = r;
      if (r >= sh.ctas) return false;
      g = sh.begin(r);
      g1 = sh.begin(r + 1);
      off = wk.find(g, cum);
      return true;
    };
    bool more = start_range(w.queue ? claim() : blockIdx.x);
    for (; more && ok; ++n_seg) {
      const Piece pc = wk.piece(off, g1 - g);
      if (pc.cnt == 0) {   // only at the end of the range
        more = start_range(claim());
        --n_seg;
        continue;
      }
      // the segment's description, row table and query rows
      const int slot = static_cast<int>(n_seg % n_slots), row0 = slot * (SM::kQRows / n_slots);
      // its first page ids are on their way meanwhile
      ld.start(wk.prefix ? a.prefix_table : a.kv.table + static_cast<int64_t>(wk.b) * a.kv.table_stride, wk.k.hi);
      int first0 = 0;
      const int n0 = ld.boxes((wk.k.t0 + pc.tile) * kRowsTile, wk.k.lo, wk.k.hi, first0);
      ld.prefetch(first0, n0);
      if (slot_free(slot)) {
        int t = 0, h = 0;   // a row per lane
        if (lane < wk.rows) {
          wk.row_of(lane, t, h);
          SeqRef s = wk.s;
          if (wk.prefix) {
            const int b = token_seq[t];
            if (b >= 0) s = seq_ref(a, b);
            else s = SeqRef{0, 0, 0, false, false};
          }
          const RowView v = row_view(a, s, t);
          RowDesc* d = reinterpret_cast<RowDesc*>(smem + SM::oRow) + row0 + lane;
          *reinterpret_cast<int4*>(d) = make_int4(v.last, v.first, t, h);
          d->word = v.word;
        }
        __syncwarp();
        if (lane == 0) {
          int4* d = reinterpret_cast<int4*>(smem + SM::oSeg + slot * sizeof(SegDesc));
          d[0] = make_int4(wk.rows, (wk.rows + kRowsUnit - 1) / kRowsUnit, wk.k.lo, wk.k.hi);
          d[1] = make_int4((wk.k.t0 + pc.tile) * kRowsTile, pc.cnt, wk.kvh,
                           (wk.prefix ? kSegPrefix : 0) | (pc.starts ? kSegStarts : 0) | (pc.ends ? kSegEnds : 0) |
                               (!wk.prefix && wk.s.bad ? kSegBad : 0) |
                               (!w.queue && range + gridDim.x >= sh.ctas && g1 - g - pc.units <= kRowsSegCost ? kSegLast : 0));
          d[2] = make_int4(wk.prefix ? wk.seg : wk.own_info_index(), range,
                           pc.starts ? sh.owner(g - static_cast<uint32_t>(off) + wk.units() - 1) : 0, wk.prefix ? 0 : wk.b);
          mbar_arrive_expect_tx(&seg_full[slot], static_cast<uint32_t>(wk.rows * HD * 2));
        }
        __syncwarp();
        if (lane < wk.rows)
          bulk_load_1d(smem + SM::oQ + (row0 + lane) * SM::kQRow, static_cast<const T*>(a.q) + t * a.q_stride + h * HD, HD * 2,
                       &seg_full[slot]);
      }
      for (int i = 0; i < pc.cnt && ok; ++i) {
        const int key0 = (wk.k.t0 + pc.tile + i) * kRowsTile;
        int first = 0;
        const int n = ld.boxes(key0, wk.k.lo, wk.k.hi, first);
        ld.prefetch(first, n);
        const bool bad = ld.bad_page(first, n);
        const int kst = st;
        if (n_ld >= SM::kStages) ok = ok && pipe_wait(&empty[kst], phase ^ 1u);
        if (++st == SM::kStages) st = 0, phase ^= 1u;
        const int vst = st;
        if (n_ld + 1 >= SM::kStages) ok = ok && pipe_wait(&empty[vst], phase ^ 1u);
        if (++st == SM::kStages) st = 0, phase ^= 1u;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        const bool edge = key0 < wk.k.lo || key0 + kRowsTile > wk.k.hi;
        const int first16 = max(key0, wk.k.lo) >> 4, n16 = ((min(key0 + kRowsTile, wk.k.hi) + 15) >> 4) - first16;
        if (lane < 2) {
          const int x = lane ? vst : kst;
          if (n > 0) {
            bad_stage[x] = bad;
            mbar_arrive_expect_tx(&full[x], static_cast<uint32_t>((edge ? n16 * 16 : n * ld.box_rows()) * HD * 2));
          } else {
            bad_stage[x] = 0;
            mbar_arrive(&full[x]);
          }
          if (bad && lane && a.status) atomicOr(a.status, DEX_ATTN_BAD_PAGE);
        }
        __syncwarp();
        if (n > 0 && edge)
          ld.load_kv16(&tm16, smem + kst * SM::kBuf, &full[kst], smem + vst * SM::kBuf, &full[vst], wk.kvh, key0, first16, n16);
        else
          ld.load_kv(smem + kst * SM::kBuf, &full[kst], smem + vst * SM::kBuf, &full[vst], wk.kvh, key0, first, n);
        n_ld += 2;
      }
      g += pc.units;
      if (g < g1) {
        wk.next();
        off = 0;
      } else {
        more = start_range(claim());
      }
    }
    if (w.queue && slot_free(static_cast<int>(n_seg % n_slots))) {   // nothing more
      const int slot = static_cast<int>(n_seg++ % n_slots);
      if (lane == 0) {
        reinterpret_cast<SegDesc*>(smem + SM::oSeg)[slot].cnt = 0;
        mbar_arrive(&seg_full[slot]);
      }
    }
    if (!ok) {   // let the copies in flight land before the CTA goes
      if (lane == 0 && a.status) atomicOr(a.status, DEX_ATTN_TIMEOUT);
      for (uint32_t j = n_ld > SM::kStages ? n_ld - SM::kStages : 0; j < n_ld; ++j)
        pipe_wait(&full[j % SM::kStages], (j / SM::kStages) & 1u);
      for (uint32_t j = n_seg > static_cast<uint32_t>(n_slots) ? n_seg - n_slots : 0; j < n_seg; ++j)
        pipe_wait(&seg_full[j % n_slots], (j / n_slots) & 1u);
    }
  } else {
    // ---------------- compute ----------------
    constexpr int NV = HD / 32;                // n8 tiles of this warp's head dims
    const int gr = lane >> 2, tq = lane & 3;   // fragment row and column pair
    float* smax = reinterpret_cast<float*>(smem + SM::oMax);
    float* ssum = reinterpret_cast<float*>(smem + SM::oSum);
    const uint32_t sp = smem_u32(smem + SM::oP);
    const float c = score_scale(a), sign = a.scale_log2 > 0.0f ? 1.0f : a.scale_log2 < 0.0f ? -1.0f : 0.0f;
    const float drop = kDrop / c, depth = kDeep / c;   // of scores
    uint32_t phase = 0, n_seg = 0;
    int st = 0;
    bool ok = true;
    auto wait = [&](uint64_t* bar, uint32_t n) {
      if (ok && !pipe_wait(bar, n & 1u)) {
        if (a.status && lane == 0) atomicOr(a.status, DEX_ATTN_TIMEOUT);
        ok = false;
      }
    };
    for (bool more = w.queue || blockIdx.x < sh.ctas; more; ++n_seg) {
      const int slot = static_cast<int>(n_seg % n_slots), row0 = slot * (SM::kQRows / n_slots);
      wait(&seg_full[slot], n_seg / n_slots);
      if (!named_bar_and(1, kRowsWarps * 32, ok)) break;   // all four warps or none: they meet at barriers
      const SegDesc d = reinterpret_cast<const SegDesc*>(smem + SM::oSeg)[slot];
      if (d.cnt == 0) break;
      const RowDesc* rd = reinterpret_cast<const RowDesc*>(smem + SM::oRow) + row0;
      const uint32_t sq = smem_u32(smem + SM::oQ) + row0 * SM::kQRow;
      uint32_t qf[MT == 1 ? HD / 16 : 1][4];   // one row tile's queries stay in registers
      if constexpr (MT == 1) {
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) ldmatrix_x4(sq + (lane & 15) * SM::kQRow + ks * 32 + (lane >> 4) * 16, qf[ks]);
      }
      float o[MT][NV][4];
      float m[MT][2], l[MT][2];
      float low[MT][2], deep[MT][2];   // fp16: m comes down to a tile's maximum between these two
      int seen_by_all = 0x7fffffff;   // keys up to this one are seen by every row of this thread
#pragma unroll
      for (int u = 0; u < MT; ++u) {
#pragma unroll
        for (int n = 0; n < NV; ++n) o[u][n][0] = o[u][n][1] = o[u][n][2] = o[u][n][3] = 0.0f;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = u * 16 + gr + 8 * h;
          m[u][h] = low[u][h] = deep[u][h] = -INFINITY;
          l[u][h] = 0.0f;
          if (r < d.rows) seen_by_all = min(seen_by_all, rd[r].last);
        }
      }
      bool bad = false;   // it has met a bad page
      for (int i = 0; i < d.cnt; ++i) {
        // ---- scores of this warp's 16 keys ----
        const int kst = st;
        wait(&full[kst], phase);
        if (++st == SM::kStages) st = 0, phase ^= 1u;
        const int vst = st;
        bad |= bad_stage[kst] != 0;
        const int key0 = d.key0 + i * kRowsTile + warp * 16;
        const int in0 = max(d.lo - key0, 0), in1 = min(d.hi - key0, 16);   // keys of the segment among them
        const bool edge = in0 > 0 || in1 < 16;
        const bool masked = __any_sync(0xffffffffu, edge || key0 + 15 > seen_by_all);
        float x[MT][2][4];   // [row half][key: 2 tq, 2 tq + 1, + 8, + 9]
        {
          uint32_t kf[HD / 16][4];
          const int kr = warp * 16 + (lane & 7) + ((lane >> 4) << 3);   // ldmatrix row: key
          const uint32_t kt = smem_u32(smem + kst * SM::kBuf) + kr * 128;
#pragma unroll
          for (int ks = 0; ks < HD / 16; ++ks)
            ldmatrix_x4(kt + (ks >> 2) * (kRowsTile * 128) + ((((ks & 3) * 2 + ((lane >> 3) & 1)) ^ (kr & 7)) << 4), kf[ks]);
          __syncwarp();
          if (lane == 0) mbar_arrive(&empty[kst]);
#pragma unroll
          for (int u = 0; u < MT; ++u) {
            if (u >= d.mt) break;
            float s[2][2][4] = {};   // two chains: even and odd k steps
#pragma unroll
            for (int ks = 0; ks < HD / 16; ++ks) {
              const int qi = MT == 1 ? ks : 0;
              if constexpr (MT > 1) ldmatrix_x4(sq + (u * 16 + (lane & 15)) * SM::kQRow + ks * 32 + (lane >> 4) * 16, qf[qi]);
              mma_16816<T>(s[ks & 1][0], qf[qi], kf[ks][0], kf[ks][1]);
              mma_16816<T>(s[ks & 1][1], qf[qi], kf[ks][2], kf[ks][3]);
            }
#pragma unroll
            for (int h = 0; h < 2; ++h) {
#pragma unroll
              for (int e = 0; e < 4; ++e)
                x[u][h][e] = (s[0][e >> 1][2 * h + (e & 1)] + s[1][e >> 1][2 * h + (e & 1)]) * sign;
              if (masked) {
                const int r = u * 16 + gr + 8 * h;
                RowView v{0x7fffffff, 0, 0, false};
                if (r < d.rows) v.last = rd[r].last, v.first = rd[r].first, v.word = rd[r].word;
                const uint32_t bits = seen_bits(v, d.lo, d.hi, key0) >> (2 * tq);
                if (!(bits & 1u)) x[u][h][0] = -INFINITY;
                if (!(bits & 2u)) x[u][h][1] = -INFINITY;
                if (!(bits & 256u)) x[u][h][2] = -INFINITY;
                if (!(bits & 512u)) x[u][h][3] = -INFINITY;
              }
              float mx = fmaxf(fmaxf(x[u][h][0], x[u][h][1]), fmaxf(x[u][h][2], x[u][h][3]));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
              mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
              if (tq == 0) smax[warp * SM::kRows + u * 16 + gr + 8 * h] = mx;
            }
          }
        }
        wait(&full[vst], phase);
        if (++st == SM::kStages) st = 0, phase ^= 1u;
        if (edge && ok) {   // rows outside the segment hold anything: p = 0 must meet a finite v
          uint8_t* vt = smem + vst * SM::kBuf;
          for (int z = lane; z < 16 * HD / 8; z += 32) {
            const int row = z / (HD / 8), ch = z % (HD / 8);
            if (row < in0 || row >= in1)
              *reinterpret_cast<uint4*>(vt + (ch >> 3) * (kRowsTile * 128) + (warp * 16 + row) * 128 + (ch & 7) * 16) =
                  make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();   // before the stage's next copy
        }
        named_bar_sync(1, kRowsWarps * 32);
        // ---- the running maximum, P of this warp's keys ----
#pragma unroll
        for (int u = 0; u < MT; ++u) {
          if (u >= d.mt) break;
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            const int r = u * 16 + gr + 8 * h;
            float mx = -INFINITY;
#pragma unroll
            for (int k = 0; k < kRowsWarps; ++k) mx = fmaxf(mx, smax[k * SM::kRows + r]);
            if constexpr (kIsHalf<T>) {
              const float tile_m = mx;
              if (!(mx > m[u][h] || (mx < low[u][h] && mx > deep[u][h]))) mx = m[u][h];
              low[u][h] = mx - drop;
              deep[u][h] = fmaxf(deep[u][h], tile_m - depth);
            } else {
              mx = fmaxf(mx, m[u][h]);
            }
            const float base = mx > -INFINITY ? mx : 0.0f;
            const float f = ex2((m[u][h] - base) * c);
            m[u][h] = mx;
            auto prob = [&](float s) { return ex2(fmaf(s - base, c, kUp<T>)); };
            const float p0 = prob(x[u][h][0]), p1 = prob(x[u][h][1]), p2 = prob(x[u][h][2]), p3 = prob(x[u][h][3]);
            l[u][h] = l[u][h] * f + ((p0 + p1) + (p2 + p3));
#pragma unroll
            for (int n = 0; n < NV; ++n) {
              o[u][n][2 * h] *= f;
              o[u][n][2 * h + 1] *= f;
            }
            const uint32_t row = sp + u * 2048 + (gr + 8 * h) * 128 + tq * 4;
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(row + (((2 * warp) ^ gr) << 4)), "r"(pack2<T>(p0, p1)) : "memory");
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(row + (((2 * warp + 1) ^ gr) << 4)), "r"(pack2<T>(p2, p3)) : "memory");
          }
        }
        named_bar_sync(1, kRowsWarps * 32);
        // ---- O of this warp's head dims ----
#pragma unroll
        for (int ks = 0; ks < kRowsTile / 16; ++ks) {
          uint32_t vf[NV / 2][4];
          const int vr = ks * 16 + (lane & 15);   // ldmatrix row: key
#pragma unroll
          for (int n = 0; n < NV / 2; ++n) {
            const int dim = warp * (HD / 4) + n * 16 + (lane >> 4) * 8;
            ldmatrix_x4_trans(smem_u32(smem + vst * SM::kBuf) + (dim >> 6) * (kRowsTile * 128) + vr * 128 +
                                  ((((dim >> 3) & 7) ^ (vr & 7)) << 4), vf[n]);
          }
#pragma unroll
          for (int u = 0; u < MT; ++u) {
            if (u >= d.mt) break;
            uint32_t pf[4];
            const int pr = lane & 15;
            ldmatrix_x4(sp + u * 2048 + pr * 128 + (((2 * ks + (lane >> 4)) ^ (pr & 7)) << 4), pf);
#pragma unroll
            for (int n = 0; n < NV / 2; ++n) {
              mma_16816<T>(o[u][2 * n], pf, vf[n][0], vf[n][1]);
              mma_16816<T>(o[u][2 * n + 1], pf, vf[n][2], vf[n][3]);
            }
          }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[vst]);
      }
      // ---- the segment's result ----
      uint32_t poison = !ok || (d.flags & kSegBad) ? 0xffffffffu : 0u;   // a bit for each of this thread's rows
      if (bad) {
        const int32_t* table = d.flags & kSegPrefix ? a.prefix_table : a.kv.table + static_cast<int64_t>(d.seq) * a.kv.table_stride;
#pragma unroll 1
        for (int i = 0; i < 2 * MT; ++i) {
          const int r = (i >> 1) * 16 + gr + 8 * (i & 1);
          if (r < d.rows && sees_bad_page(a.kv, table, RowView{rd[r].last, rd[r].first, rd[r].word, true}, max(d.lo, d.key0),
                                          min(d.hi, d.key0 + d.cnt * kRowsTile)))
            poison |= 1u << i;
        }
        __syncwarp();
      }
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        if (u >= d.mt) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          l[u][h] += __shfl_xor_sync(0xffffffffu, l[u][h], 1);
          l[u][h] += __shfl_xor_sync(0xffffffffu, l[u][h], 2);
          if (poison >> (2 * u + h) & 1u) l[u][h] = quiet_nan();
          if (tq == 0) ssum[warp * SM::kRows + u * 16 + gr + 8 * h] = l[u][h];
        }
      }
      named_bar_sync(1, kRowsWarps * 32);
      const bool starts = d.flags & kSegStarts, whole = starts && (d.flags & kSegEnds), prefix = d.flags & kSegPrefix;
      const int rows_all = a.n_tokens * a.G;
#pragma unroll
      for (int u = 0; u < MT; ++u) {
        if (u >= d.mt) break;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int r = u * 16 + gr + 8 * h;
          if (r >= d.rows) continue;
          float L = 0.0f;
#pragma unroll
          for (int k = 0; k < kRowsWarps; ++k) L += ssum[k * SM::kRows + r];
          const int t = rd[r].token;
          const int head = rd[r].head, hg = head - d.kvh * a.G;
          const int dim = warp * (HD / 4) + 2 * tq;
          if (whole && !w.joined) {
            const float inv = isnan(L) ? L : L > 0.0f ? 1.0f / L : 0.0f;
            T* dst = static_cast<T*>(a.out) + t * a.out_stride + static_cast<int64_t>(head) * HD + dim;
#pragma unroll
            for (int n = 0; n < NV; ++n)
              *reinterpret_cast<uint32_t*>(dst + n * 8) = pack2<T>(o[u][n][2 * h] * inv, o[u][n][2 * h + 1] * inv);
            if (a.lse && warp == 0 && tq == 0)
              a.lse[static_cast<int64_t>(t) * a.H + head] = log_sum<T>(m[u][h], L, c);
          } else {
            const PartRef p = whole ? joined_part<HD>(prefix ? w.pre_o : w.own_o, prefix ? w.pre_ml : w.own_ml, d.kvh, rows_all,
                                                      t * a.G + hg)
                                    : slot_part<HD>(w.part_o, w.part_ml, 2 * d.range + (starts ? 1 : 0), SM::kRows, r);
#pragma unroll
            for (int n = 0; n < NV; ++n)
              *reinterpret_cast<float2*>(p.o + static_cast<int64_t>((dim + n * 8) >> 2) * p.step + (tq & 1) * 2) =
                  make_float2(o[u][n][2 * h], o[u][n][2 * h + 1]);
            if (warp == 0 && tq == 0) *p.ml = make_float2(m[u][h], L);
          }
        }
      }
      if (starts && tid == 0) (prefix ? w.pre_info : w.own_info)[d.info] = make_int2(d.range, d.last_range);
      more = !(d.flags & kSegLast);
      __syncwarp();
      if (lane == 0) mbar_arrive(&seg_empty[slot]);
    }
  }
  griddep_wait();   // a launch that follows must not overtake the one before this
}

// ============================================================================================
// Up to 256 rows per segment, on the 5th-generation tensor cores.  Two teams of four softmax warps
// own one 128-row S / P tile and one O accumulator in TMEM each:
//   S = Q K^T   (M = 128 rows, N = 128 keys, both operands in shared memory)
//   O += P V    (P from TMEM, where it replaces S; V an MN-major operand as loaded)
// One thread holds one row of S, so the softmax needs no exchange between threads.  With more than 128
// rows the teams take one row tile each and share every K and V tile; with fewer they share the rows
// and take alternate key tiles, and join at the segment's end.  Either way one team's softmax runs
// while the tensor cores work for the other.
// The running maximum of a row moves only when a score exceeds it by more than 2^8 (P then stays
// within 2^8, in fp16 within 2^15), so O is rescaled rarely: a rescale reads and writes
// all of it through registers between two MMAs.  c s - c m is one FMA with the rounded product c m, which is good
// while that is off by far less than one; of rows with larger products (kFar) the scores in TMEM are replaced by
// s - m first.  Difference and product apart for every score: 3.5 us more of 203 for 1752 prompt tokens behind
// 8192 positions.
// ============================================================================================
constexpr int kTileThreads = 384;   // two softmax teams; producer, an MMA issuer for each team, an idle warp
constexpr int kMetBadPage = 1, kMetTimeout = 2;   // what an issuer has met in a segment
constexpr float kRescale = 8.0f;
constexpr float kMostSum = 1099511627776.0f;   // 2^40: m comes down to a tile's (fp16) while l is below this
constexpr float kFar = 1048576.0f;   // 2^20, where fp32 neighbours are 2^-3 apart


template <int HD>
struct TileSmem {
  static constexpr uint32_t kBuf = kTileKeys * HD * 2;               // a Q, K or V tile
  static constexpr int kStages = HD == 128 ? 5 : 8;
  static constexpr uint32_t oQ = 0, oRing = 2 * kBuf;                // Q tiles (at a segment's end: O of team 1)
  static constexpr uint32_t oMl = oRing + kStages * kBuf;            // float2 [128]
  static constexpr uint32_t oBar = oMl + 128 * 8;
  static constexpr uint32_t kBars = 2 * kStages + 9;
  static constexpr uint32_t oMisc = oBar + kBars * 8;                // bad flags [stages], scratch [12], TMEM address, segment flags [4]
  static constexpr uint32_t kTotal = oMisc + (kStages + 17) * 4 + 1024;
  static_assert(kStages * kBuf >= kMaxBatch * 4, "the counts use the ring before the first copy");
};
static_assert(TileSmem<128>::kTotal <= 227 * 1024, "tile_kernel shared memory");

namespace {

__device__ __forceinline__ uint32_t sw_off(int row, int col) {   // element offset in a [128 rows][HD] tile, 64-column halves
  return static_cast<uint32_t>((col >> 6) * (128 * 128) + row * 128 + ((((col >> 3) & 7) ^ (row & 7)) << 4));
}
// Shared-memory operand descriptors (128-byte swizzle, 1024-byte atoms) as two words; the upper one is the
// same for all.  K-major (Q, K): rows of 64 dims; MN-major (V as the B operand): 64 dims per
// 128-byte row, keys 128 bytes apart, the 64-dim halves 16 KB apart.  The issuing thread adds 16-byte
// units to the lower word and nothing else: with descriptors built from scratch for every MMA it, not
// the tensor pipe, set the pace (95 cycles per MMA of 64).
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t k_desc(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (1u << 16); }
__device__ __forceinline__ uint32_t mn_desc(uint32_t saddr) { return ((saddr & 0x3FFFFu) >> 4) | (((128u * 128u) >> 4) << 16); }
// kind::f16 with fp32 accumulators: type bits of A and B (0 fp16, 1 bf16), B MN-major or not
__host__ __device__ constexpr uint32_t idesc(bool fp16, bool b_mn, int N) {
  return (1u << 4) | (fp16 ? 0u : (1u << 7) | (1u << 10)) | (b_mn ? 1u << 16 : 0u) | (static_cast<uint32_t>(N >> 3) << 17) |
         (8u << 24);
}
// D (+)= A B with A in shared memory (descriptor) or in TMEM; accumulate is a compile-time choice but for
// an accumulator's first MMA.
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t a_lo, uint32_t b_lo, uint32_t id, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %5};\n\tmov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}" ::"r"(d),
      "r"(a_lo), "r"(b_lo), "r"(id), "r"(static_cast<uint32_t>(accumulate)), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint32_t b_lo, uint32_t id, bool accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}" ::"r"(d),
      "r"(a_tmem), "r"(b_lo), "r"(id), "r"(static_cast<uint32_t>(accumulate)), "n"(kDescHi)
      : "memory");
}
__device__ __forceinline__ void tmem_st32(uint32_t addr, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}
__device__ __forceinline__ void tmem_st16(uint32_t addr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(addr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}
// Pairs of fp32 in one 64-bit register, two operations per instruction.
__device__ __forceinline__ uint64_t u32x2(uint32_t lo, uint32_t hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "r"(lo), "r"(hi));
  return r;
}
__device__ __forceinline__ uint64_t f32x2(float lo, float hi) { return u32x2(__float_as_uint(lo), __float_as_uint(hi)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Loads of a segment's cnt tiles: K of the first `ahead` tiles, then V of tile j and K of tile
// j + ahead in turn -- the order in which the MMAs take them.
__device__ __forceinline__ int k_load(int j, int ahead) { return j < ahead ? j : ahead + 2 * (j - ahead) + 1; }
__device__ __forceinline__ int v_load(int j, int cnt, int ahead) {   // index of V_j among the 2 cnt loads
  const int a = min(ahead, cnt);
  return a + j + min(j, cnt - a);
}

}  // namespace

template <typename T, int HD>
__global__ void __launch_bounds__(kTileThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap tm, const __grid_constant__ SegWork w) {
  using SM = TileSmem<HD>;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + SM::oBar);
  uint64_t* empty = full + SM::kStages;
  uint64_t* q_full = empty + SM::kStages;   // [2] query tile of a team written
  uint64_t* s_full = q_full + 2;            // [2] scores of a team's tile in TMEM
  uint64_t* p_full = s_full + 2;            // [2] its probabilities in TMEM
  uint64_t* turn = p_full + 2;              // [2] a team's issuer may go (two row tiles)
  uint64_t* o_full = turn + 2;              // every MMA of the segment complete
  volatile int* bad_stage = reinterpret_cast<volatile int*>(smem + SM::oMisc);
  uint32_t* scratch = reinterpret_cast<uint32_t*>(smem + SM::oMisc) + SM::kStages;
  uint32_t* tmem_slot = scratch + 12;
  volatile int* seg_met = reinterpret_cast<volatile int*>(tmem_slot + 1);   // [2 segments][2 teams] kMet* bits (before o_full)
  uint32_t* cum = reinterpret_cast<uint32_t*>(smem + SM::oRing);
  const PrefixAttnArgs& a = w.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < SM::kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 2);   // both teams
    }
    for (int i = 0; i < 2; ++i) {
      // one arrival per warp: 128 of them on one word take longer than a softmax
      mbar_init(&q_full[i], 4);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&turn[i], 1);
    }
    // both issuers, their MMAs and their word on the segment's pages; and the warps of the teams as they enter the
    // segment: one team's issuer may need nothing of the other team, which has to have seen the phase before
    mbar_init(o_full, 4 + 8);
    fence_mbar_init();
    tma_prefetch(&tm);
  }
  if (warp == 9) {
    tmem_alloc(tmem_slot, 512);   // S / P of the teams: 128 columns each, then their O
    tmem_relinquish();
  }
  if (w.first) griddep_wait();
  Walker<kTileRows, kTileKeys, kTileSegCost> wk(w);
  const uint32_t total = count_units<kTileThreads>(wk, cum, scratch);
  uint32_t ctas = gridDim.x;
  if (w.behind_rt) {   // the other SMs go to rows_kernel at once
    const float mine = kTileWeight * static_cast<float>(total);
    const float other = static_cast<float>(units_behind<kTileThreads>(w, scratch));
    ctas = max(static_cast<uint32_t>(ceilf(static_cast<float>(ctas) * (mine / (mine + other)))), 1u);
  }
  const Share sh(total, ctas, kTileMinUnits);
  // rows_kernel starts when every CTA here has allowed it, which this one does after it has opened the queue
  if (w.queue && blockIdx.x == 0 && tid == 0) {
    w.queue->next = 0;
    store_release(&w.queue->gate, kGate + kRowsPerSm * (gridDim.x - sh.ctas));
  }
  const bool work = blockIdx.x < sh.ctas;
  const uint32_t g0 = work ? sh.begin(blockIdx.x) : 0, g1 = work ? sh.begin(blockIdx.x + 1) : 0;
  int off = work ? wk.find(g0, cum) : 0;
  fence_proxy_async_smem();   // the counts in the ring are read before its first copy
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  griddep_launch_dependents();
  const uint32_t tmem = *tmem_slot;
  auto timed_out = [&] {
    if (a.status) atomicOr(a.status, DEX_ATTN_TIMEOUT);
  };

  if (warp < 8) {
    // ---------------- softmax teams: one row per thread ----------------
    const int team = warp >> 2, r128 = tid & 127;
    const uint32_t t_lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    const uint32_t t_s = tmem + static_cast<uint32_t>(team) * 128 + t_lane;
    const uint32_t t_o = tmem + 256 + static_cast<uint32_t>(team) * 128 + t_lane;
    const float c = score_scale(a);
    float* join = reinterpret_cast<float*>(smem + SM::oQ);   // [HD][128] O of team 1
    float2* join_ml = reinterpret_cast<float2*>(smem + SM::oMl);
    uint32_t n_s = 0, n_seg = 0, base = 0;   // score tiles of this team, segments, loads so far
    auto stage_of = [&](int load) { return &empty[(base + static_cast<uint32_t>(load)) % SM::kStages]; };
    auto free_stage = [&](uint64_t* bar, bool both) {   // a load's stage goes back (both: for the other team too)
      mbar_arrive(bar);
      if (both) mbar_arrive(bar);
    };
    bool ok = true;
    for (uint32_t g = g0; g < g1;) {
      const Piece pc = wk.piece(off, g1 - g);
      const int tile = pc.tile, cnt = pc.cnt;
      if (cnt == 0) break;   // only at the end of the range
      __syncwarp();
      if (lane == 0) mbar_arrive(o_full);   // this warp has read the segment before
      const bool alt = wk.rows <= 128;   // the teams share the rows and take alternate key tiles
      const int ahead = alt ? 2 : 1;
      const int r = alt ? r128 : team * 128 + r128;
      const bool on = r < wk.rows;
      if (!alt || team == 0) {
        // the team's query rows, HD / 8 threads per row; zero beyond the segment
        constexpr int kStep = 1024 / HD;   // rows of one pass, a multiple of the swizzle's eight
        const int row0 = alt ? 0 : team * 128, e = (r128 % (HD / 8)) * 8;
        uint8_t* dst = smem + SM::oQ + (alt ? 0 : team) * SM::kBuf + sw_off(r128 / (HD / 8), e);
#pragma unroll 4
        for (int rr = r128 / (HD / 8); rr < 128; rr += kStep, dst += kStep * 128) {
          if (row0 + rr < wk.rows) {
            int t, h;
            wk.row_of(row0 + rr, t, h);
            cp_async_16(smem_u32(dst), static_cast<const T*>(a.q) + t * a.q_stride + h * HD + e);
          } else {
            *reinterpret_cast<uint4*>(dst) = make_uint4(0u, 0u, 0u, 0u);
          }
        }
        cp_async_commit();
        cp_async_wait_all();
        if (a.scale_log2 <= 0.0f) {   // c is positive: the queries take the sign (zero for a zero scale)
          for (int i = 0; i < HD / 8; ++i) {
            uint4* v = reinterpret_cast<uint4*>(dst -= kStep * 128);
            const uint32_t keep = a.scale_log2 < 0.0f ? 0xffffffffu : 0u, flip = a.scale_log2 < 0.0f ? 0x80008000u : 0u;
            *v = make_uint4((v->x & keep) ^ flip, (v->y & keep) ^ flip, (v->z & keep) ^ flip, (v->w & keep) ^ flip);
          }
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(&q_full[team]);
      }
      int t_row = 0, h_row = 0;   // the thread's row
      if (on) wk.row_of(r, t_row, h_row);
      RowView rv{0x7fffffff, 0, 0, false};
      if (on) rv = wk.prefix ? row_view(a, seq_ref(a, seq_of_token(a, t_row)), t_row) : row_view(a, wk.s, t_row);
      float m = -INFINITY, l = 0.0f;
      bool any = false;   // this team had a tile
      // stages of K of its next tile and V of its last one (thread 0), at hand before they are to be freed: the
      // loads that wait for them are needed within a tile's time
      uint64_t *k_stage = stage_of(k_load(alt ? team : 0, ahead)), *v_stage = nullptr;
      for (int j = alt ? team : 0; j < cnt; j += ahead == 2 ? 2 : 1) {
        if (ok && !pipe_wait(&s_full[team], n_s & 1u)) {
          timed_out();
          ok = false;
        }
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        tc_fence_after();
        if (r128 == 0) {   // K of this tile and V of the team's tile before it are read
          free_stage(k_stage, alt);
          if (any) free_stage(v_stage, alt);
        }
        const int key0 = (wk.k.t0 + tile + j) * kTileKeys;
        const bool whole = wk.k.lo <= key0 && wk.k.hi >= key0 + kTileKeys;
        uint32_t s[2][32];
        float tile_l, tile_m = -INFINITY;   // sum and maximum of this tile
        float c_off = c;                    // 0 when the scores in TMEM are s - m
        auto moves = [&] {
          const float d = (tile_m - m) * c;
          // at m = -inf too, unless tile_m is -inf as well
          return d > kRescale || (kIsHalf<T> && d < -kDrop && d > -kDeep && l < kMostSum);
        };
        auto far = [&] { return m > -INFINITY && fabsf(m) * c >= kFar; };
        // m and the scores have to be looked at before P: masked scores, or such a row
        bool settle = !__all_sync(0xffffffffu, whole && rv.last >= key0 + kTileKeys - 1 && !far());
        if (settle) {
          // masked scores go back to TMEM as -inf
#pragma unroll 1
          for (int q = 0; q < 4; ++q) {
            tmem_ld32_nowait(t_s + q * 32, s[0]);
            tmem_wait_ld();
            const uint32_t bits = seen_bits(rv, wk.k.lo, wk.k.hi, key0 + q * 32);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              if (!(bits >> i & 1u)) s[0][i] = 0xff800000u;   // -inf
              tile_m = fmaxf(tile_m, __uint_as_float(s[0][i]));
            }
            tmem_st32(t_s + q * 32, s[0]);
          }
          tmem_wait_st();
        } else if (!any) {
          // the first tile's maximum: a pass of loads, where the exponentials below would be taken twice
          float mx[2] = {-INFINITY, -INFINITY};
          tmem_ld32_nowait(t_s, s[0]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            tmem_wait_ld();
            if (q < 3) tmem_ld32_nowait(t_s + (q + 1) * 32, s[(q + 1) & 1]);
#pragma unroll
            for (int i = 0; i < 16; ++i)
              mx[i & 1] = max3(mx[i & 1], __uint_as_float(s[q & 1][2 * i]), __uint_as_float(s[q & 1][2 * i + 1]));
          }
          tile_m = m = fmaxf(mx[0], mx[1]);
          settle = __any_sync(0xffffffffu, far());
        }
        if (!whole) {
          // rows of V outside the segment hold anything, and P = 0 must meet a finite v
          const uint32_t vl = base + static_cast<uint32_t>(v_load(j, cnt, ahead));
          const int st = static_cast<int>(vl % SM::kStages);
          if (!pipe_wait(&full[st], (vl / SM::kStages) & 1u)) {
            timed_out();
            ok = false;
          }
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          uint8_t* vt = smem + SM::oRing + st * SM::kBuf;
          for (int x = r128; x < kTileKeys * HD / 8; x += 128) {
            const int row = x / (HD / 8), ch = x % (HD / 8);
            if (key0 + row < wk.k.lo || key0 + row >= wk.k.hi)
              *reinterpret_cast<uint4*>(vt + (ch >> 3) * (128 * 128) + row * 128 + (ch & 7) * 16) = make_uint4(0u, 0u, 0u, 0u);
          }
          fence_proxy_async_smem();
        }
        // P with the m at hand, and the maximum on the way: it rarely asks for another m, and the scores are still
        // in TMEM then
        uint32_t p[4][16];
        for (;;) {
          if (settle) {
            // the row's m moves to the tile's maximum where that is larger by more than kRescale (or the first), and
            // in fp16 where it is smaller by more than kDrop
            const bool move = moves();
            if (__any_sync(0xffffffffu, move)) {
              // by the products that the probabilities are relative to, or by the exact difference where those are
              const float f = !move ? 1.0f : ex2(far() ? (m - tile_m) * c : __fmul_rn(m, c) - __fmul_rn(tile_m, c));
              if (any) {   // the PV before is complete: its issuer committed the scores after it
#pragma unroll 1
                for (int q = 0; q < HD / 32; ++q) {
                  uint32_t(&o)[32] = s[0];
                  tmem_ld32_nowait(t_o + q * 32, o);
                  tmem_wait_ld();
#pragma unroll
                  for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * f);
                  tmem_st32(t_o + q * 32, o);
                }
                tmem_wait_st();
              }
              if (move) m = tile_m;
              l *= f;
            }
            if (__any_sync(0xffffffffu, far())) {
              const float sub = m > -INFINITY ? m : 0.0f;
#pragma unroll 1
              for (int q = 0; q < 4; ++q) {
                tmem_ld32_nowait(t_s + q * 32, s[0]);
                tmem_wait_ld();
#pragma unroll
                for (int i = 0; i < 32; ++i) s[0][i] = __float_as_uint(__uint_as_float(s[0][i]) - sub);
                tmem_st32(t_s + q * 32, s[0]);
              }
              tmem_wait_st();
              c_off = 0.0f;
            }
          }
          const float sub = (m > -INFINITY ? m * c_off : 0.0f) - kUp<T>;
          uint64_t l2[2] = {0ull, 0ull};   // two fp32 sums each
          const uint64_t c2 = f32x2(c, c), sub2 = f32x2(-sub, -sub);
          float mx[2] = {-INFINITY, -INFINITY};
          tmem_ld32_nowait(t_s, s[0]);
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            tmem_wait_ld();
            if (q < 3) tmem_ld32_nowait(t_s + (q + 1) * 32, s[(q + 1) & 1]);
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const uint32_t s0 = s[q & 1][2 * i], s1 = s[q & 1][2 * i + 1];
              mx[i & 1] = max3(mx[i & 1], __uint_as_float(s0), __uint_as_float(s1));
              const uint64_t x = fma2(u32x2(s0, s1), c2, sub2);
              const float p0 = ex2(__uint_as_float(static_cast<uint32_t>(x))), p1 = ex2(__uint_as_float(static_cast<uint32_t>(x >> 32)));
              l2[i & 1] = add2(l2[i & 1], f32x2(p0, p1));
              p[q][i] = pack2<T>(p0, p1);
            }
          }
          const uint64_t t2 = add2(l2[0], l2[1]);
          tile_l = __uint_as_float(static_cast<uint32_t>(t2)) + __uint_as_float(static_cast<uint32_t>(t2 >> 32));
          tile_m = fmaxf(mx[0], mx[1]);
          settle = c_off > 0.0f && __any_sync(0xffffffffu, moves());
          if (!settle) break;
        }
        l += tile_l;
        any = true;
#pragma unroll
        for (int q = 0; q < 4; ++q) tmem_st16(t_s + q * 16, p[q]);   // over the scores
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[team]);
        v_stage = stage_of(v_load(j, cnt, ahead));
        k_stage = stage_of(k_load(j + ahead, ahead));
        ++n_s;
      }
      // ---------------- the segment's result ----------------
      if (ok && !pipe_wait(o_full, n_seg & 1u)) {
        timed_out();
        ok = false;
      }
      ok = __all_sync(0xffffffffu, ok);
      tc_fence_after();
      if (r128 == 0 && any) free_stage(v_stage, alt);
      const volatile int* met = seg_met + 2 * (n_seg & 1u);
      const int met_any = met[0] | met[1];
      if (!ok || (met_any & kMetTimeout) || (!wk.prefix && wk.s.bad)) l = quiet_nan();
      if (met_any & kMetBadPage) {
        const int32_t* table = wk.prefix ? a.prefix_table : a.kv.table + static_cast<int64_t>(wk.b) * a.kv.table_stride;
        const int at = (wk.k.t0 + tile) * kTileKeys;
        if (on && sees_bad_page(a.kv, table, rv, max(wk.k.lo, at), min(wk.k.hi, at + cnt * kTileKeys))) l = quiet_nan();
        __syncwarp();
      }
      const bool read = ok && any;   // warp-uniform
      if (alt && team == 1) {
        join_ml[r128] = make_float2(m, l);
        if (read) {
#pragma unroll
          for (int q = 0; q < HD / 32; ++q) {
            uint32_t o[32];
            tmem_ld32_nowait(t_o + q * 32, o);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) join[(q * 32 + i) * 128 + r128] = __uint_as_float(o[i]);
          }
        }
      }
      if (alt) named_bar_sync(1, 256);
      if (!alt || team == 0) {
        float f0 = 1.0f, f1 = 0.0f;
        const bool both = alt && cnt > 1;
        if (both) {
          const float2 other = join_ml[r128];
          const float M = fmaxf(m, other.x), sub = M > -INFINITY ? M : 0.0f;
          f0 = ex2((m - sub) * c);
          f1 = ex2((other.x - sub) * c);
          l = l * f0 + other.y * f1;
          m = M;
        }
        const bool starts = pc.starts, ends = pc.ends;
        const bool direct = starts && ends && !w.joined;
        const int t = t_row, h = h_row;
        const int64_t row = static_cast<int64_t>(t) * a.H + h;
        const PartRef part = starts && ends ? joined_part<HD>(wk.prefix ? w.pre_o : w.own_o, wk.prefix ? w.pre_ml : w.own_ml,
                                                              wk.kvh, a.n_tokens * a.G, t * a.G + h - wk.kvh * a.G)
                                            : slot_part<HD>(w.part_o, w.part_ml, 2 * blockIdx.x + (starts ? 1 : 0), kTileRows, r);
        const float inv = isnan(l) ? l : l > 0.0f ? 1.0f / l : 0.0f;
        T* dst = static_cast<T*>(a.out) + t * a.out_stride + static_cast<int64_t>(h) * HD;
#pragma unroll
        for (int q = 0; q < HD / 32; ++q) {
          uint32_t o[32];
          if (read) {
            tmem_ld32_nowait(t_o + q * 32, o);
            tmem_wait_ld();
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0u;
          }
          float x[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) x[i] = __uint_as_float(o[i]);
          if (both) {
#pragma unroll
            for (int i = 0; i < 32; ++i) x[i] = x[i] * f0 + join[(q * 32 + i) * 128 + r128] * f1;
          }
          if (on && direct) {
#pragma unroll
            for (int i = 0; i < 32; i += 8)
              *reinterpret_cast<uint4*>(dst + q * 32 + i) =
                  make_uint4(pack2<T>(x[i] * inv, x[i + 1] * inv), pack2<T>(x[i + 2] * inv, x[i + 3] * inv),
                             pack2<T>(x[i + 4] * inv, x[i + 5] * inv), pack2<T>(x[i + 6] * inv, x[i + 7] * inv));
          } else if (on) {
#pragma unroll
            for (int i = 0; i < 32; i += 4)
              *reinterpret_cast<float4*>(part.o + (q * 8 + i / 4) * part.step) = make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]);
          }
        }
        if (on && direct) {
          if (a.lse) a.lse[row] = log_sum<T>(m, l, c);
        } else if (on) {
          *part.ml = make_float2(m, l);
        }
        if (starts && tid == 0) {
          int2* info = wk.prefix ? w.pre_info + wk.seg : w.own_info + wk.own_info_index();
          *info = make_int2(blockIdx.x, sh.owner(g - static_cast<uint32_t>(off) + wk.units() - 1));
        }
      }
      if (alt) named_bar_sync(2, 256);   // the query tiles may be written again
      tc_fence_before();                 // O is read before the next segment's p_full
      ++n_seg;
      base += 2u * static_cast<uint32_t>(cnt);
      g += pc.units;
      if (g < g1) wk.next();
      off = 0;
    }
  } else {
    if (warp == 8) {
      // ---------------- producer ----------------
      PageLoader<HD, kTileKeys> lk, lv;
      lk.map = lv.map = &tm;
      lk.kv = lv.kv = &a.kv;
      lk.lane = lv.lane = lane;
      uint32_t n_ld = 0;
      bool ok = true;
      auto load = [&](PageLoader<HD, kTileKeys>& ld, int which, int j) {   // j: tile of the segment
        const int st = static_cast<int>(n_ld % SM::kStages), key0 = (wk.k.t0 + j) * kTileKeys;
        int first = 0;
        const int n = ld.boxes(key0, wk.k.lo, wk.k.hi, first);
        ld.prefetch(first, n);
        if (n_ld >= SM::kStages && !pipe_wait(&empty[st], (n_ld / SM::kStages - 1) & 1u)) ok = false;
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {
          if (lane == 0) timed_out();
          return;
        }
        const bool bad = ld.bad_page(first, n);
        if (lane == 0) {
          bad_stage[st] = bad;
          if (bad && a.status) atomicOr(a.status, DEX_ATTN_BAD_PAGE);
          if (n > 0) mbar_arrive_expect_tx(&full[st], static_cast<uint32_t>(n * ld.box_rows() * HD * 2));
          else mbar_arrive(&full[st]);
        }
        __syncwarp();
        ld.load(smem + SM::oRing + st * SM::kBuf, &full[st], which, wk.kvh, key0, first, n);
        ++n_ld;
      };
      for (uint32_t g = g0; g < g1 && ok;) {
        const Piece pc = wk.piece(off, g1 - g);
        const int tile = pc.tile, cnt = pc.cnt;
        const int ahead = wk.rows <= 128 ? 2 : 1;
        const int32_t* tab = wk.prefix ? a.prefix_table : a.kv.table + static_cast<int64_t>(wk.b) * a.kv.table_stride;
        lk.start(tab, wk.k.hi);
        lv.start(tab, wk.k.hi);
        for (int j = 0; j < min(ahead, cnt) && ok; ++j) load(lk, 0, tile + j);
        for (int j = 0; j < cnt && ok; ++j) {
          load(lv, 1, tile + j);
          if (ok && j + ahead < cnt) load(lk, 0, tile + j + ahead);
        }
        g += pc.units;
        if (g < g1) wk.next();
        off = 0;
      }
      if (!ok) {   // let the copies in flight land before the CTA goes
        for (uint32_t i = n_ld > SM::kStages ? n_ld - SM::kStages : 0; i < n_ld; ++i)
          pipe_wait(&full[i % SM::kStages], (i / SM::kStages) & 1u);
      }
    } else if (warp < 11 && lane == 0) {
      // ---------------- MMA issuer of a team ----------------
      // One thread for both teams cannot keep the tensor pipe fed: waits, commits and bookkeeping between
      // two blocks of MMAs take longer than the few MMAs that are queued (850 cycles per block of 512).
      // With two row tiles the issuers take turns, a PV and the next scores each: left alone the teams fall
      // into step, both in their softmax and then both waiting for their MMAs (3900 cycles per pair of
      // tiles; 2900 in turns).  The turn is passed on while the scores are being issued, so the other
      // thread wakes under the rest of them (1752 prompt tokens behind 8192: 209 us when it is passed before
      // them, 203 after two of their eight MMAs, 208 after six).
      // A commit costs it as much as an MMA, so there is one per key tile: the scores' commit also tells the
      // team that its PV before is complete and that the stages of both are free.
      const int team = warp - 9;
      constexpr bool kFp16 = std::is_same<T, __half>::value;
      constexpr uint32_t id_qk = idesc(kFp16, false, kTileKeys), id_pv = idesc(kFp16, true, HD);
      const uint32_t q_desc = k_desc(smem_u32(smem + SM::oQ)), ring_k = k_desc(smem_u32(smem + SM::oRing));
      const uint32_t ring_v = mn_desc(smem_u32(smem + SM::oRing));
      const uint32_t t_s = tmem + static_cast<uint32_t>(team) * 128, t_o = t_s + 256;
      uint32_t n_seg = 0, n_q1 = 0, n_p = 0, n_turn = 0, st = 0, phase = 0;   // st, phase: the next load of the ring
      bool ok = true;
      auto wait = [&](uint64_t* bar, uint32_t n) {
        if (ok && !pipe_wait(bar, n & 1u)) {
          timed_out();
          ok = false;
        }
        tc_fence_after();
        return ok;
      };
      auto skip_load = [&] {   // the next load's stage, without waiting for it
        const uint32_t at = st;
        if (++st == SM::kStages) st = 0, phase ^= 1u;
        return at;
      };
      auto next_load = [&] {
        wait(&full[st], phase);
        return skip_load();
      };
      auto qk = [&](uint32_t q, uint32_t stage, bool pass) {   // pass: the turn goes on meanwhile
        const uint32_t a0 = q_desc + q, b0 = ring_k + stage * (SM::kBuf >> 4);
#pragma unroll
        for (int ks = 0; ks < HD / 16; ++ks) {
          const uint32_t off = static_cast<uint32_t>((ks >> 2) * 128 * 128 + (ks & 3) * 32) >> 4;
          if (pass && ks == 2) mbar_arrive(&turn[team ^ 1]);
          umma_ss(t_s, a0 + off, b0 + off, id_qk, ks > 0);
        }
        umma_commit(&s_full[team]);
      };
      auto pv = [&](uint32_t stage, bool first) {
        const uint32_t b0 = ring_v + stage * (SM::kBuf >> 4);
#pragma unroll
        for (int ks = 0; ks < kTileKeys / 16; ++ks)
          umma_ts(t_o, t_s + ks * 8, b0 + ks * 128, id_pv, ks > 0 || !first);
      };
      for (uint32_t g = g0; g < g1 && ok; ++n_seg) {
        const Piece pc = wk.piece(off, g1 - g);
        const int cnt = pc.cnt;
        if (cnt == 0) break;
        const bool alt = wk.rows <= 128;
        const int ahead = alt ? 2 : 1;
        const uint32_t q = alt ? 0 : static_cast<uint32_t>(team) * (SM::kBuf >> 4);
        int bad = 0;
        if (alt || team == 0) wait(&q_full[0], n_seg);
        else wait(&q_full[1], n_q1++);
        for (int j = 0; j < min(ahead, cnt) && ok; ++j) {
          if (alt && j != team) {
            skip_load();
            continue;
          }
          const uint32_t k = next_load();
          if (!ok) break;
          qk(q, k, false);
        }
        for (int j = 0; j < cnt && ok; ++j) {
          const bool more = j + ahead < cnt;
          if (alt && (j & 1) != team) {
            skip_load();
            if (more) skip_load();
            continue;
          }
          const uint32_t v = next_load();
          if (!ok) break;
          bad |= bad_stage[v];
          const uint32_t k = more ? next_load() : 0;
          if (!alt) {
            if (team == 1) wait(&turn[1], n_turn);
            else if (n_turn > 0) wait(&turn[0], n_turn - 1);
            ++n_turn;
          }
          if (!wait(&p_full[team], n_p++)) break;
          pv(v, j < ahead);
          if (more) qk(q, k, !alt);
          else if (!alt) mbar_arrive(&turn[team ^ 1]);
        }
        // The teams read it after o_full.  The word was last that of the segment before the last one, which every
        // warp had read before it let o_full of the last one complete, and q_full came after that.
        seg_met[2 * (n_seg & 1u) + team] = (bad ? kMetBadPage : 0) | (ok ? 0 : kMetTimeout);
        umma_commit(o_full);
        mbar_arrive(o_full);
        g += pc.units;
        if (g < g1) wk.next();
        off = 0;
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 9) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  griddep_wait();
}

// ============================================================================================
// Joins the parts of the rows that have several.  A block takes 2^row_bits <= 32 rows of one K/V head and
// DIMS of their head dims; each of DIMS / 16 warps sums 16 of them over the parts, with the running
// maximum of the softmax.  Lanes beyond the rows, and in a call of few rows SPLIT groups of warps, take the
// parts in turn and join by shuffles and through shared memory: one after the other, the 38 parts of
// a 128k-token sequence are a chain of loads.  Parts lie as [head_dim / 4][rows][4], so 32 rows of
// four head dims are 512 contiguous bytes.
// ============================================================================================
struct CombineWork {
  SegWork own, pre;        // the kernels that computed own and prefix segments
  int32_t own_rt, pre_rt;  // their rows per segment
  int32_t own_ranges, pre_ranges;   // and ranges: the workspace holds two parts of each
  int32_t own_tile;        // their keys per tile (own segments)
  int32_t share;
  int32_t row_bits;
};

// (M, L, O) of a row over some parts, joined with that over others.
__device__ __forceinline__ void join_parts(float c, float& M, float& L, float4 (&o)[4], float m2, float l2, const float4 (&o2)[4]) {
  const float M1 = fmaxf(M, m2), base = M1 > -INFINITY ? M1 : 0.0f;
  const float f = ex2((M - base) * c), g = ex2((m2 - base) * c);
  M = M1;
  L = L * f + l2 * g;   // a poisoned part is NaN whatever its weight
#pragma unroll
  for (int q = 0; q < 4; ++q)
    o[q] = make_float4(o[q].x * f + o2[q].x * g, o[q].y * f + o2[q].y * g, o[q].z * f + o2[q].z * g, o[q].w * f + o2[q].w * g);
}

template <typename T, int HD, int DIMS, int SPLIT>
__global__ void __launch_bounds__(DIMS * 2 * SPLIT) combine_kernel(const __grid_constant__ CombineWork w) {
  constexpr int kThreads = DIMS * 2 * SPLIT;
  __shared__ int row_seq[32];
  __shared__ float join[SPLIT > 1 ? SPLIT / 2 : 1][SPLIT > 1 ? 18 : 1][DIMS * 2];
  const PrefixAttnArgs& a = w.own.a;
  const int tid = threadIdx.x, lane = tid & 31, group = tid / (DIMS * 2), kvh = blockIdx.y;
  const int warp = blockIdx.z * (DIMS / 16) + (tid >> 5) % (DIMS / 16);   // 16 head dims
  const int n_rows = 1 << w.row_bits, li = lane & (n_rows - 1), slot = lane >> w.row_bits, n_slots = 32 >> w.row_bits;
  const int rows_all = a.n_tokens * a.G, rg0 = blockIdx.x << w.row_bits;
  const int rg = rg0 + li;   // row: token * G + head within the K/V head
  const int t = w.own.by_g.div(rg);
  if (tid < 32) row_seq[tid] = -1;
  __syncthreads();
  {
    const int t0 = w.own.by_g.div(rg0), t1 = w.own.by_g.div(rg0 + n_rows - 1);
    for (int b = tid; b < a.kv.batch; b += kThreads) {
      const SeqRef s = seq_ref(a, b);
      if (!s.valid) continue;
      const int first = max(s.q0, t0), last = min(s.q0 + s.n - 1, t1);   // tokens of the block, then rows
      for (int r = max(first * a.G, rg0); first <= last && r < min((last + 1) * a.G, rg0 + n_rows); ++r) row_seq[r - rg0] = b;
    }
  }
  __syncthreads();
  const int b = row_seq[li];
  const SeqRef s = seq_ref(a, max(b, 0));
  const int r = rg - s.q0 * a.G, rt = b >= 0 ? r / w.own_rt : 0, r1 = min((rt + 1) * w.own_rt, s.n * a.G);
  const int pre_r = w.share ? rg % w.pre_rt : 0, own_r = r - rt * w.own_rt;   // row within its segments
  const int nt = w.own_tile == kRowsTile ? own_range<kRowsTile>(w.own, s, r1).nt : own_range<kTileKeys>(w.own, s, r1).nt;
  const int2* pre_at = b >= 0 && w.share ? w.pre.pre_info + rg / w.pre_rt * a.kv.KVH + kvh : nullptr;
  const int2* own_at = b >= 0 && nt > 0 ? w.own.own_info + own_info_of(a, w.own_rt, s.q0, b, rt, kvh) : nullptr;
  griddep_wait();
  if (w.own.queue && tid == 0 && blockIdx.x == 0 && blockIdx.y == 0 && blockIdx.z == 0) w.own.queue->gate = 0;
  // this row's parts: prefix parts of ranges pre_c0 .., then own parts of ranges own_c0 ..  A kernel that gave up
  // waiting leaves entries that hold anything: none of them is followed.
  const int2 pre_info = pre_at ? __ldcg(pre_at) : make_int2(0, -1), own_info = own_at ? __ldcg(own_at) : make_int2(0, -1);
  const int pre_c0 = pre_info.x, n_pre = parts_in(pre_info.x, pre_info.y, w.pre_ranges), own_c0 = own_info.x;
  int n_own = parts_in(own_info.x, own_info.y, w.own_ranges);
  if (n_own == 1 && !w.share) n_own = 0;   // written where it was computed
  const int n = n_pre + n_own;
  if (__all_sync(0xffffffffu, n <= 0)) return;   // the same in all warps
  const float c = score_scale(a);
  float M = -INFINITY, L = 0.0f;
  float4 o[4];
#pragma unroll
  for (int q = 0; q < 4; ++q) o[q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  constexpr int kUnroll = 2;
  const int step = n_slots * SPLIT;   // parts taken at once
  for (int k0 = slot * SPLIT + group; k0 < n; k0 += kUnroll * step) {
    float2 ml[kUnroll];
    float4 x[kUnroll][4];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int k = k0 + u * step;
      ml[u] = make_float2(-INFINITY, 0.0f);
      if (k < n) {
        const bool pre = k < n_pre;
        const SegWork& sw = pre ? w.pre : w.own;
        const int i = pre ? k : k - n_pre, rows = pre ? w.pre_rt : w.own_rt;
        const PartRef p = (pre ? n_pre : n_own) == 1
                              ? joined_part<HD>(pre ? sw.pre_o : sw.own_o, pre ? sw.pre_ml : sw.own_ml, kvh, rows_all, rg)
                              : slot_part<HD>(sw.part_o, sw.part_ml, 2 * ((pre ? pre_c0 : own_c0) + i) + (i == 0 ? 1 : 0), rows,
                                              pre ? pre_r : own_r);
        ml[u] = __ldcg(p.ml);
#pragma unroll
        for (int q = 0; q < 4; ++q) x[u][q] = __ldcg(reinterpret_cast<const float4*>(p.o + (warp * 4 + q) * p.step));
      } else {
#pragma unroll
        for (int q = 0; q < 4; ++q) x[u][q] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) join_parts(c, M, L, o, ml[u].x, ml[u].y, x[u]);
  }
  for (int other = n_rows; other < 32; other <<= 1) {   // lanes that took other parts of the row
    float4 o2[4];
    const float m2 = __shfl_xor_sync(0xffffffffu, M, other), l2 = __shfl_xor_sync(0xffffffffu, L, other);
#pragma unroll
    for (int q = 0; q < 4; ++q)
      o2[q] = make_float4(__shfl_xor_sync(0xffffffffu, o[q].x, other), __shfl_xor_sync(0xffffffffu, o[q].y, other),
                          __shfl_xor_sync(0xffffffffu, o[q].z, other), __shfl_xor_sync(0xffffffffu, o[q].w, other));
    join_parts(c, M, L, o, m2, l2, o2);
  }
  if constexpr (SPLIT > 1) {
#pragma unroll
    for (int half = SPLIT / 2; half > 0; half >>= 1) {   // groups half .. 2 half - 1 join groups 0 .. half - 1
      const int x = tid % (DIMS * 2);
      if (group >= half && group < 2 * half) {
        float(*dst)[DIMS * 2] = join[group - half];
        dst[0][x] = M;
        dst[1][x] = L;
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          dst[2 + 4 * q][x] = o[q].x;
          dst[3 + 4 * q][x] = o[q].y;
          dst[4 + 4 * q][x] = o[q].z;
          dst[5 + 4 * q][x] = o[q].w;
        }
      }
      __syncthreads();
      if (group < half) {
        const float(*src)[DIMS * 2] = join[group];
        float4 o2[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) o2[q] = make_float4(src[2 + 4 * q][x], src[3 + 4 * q][x], src[4 + 4 * q][x], src[5 + 4 * q][x]);
        join_parts(c, M, L, o, src[0][x], src[1][x], o2);
      }
      __syncthreads();
    }
    if (group > 0) return;
  }
  if (n <= 0 || slot > 0) return;
  const float inv = isnan(L) ? L : L > 0.0f ? 1.0f / L : 0.0f;
  const int h = kvh * a.G + rg - t * a.G;
  uint4* dst = reinterpret_cast<uint4*>(static_cast<T*>(a.out) + t * a.out_stride + h * HD + warp * 16);
#pragma unroll
  for (int q = 0; q < 4; q += 2)
    dst[q / 2] = make_uint4(pack2<T>(o[q].x * inv, o[q].y * inv), pack2<T>(o[q].z * inv, o[q].w * inv),
                            pack2<T>(o[q + 1].x * inv, o[q + 1].y * inv), pack2<T>(o[q + 1].z * inv, o[q + 1].w * inv));
  if (a.lse && warp == 0)
    a.lse[static_cast<int64_t>(t) * a.H + h] = log_sum<T>(M, L, c);
}

// ---- host ------------------------------------------------------------------------------------
namespace {

// One function attribute per device, set before its first launch there.
template <typename F>
cudaError_t set_smem(F* func, uint32_t bytes, std::atomic<uint64_t>& done, int dev) {
  if (dev < 64 && (done.load(std::memory_order_relaxed) >> dev & 1)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(bytes));
  if (e == cudaSuccess && dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  return e;
}

// 4-D map of the pages: head_dim, position in the page, (K|V) x K/V head, page; boxes of 64 dims x
// `rows` positions, 128-byte swizzle.
bool page_map(CUtensorMap* map, const PagedKv& kv, int rows) {
  const uint64_t page = uint64_t(1) << kv.page_shift;
  const cuuint64_t dims[4] = {static_cast<cuuint64_t>(kv.hd), page, static_cast<cuuint64_t>(2) * kv.KVH, static_cast<cuuint64_t>(kv.n_pages)};
  const cuuint64_t strides[3] = {static_cast<cuuint64_t>(kv.hd) * 2, page * kv.hd * 2, static_cast<cuuint64_t>(kv.page_stride) * 2};
  const cuuint32_t box[4] = {64, static_cast<cuuint32_t>(rows), 1, 1};
  return encode_tensor_map(map, kv.fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, kv.pages, dims,
                           strides, box);
}

template <typename K, typename... A>
cudaError_t launch(K* kernel, dim3 grid, int threads, uint32_t smem, cudaStream_t st, bool pdl, const A&... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = dim3(static_cast<unsigned>(threads));
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = pdl ? 1 : 0;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

template <typename T, int HD>
cudaError_t launch_hd(const PrefixAttnArgs& a, const Plan& p, uint8_t* ws, cudaStream_t st, int dev, int n_sm) {
  static std::atomic<uint64_t> rows1_set{0}, rows2_set{0}, tile_set{0};
  SegWork base = {};
  base.a = a;
  base.by_g = FastDiv(static_cast<uint32_t>(a.G));
  base.by_kvh = FastDiv(static_cast<uint32_t>(a.kv.KVH));
  base.share = p.share;
  base.joined = p.share;
  base.pre_o = reinterpret_cast<float*>(ws + p.o_pre);
  base.pre_ml = reinterpret_cast<float2*>(ws + p.o_pre_ml);
  base.own_o = reinterpret_cast<float*>(ws + p.o_own);
  base.own_ml = reinterpret_cast<float2*>(ws + p.o_own_ml);
  base.pre_info = reinterpret_cast<int2*>(ws + p.o_pre_info);
  base.own_info = reinterpret_cast<int2*>(ws + p.o_own_info);
  if (p.queue()) base.queue = reinterpret_cast<RangeQueue*>(ws + p.o_queue);
  SegWork rows = base, tile = base;
  rows.part_o = reinterpret_cast<float*>(ws + p.o_rows_part);
  rows.part_ml = reinterpret_cast<float2*>(ws + p.o_rows_ml);
  rows.slots = p.slots;
  rows.per_cta = p.rows_per_cta();
  rows.do_own = !p.own_tile;
  rows.do_prefix = p.share && !p.prefix_tile;
  tile.part_o = reinterpret_cast<float*>(ws + p.o_tile_part);
  tile.part_ml = reinterpret_cast<float2*>(ws + p.o_tile_ml);
  tile.do_own = p.own_tile;
  tile.do_prefix = p.prefix_tile;
  tile.first = 1;
  tile.behind_rt = p.queue() ? p.own_rt() : 0;
  rows.first = !(tile.do_own || tile.do_prefix);
  const int page = 1 << a.kv.page_shift;
  const int sms = n_sm < kSms ? n_sm : kSms;
  cudaError_t e = cudaSuccess;
  if (tile.do_own || tile.do_prefix) {
    CUtensorMap tm;
    if (!page_map(&tm, a.kv, page < kTileKeys ? page : kTileKeys)) return cudaErrorInvalidValue;
    e = set_smem(tile_kernel<T, HD>, TileSmem<HD>::kTotal, tile_set, dev);
    if (e == cudaSuccess)
      e = launch(tile_kernel<T, HD>, dim3(static_cast<unsigned>(sms)), kTileThreads, TileSmem<HD>::kTotal, st, true, tm, tile);
  }
  if (e == cudaSuccess && (rows.do_own || rows.do_prefix)) {
    CUtensorMap tm, tm16;
    if (!page_map(&tm, a.kv, page < kRowsTile ? page : kRowsTile) || !page_map(&tm16, a.kv, 16)) return cudaErrorInvalidValue;
    const dim3 grid(static_cast<unsigned>(kRowsPerSm * sms));
    if (p.rows_mt == 1) {
      e = set_smem(rows_kernel<T, HD, 1>, RowsSmem<HD, 1>::kTotal, rows1_set, dev);
      if (e == cudaSuccess) e = launch(rows_kernel<T, HD, 1>, grid, kRowsThreads, RowsSmem<HD, 1>::kTotal, st, true, tm, tm16, rows);
    } else {
      e = set_smem(rows_kernel<T, HD, 2>, RowsSmem<HD, 2>::kTotal, rows2_set, dev);
      if (e == cudaSuccess) e = launch(rows_kernel<T, HD, 2>, grid, kRowsThreads, RowsSmem<HD, 2>::kTotal, st, true, tm, tm16, rows);
    }
  }
  if (e == cudaSuccess) {
    CombineWork c = {};
    c.own = p.own_tile ? tile : rows;
    c.pre = p.prefix_tile ? tile : rows;
    c.own_rt = p.own_rt();
    c.pre_rt = p.pre_rt();
    c.own_ranges = p.own_ranges();
    c.pre_ranges = p.pre_ranges();
    c.own_tile = p.own_tile ? kTileKeys : kRowsTile;
    c.share = p.share;
    while (c.row_bits < 5 && (1 << c.row_bits) < a.n_tokens * a.G) ++c.row_bits;
    const unsigned groups = static_cast<unsigned>((a.n_tokens * a.G + (1 << c.row_bits) - 1) >> c.row_bits);
    const dim3 grid(groups, static_cast<unsigned>(a.kv.KVH));
    // The fewer blocks there are, the more warps share a row's parts and head dims.  Whole calls, us: 1 block
    // of parts per K/V head and 8 K/V heads 85.4 with eight groups, 86.5 with four; 64 blocks 36.9 with four, 38.0
    // with two; 160 blocks 32.5 with two, 34.4 with one; 256 blocks 146.9 with four, 144.7 with two; 1752 blocks
    // 215 with two, 208 with one.
    const unsigned blocks = groups * static_cast<unsigned>(a.kv.KVH);
    const dim3 split(groups, static_cast<unsigned>(a.kv.KVH), HD / 32);
    if (blocks < 64) e = launch(combine_kernel<T, HD, 32, 8>, split, 512, 0, st, true, c);
    else if (blocks < 128) e = launch(combine_kernel<T, HD, 32, 4>, split, 256, 0, st, true, c);
    else if (blocks < 4u * sms) e = launch(combine_kernel<T, HD, 32, 2>, split, 128, 0, st, true, c);
    else e = launch(combine_kernel<T, HD, HD, 1>, grid, HD * 2, 0, st, true, c);
  }
  return e;
}

}  // namespace

size_t prefix_attention_workspace(const PrefixAttnArgs& a) { return make_plan(a).total; }

cudaError_t launch_prefix_attention(const PrefixAttnArgs& a, void* workspace, cudaStream_t st) {
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  const Plan p = make_plan(a);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  if (a.kv.fp16)
    return a.kv.hd == 128 ? launch_hd<__half, 128>(a, p, ws, st, dev, n_sm) : launch_hd<__half, 64>(a, p, ws, st, dev, n_sm);
  return a.kv.hd == 128 ? launch_hd<__nv_bfloat16, 128>(a, p, ws, st, dev, n_sm)
                        : launch_hd<__nv_bfloat16, 64>(a, p, ws, st, dev, n_sm);
}

}  // namespace dex
