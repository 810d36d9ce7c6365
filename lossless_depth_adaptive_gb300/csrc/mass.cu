// The attention weight that the positions of a paged K/V cache receive:
//   mass[b][g][j] (+)= sum_i sum_h exp(scale q_ih . k_jg - lse_ih)
// over the last min(n, window) queries i of sequence b that see position j and the query heads h of K/V head g.
//
// An item is 256 keys of one K/V head of a sequence, in two halves of 128, against all query rows (query, head of the
// group) that see any of them, in blocks of at most 192 rows:
//   S^T = K Q^T   (tcgen05, M = 128 keys, N = query rows; K stays, Q blocks pass by)
// Keys are the rows of S^T, so two threads hold one key, half of the columns each, and add up weights in registers: no
// softmax maximum (lse is given), no exchange but of the two sums at an item's end, no atomics, and results depend on
// lengths alone.  An item's masses are written once, and every key is read once.
//
// What bounds it.  Few query rows: HBM and the way to the first tile (one token each of 64 sequences of up to 2560 positions, 32
// heads x 128: 102 us, 5.0 TB/s, the loads alone 87; added to masses that are there 125; 32 queries of four prompts of up to 32768 positions, 32 / 8
// heads: 51 us, the loads alone 39, some 4300 cycles per item, of which its summing warps take 1800 for the way to the next item and the join; one
// token each of 8 sequences of 2100: 13.1 us, 5 of them before the first scores).  Whole prompts: the chain of a half's
// columns, read up to the release of their buffer (half of a block's time), its next MMAs and the handovers, beside the MMAs and the
// exponentials of both halves, which take 1536 cycles each per 192 rows and 256
// keys (three of 3500-7000 tokens, 32 / 8 heads: 379 us at 1.95 GHz, 2900 cycles for each of the fullest CTA's 255 blocks, the mean CTA has 232;
// tensor pipe 52 % active).
//
// Scores and lse meet in base 2 in fp32, and the exponential is the approximate one: a weight is off by some 2^-22 of |score| + |lse| + 2, which
// is what fp32 inputs of that size say about it; a wider form would cost the loops that bound the call.
#include <math.h>

#include "../../include/dex.h"
#include "paged_tile.cuh"

namespace dex {

namespace {

constexpr int kHalf = 128, kItem = 2 * kHalf;   // keys
constexpr int kBlock = 128, kLongBlock = 192;   // query rows of a block, at most
constexpr int kTeams = 16;                      // warps that add up weights: (half of the item, half of the columns) x 4
constexpr int kTeamWarps = kTeams / 2;
constexpr int kThreads = 32 * (kTeams + 3);     // and one each for keys, MMAs and queries
constexpr int kMaxBatch = 1024;

constexpr int kRowStages = 4;                   // blocks whose rows' lse are at hand
constexpr uint32_t kPool = 6 * kHalf * 128 * 2; // bytes of key and query tiles

// Shared memory: the query stages, the key stages behind them (MassWork says how many), then:
constexpr uint32_t oRow = kPool;                           // float -lse log2(e), int last key seen: [stages][kLongBlock] each
constexpr uint32_t oJoin = oRow + kRowStages * kLongBlock * 8; // float [256]: sums of the second half of the columns
constexpr uint32_t oCum = oJoin + kItem * 4;               // int [batch + 1]: tiles of the sequences, or a running total
constexpr uint32_t oSeq = oCum + (kMaxBatch + 4) * 4;      // SeqPart [batch]
constexpr uint32_t oBar = oSeq + kMaxBatch * 12;
constexpr int kMaxStages = 12;                             // of keys or queries
constexpr uint32_t kBars = 4 * kMaxStages + 2 * kRowStages + 10;
constexpr uint32_t oDesc = oBar + kBars * 8;               // ItemDesc [key stages]
constexpr uint32_t oMisc = oDesc + kMaxStages * 8;         // TMEM address, flags of the query blocks, scratch
constexpr uint32_t kSmem = oMisc + (1 + kRowStages + 2) * 4 + 1024;
static_assert(kSmem <= 227 * 1024, "mass_kernel shared memory");

__device__ __forceinline__ void tma_load_3d(void* dst, const CUtensorMap* map, uint64_t* bar, int x, int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// The columns of a tmem_ld32_nowait are there; nothing that uses them moves ahead of this.
__device__ __forceinline__ void tmem_wait_ld32(uint32_t (&r)[32]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]),
                 "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]),
                 "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]),
                 "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31])::"memory");
}

// In which order items go to CTAs: in rounds, one to each, by sequence, tile and K/V head.
enum Order : int {
  kForward = 0,   // at most one query block per item: all items cost the same, and a CTA's next one may have its query block
  kSnake = 1,     // every other round backwards: a sequence's tiles have fewer and fewer query blocks
  kByLevel = 2    // the same, with tiles counted from the sequences' ends: the items with the most query blocks first
};
// One thread of the warp, the same each time, in a form that keeps what is uniform over the warp so.
__device__ __forceinline__ bool elect_one() {
  uint32_t is;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(is));
  return is != 0;
}

// 16 columns, with the wait.
__device__ __forceinline__ void tmem_ld16_wait(uint32_t addr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]),
        "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(addr)
      : "memory");
}

struct MassWork {
  MassArgs a;
  FastDiv by_g;
  int order;
  int tokens_per_block;              // at most kBlock / G
  int q_stages, k_stages;
  uint32_t q_half, q_bytes, k_base;  // bytes of 64 dims of a query block, of a block; first key stage
};

// Queries and length of a sequence; used 0: nothing to do.
struct SeqPart {
  int q1, used, len;
};
__device__ __forceinline__ SeqPart seq_part(const MassArgs& a, int b, bool* bad = nullptr) {
  const int q0 = a.q_start[b], q1 = a.q_start[b + 1], len = a.seq_len[b];
  const bool ok = q0 >= 0 && q1 >= q0 && q1 <= a.n_tokens && len >= 0 &&
                  len <= static_cast<int64_t>(a.kv.table_width) << a.kv.page_shift;
  if (bad) *bad = !ok;
  return SeqPart{q1, ok ? min(q1 - q0, a.window) : 0, len};
}
__device__ __forceinline__ int tiles_of(const MassArgs& a, const SeqPart& s) {   // items per K/V head
  return s.used > 0 && s.len > a.first ? (s.len + kItem - 1) / kItem - a.first / kItem : 0;
}

struct Item {
  int b, g, key0, len;
  int t0, q1, blocks;   // first query token that sees a key of the item, and the blocks from there to q1
  int at0;              // position of token t0
  __device__ __forceinline__ bool half(const MassArgs& a, int h) const {   // it has keys
    return key0 + h * kHalf < len && key0 + (h + 1) * kHalf > a.first;
  }
};
// A role's way through the items; the whole warp takes part.  Lengths are in shared memory: loaded by every role at every
// item they would take 1200 cycles each.
struct Walk {
  const MassWork& w;
  const int* totals;   // running totals of items, or with kByLevel tiles per sequence
  const SeqPart* seqs;
  int b = -1;
  __device__ __forceinline__ Walk(const MassWork& work, const int* t, const SeqPart* s) : w(work), totals(t), seqs(s) {}
  __device__ __forceinline__ Item operator()(int index) {
    const MassArgs& a = w.a;
    Item it;
    int tile, seq = b;
    if (w.order == kByLevel) {   // at most 32 sequences, one per lane
      const int lane = threadIdx.x & 31, tiles = lane < a.kv.batch ? totals[lane + 1] : 0;
      const int i = index / a.kv.KVH;
      it.g = index - i * a.kv.KVH;
      int lo = 0, hi = __reduce_max_sync(0xffffffffu, tiles);   // the lowest level with at most i tiles above it
      while (lo < hi) {
        const int mid = (lo + hi) / 2, n = __reduce_add_sync(0xffffffffu, max(tiles - 1 - mid, 0));
        if (n <= i) hi = mid;
        else lo = mid + 1;
      }
      const int above = __reduce_add_sync(0xffffffffu, max(tiles - 1 - lo, 0));
      seq = static_cast<int>(__fns(__ballot_sync(0xffffffffu, tiles > lo), 0, i - above + 1));
      tile = __shfl_sync(0xffffffffu, tiles, seq) - 1 - lo;
    } else {
      if (seq < 0 || index < totals[seq] || index >= totals[seq + 1]) {
        int lo = 0, hi = a.kv.batch;   // the last sequence with a total <= index
        while (hi - lo > 1) {
          const int mid = (lo + hi) / 2;
          if (totals[mid] <= index) lo = mid;
          else hi = mid;
        }
        seq = lo;
      }
      const int i = index - totals[seq];
      tile = i / a.kv.KVH;
      it.g = i - tile * a.kv.KVH;
    }
    b = seq;
    const SeqPart s = seqs[seq];
    it.b = seq;
    it.key0 = (a.first / kItem + tile) * kItem;
    it.len = s.len;
    it.q1 = s.q1;
    it.t0 = max(s.q1 - s.used, s.q1 - (s.len - max(it.key0, a.first)));
    it.blocks = (s.q1 - it.t0 + w.tokens_per_block - 1) / w.tokens_per_block;
    it.at0 = s.len - (s.q1 - it.t0);
    return it;
  }
};
// What the MMAs need of an item, beside its first half tile of keys.
struct ItemDesc {
  int tokens;          // that see a key of it
  uint32_t halves;     // bit h: half h has keys; bit 2: the query block of the item before
};
// Counts blocks through a ring of n stages.
struct Ring {
  int n, stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ explicit Ring(int stages) : n(stages) {}
  __device__ __forceinline__ void next() {
    if (++stage == n) {
      stage = 0;
      phase ^= 1;
    }
  }
};
// Whether an item's query block is the one of the item before it (kForward): it stays where it is.
struct LastBlock {
  int b = -1, g = 0, t0 = 0;
  __device__ __forceinline__ bool same(const MassWork& w, const Item& it) {
    const bool is = w.order == kForward && b == it.b && g == it.g && t0 == it.t0;
    b = it.b;
    g = it.g;
    t0 = it.t0;
    return is;
  }
};

}  // namespace

// kTensorKeys: for items with many blocks.  The keys go from shared memory to TMEM once per item, so that an MMA reads its
// query block alone from shared memory (both operands take all of its 128 bytes per clock).  Beside them there is room for
// one block's scores of either half: the halves take turns, one computes while the MMAs run for the other.  Blocks are as long
// as that allows, because a block's handovers between the warps take about 1000 cycles however long it is.
// kRagged: the rows of a whole block may be no multiple of 16.  Columns behind the last row are zeros times a key, which is no number where
// the key is infinite, so they are cleared.  (In the loop of the long blocks that would take 2 % of a call over whole prompts.)
template <typename T, int HD, bool kTensorKeys, bool kRagged>
__global__ void __launch_bounds__(kThreads, 1)
    mass_kernel(const __grid_constant__ CUtensorMap tm_k, const __grid_constant__ CUtensorMap tm_q, const __grid_constant__ MassWork w) {
  constexpr uint32_t kKeyBytes = kHalf * HD * 2;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* k_full = reinterpret_cast<uint64_t*>(smem + oBar);
  uint64_t* k_empty = k_full + kMaxStages;
  uint64_t* q_full = k_empty + kMaxStages;
  uint64_t* q_empty = q_full + kMaxStages;
  uint64_t* row_full = q_empty + kMaxStages;      // lse of a block's rows written
  uint64_t* row_empty = row_full + kRowStages;
  uint64_t* s_full = row_empty + kRowStages;      // [2 teams][2 buffers] scores in TMEM
  uint64_t* s_empty = s_full + 4;                 // they have been read
  uint64_t* t_full = s_empty + 4;                 // [2] keys of a half in TMEM
  int* totals = reinterpret_cast<int*>(smem + oCum);
  SeqPart* seqs = reinterpret_cast<SeqPart*>(smem + oSeq);
  float* join = reinterpret_cast<float*>(smem + oJoin);
  volatile ItemDesc* descs = reinterpret_cast<volatile ItemDesc*>(smem + oDesc);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + oMisc);
  volatile uint32_t* plain_block = tmem_slot + 1;   // [stages] every row counts
  int* count = reinterpret_cast<int*>(tmem_slot + 1 + kRowStages);
  float* row_lse = reinterpret_cast<float*>(smem + oRow);
  int* row_at = reinterpret_cast<int*>(row_lse + kRowStages * kLongBlock);
  const MassArgs& a = w.a;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  if (tid == 0) {
    for (int s = 0; s < kMaxStages; ++s) {
      mbar_init(&k_full[s], 1);
      mbar_init(&k_empty[s], kTensorKeys ? 1 + kTeamWarps : 1);   // the MMAs (their warp), and who moves the keys
      mbar_init(&q_full[s], 1);
      mbar_init(&q_empty[s], 1);
    }
    for (int s = 0; s < kRowStages; ++s) {
      mbar_init(&row_full[s], 1);
      mbar_init(&row_empty[s], kTeams);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], kTeamWarps);
    }
    for (int i = 0; i < 2; ++i) mbar_init(&t_full[i], kTeamWarps);
    fence_mbar_init();
    tma_prefetch(&tm_k);
    tma_prefetch(&tm_q);
  }
  if (warp == kTeams + 1) {
    tmem_alloc(tmem_slot, 512);
    tmem_relinquish();
  }
  // rows of a query block that no copy fills are columns of S^T that count for nothing, but have to be numbers
  for (uint32_t i = tid; i < w.k_base / 16; i += kThreads) reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
  griddep_wait();
  griddep_launch_dependents();
  for (int b = tid; b < a.kv.batch; b += kThreads) {
    bool bad;
    seqs[b] = seq_part(a, b, &bad);
    const int tiles = tiles_of(a, seqs[b]);
    totals[b + 1] = w.order == kByLevel ? tiles : tiles * a.kv.KVH;
    if (bad && a.status && blockIdx.x == 0) atomicOr(a.status, DEX_ATTN_BAD_RANGE);
  }
  __syncthreads();
  if (warp == 0) {
    int before = 0;
    for (int b0 = 0; b0 < a.kv.batch; b0 += 32) {
      const int b = b0 + lane;
      int n = b < a.kv.batch ? totals[b + 1] : 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, n, o);
        if (lane >= o) n += x;
      }
      if (b < a.kv.batch && w.order != kByLevel) totals[b + 1] = before + n;
      before += __shfl_sync(0xffffffffu, n, 31);
    }
    if (lane == 0) {
      totals[0] = 0;
      *count = w.order == kByLevel ? before * a.kv.KVH : before;
    }
  }
  fence_proxy_async_smem();   // the zeros in the query stages come before the first copy
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int n_items = *count, grid = static_cast<int>(gridDim.x), cta = static_cast<int>(blockIdx.x);
  // the CTA's items are index_of(0), index_of(1), ... below n_items
  auto index_of = [&](int r) { return r * grid + (w.order != kForward && r & 1 ? grid - 1 - cta : cta); };
  auto timed_out = [&] {
    if (a.status) atomicOr(a.status, DEX_ATTN_TIMEOUT);
  };
  // scores of half h in buffer b (with keys in TMEM there is one, behind their 128 columns)
  auto scores_at = [&](int h, uint32_t b) {
    return tmem + (kTensorKeys ? 128 + static_cast<uint32_t>(h) * kLongBlock : static_cast<uint32_t>(h) * 256 + b * 128);
  };
  auto wait_all = [&](uint64_t* bar, uint32_t parity) { return __all_sync(0xffffffffu, pipe_wait(bar, parity)); };

  if (warp < kTeams) {
    // ---------------- a key per thread ----------------
    const int team = warp / kTeamWarps, part = warp >> 2 & 1;   // half of the item, of the columns
    const uint32_t t_lane = static_cast<uint32_t>((warp & 3) * 32) << 16;
    Ring keys(w.k_stages);
    uint32_t buf = 0, s_phase = 0;   // of the next score tile
    const uint64_t c2 = f32x2(a.scale_log2, a.scale_log2);
    Ring rows_at(kRowStages);
    int stage = -1;     // of the current block's rows
    LastBlock last;
    Walk item_at(w, totals, seqs);
    bool ok = true;
    for (int r = 0, index; ok && (index = index_of(r)) < n_items; ++r) {
      const Item it = item_at(index);
      const bool active = it.half(a, team), same = last.same(w, it);
      const int half0 = it.key0 + team * kHalf, key = half0 + (tid & 127);
      const bool mine = key >= a.first && key < it.len;
      int page = 0;
      if (mine) page = a.kv.table[static_cast<int64_t>(it.b) * a.kv.table_stride + (key >> a.kv.page_shift)];
      if (kTensorKeys) {   // half of this thread's key goes to TMEM (the half's MMAs of the item before are complete)
        int k_stage = 0;
        uint32_t k_phase = 0;
#pragma unroll
        for (int h = 0; h < 2; ++h)
          if (it.half(a, h)) {
            if (h == team) {
              k_stage = keys.stage;
              k_phase = keys.phase;
            }
            keys.next();
          }
        if (active) {
          ok = wait_all(&k_full[k_stage], k_phase);
          if (ok) {
            constexpr int kWords = HD / 4, kChunk0 = HD == 128 ? 0 : 4;   // 32-bit words of a part
            const int row = tid & 127;
            const uint8_t* src = smem + w.k_base + k_stage * kKeyBytes + (HD == 128 ? part * kHalf * 128 : 0) + row * 128;
            uint32_t v[kWords];
#pragma unroll
            for (int c = 0; c < kWords / 4; ++c) {
              const uint4 x = *reinterpret_cast<const uint4*>(src + (((c + part * kChunk0) ^ (row & 7)) << 4));
              v[4 * c] = x.x;
              v[4 * c + 1] = x.y;
              v[4 * c + 2] = x.z;
              v[4 * c + 3] = x.w;
            }
            const uint32_t to = tmem + static_cast<uint32_t>(team * 64 + part * kWords) + t_lane;
            if constexpr (HD == 128) tmem_st32(to, v);
            else tmem_st16(to, v);
            tmem_wait_st();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) {
              mbar_arrive(&t_full[team]);
              mbar_arrive(&k_empty[k_stage]);
            }
          }
        }
      }
      float sum = 0.0f, low = 0.0f;   // compensated over the blocks
      for (int blk = 0; blk < it.blocks && ok; ++blk) {
        if (!same) {
          __syncwarp();
          if (stage >= 0 && lane == 0) mbar_arrive(&row_empty[stage]);
          stage = rows_at.stage;
          ok = wait_all(&row_full[stage], rows_at.phase);
          if (!ok) break;
          rows_at.next();
        }
        if (!active) continue;
        ok = wait_all(&s_full[team * 2 + buf], s_phase);
        if (!ok) break;
        tc_fence_after();
        const uint32_t t_s = scores_at(team, buf) + t_lane;
        const int first_at = it.at0 + blk * w.tokens_per_block;
        const int rows = min(it.q1 - it.t0 - blk * w.tokens_per_block, w.tokens_per_block) * a.G;
        const float* lse = row_lse + stage * kLongBlock;
        const int* at = row_at + stage * kLongBlock;
        const int mid = (rows + 31) / 32 * 16, from = part ? mid : 0, to = part ? rows : min(mid, rows);
        auto release = [&] {   // the scores' buffer, when the last columns are in registers
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[team * 2 + buf]);
        };
        uint64_t acc0 = 0, acc1 = 0;
        if (plain_block[stage] && first_at >= half0 + kHalf - 1) {
          auto add = [&](const uint32_t* v, int n, int c0) {
#pragma unroll
            for (int i = 0; i < n; i += 4) {
              const ulonglong2 l = *reinterpret_cast<const ulonglong2*>(lse + c0 + i);
              const uint64_t x = fma2(u32x2(v[i], v[i + 1]), c2, l.x), y = fma2(u32x2(v[i + 2], v[i + 3]), c2, l.y);
              acc0 = add2(acc0, f32x2(ex2(__uint_as_float(static_cast<uint32_t>(x))), ex2(__uint_as_float(static_cast<uint32_t>(x >> 32)))));
              acc1 = add2(acc1, f32x2(ex2(__uint_as_float(static_cast<uint32_t>(y))), ex2(__uint_as_float(static_cast<uint32_t>(y >> 32)))));
            }
          };
          auto clear = [&](uint32_t* v, int n, int c0) {
            if (!kRagged || c0 + n <= rows) return;
#pragma unroll
            for (int i = 0; i < n; ++i) v[i] = c0 + i < rows ? v[i] : 0u;
          };
          int c0 = from;
          for (; c0 + 16 < to; c0 += 32) {
            uint32_t v[32];
            tmem_ld32_nowait(t_s + c0, v);
            tmem_wait_ld32(v);
            if (c0 + 32 >= to) {
              release();
              clear(v, 32, c0);
            }
            add(v, 32, c0);
          }
          if (c0 < to) {
            uint32_t v[16];
            tmem_ld16_wait(t_s + c0, v);
            release();
            clear(v, 16, c0);
            add(v, 16, c0);
          }
          if (from >= to) release();
        } else {
          float s0 = 0.0f, s1 = 0.0f;
          for (int c0 = from; c0 < to; c0 += 16) {
            uint32_t v[16];
            tmem_ld16_wait(t_s + c0, v);
            if (c0 + 16 >= to) release();
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float x = ex2(fmaf(__uint_as_float(v[i]), a.scale_log2, lse[c0 + i]));
              const float y = ex2(fmaf(__uint_as_float(v[i + 1]), a.scale_log2, lse[c0 + i + 1]));
              s0 += key <= at[c0 + i] ? x : 0.0f;
              s1 += key <= at[c0 + i + 1] ? y : 0.0f;
            }
          }
          if (from >= to) release();
          acc0 = f32x2(s0, s1);
        }
        if (!kTensorKeys) buf ^= 1;
        if (buf == 0) s_phase ^= 1;
        acc0 = add2(acc0, acc1);
        const float more = __uint_as_float(static_cast<uint32_t>(acc0)) + __uint_as_float(static_cast<uint32_t>(acc0 >> 32));
        const float y = __fsub_rn(more, low), t = __fadd_rn(sum, y);
        low = __fsub_rn(__fsub_rn(t, sum), y);
        sum = t;
      }
      if (!ok) {
        timed_out();
        sum = quiet_nan();
      }
      // the parts join; the first one waits for the second, which waits until its sums before were taken
      if (part) join[team * kHalf + (tid & 127)] = sum;
      named_bar_sync(1 + team, 32 * kTeamWarps);
      if (!part) sum += join[team * kHalf + (tid & 127)];
      ok = named_bar_and(1 + team, 32 * kTeamWarps, ok);   // they leave together
      if (mine && !part) {
        if (page < 0 || page >= a.kv.n_pages) {
          sum = quiet_nan();
          if (a.status) atomicOr(a.status, DEX_ATTN_BAD_PAGE);
        }
        float* out = a.mass + (static_cast<int64_t>(it.b) * a.kv.KVH + it.g) * a.mass_stride + key;
        *out = a.accumulate ? *out + sum : sum;
      }
    }
  } else if (warp == kTeams) {
    // ---------------- keys: half tiles by TMA ----------------
    Ring ring(w.k_stages);
    int loads = 0;
    Walk item_at(w, totals, seqs);
    LastBlock last;
    bool ok = true;
    // An item's pages, one table entry per lane: 16 at most, fetched an item ahead.  A bad id becomes n_pages, beyond the
    // tensor: the copy fills zeros.
    const int shift = a.kv.page_shift, box_rows = min(1 << shift, kHalf);
    auto fetch = [&](const Item& it) {
      const int entry = (it.key0 >> shift) + lane;
      const bool in = lane < (kItem >> shift) && (entry << shift) < it.len;
      const int page = in ? a.kv.table[static_cast<int64_t>(it.b) * a.kv.table_stride + entry] : -1;
      return page < 0 || page >= a.kv.n_pages ? a.kv.n_pages : page;
    };
    int index = index_of(0), ids = 0;
    Item it;
    if (index < n_items) {
      it = item_at(index);
      ids = fetch(it);
    }
    for (int r = 0; ok && index < n_items; ++r) {
      const int next = index_of(r + 1);
      Item next_it;
      int next_ids = 0;
      if (next < n_items) {
        next_it = item_at(next);
        next_ids = fetch(next_it);
      }
      const uint32_t halves = it.half(a, 0) | it.half(a, 1) << 1 | last.same(w, it) << 2;
      for (int h = 0; h < 2; ++h) {
        if (!(halves >> h & 1)) continue;
        const int key0 = it.key0 + h * kHalf, lo = max(key0, a.first) >> shift, hi = (min(key0 + kHalf, it.len) - 1) >> shift;
        const int n = hi - lo + 1;   // pages with keys, a box of 64 dims of each per lane
        ok = wait_all(&k_empty[ring.stage], ring.phase ^ 1);
        if (!ok) break;
        if (lane == 0) {
          descs[ring.stage].tokens = it.q1 - it.t0;   // (read in the first half's stage)
          descs[ring.stage].halves = halves;
          mbar_arrive_expect_tx(&k_full[ring.stage], static_cast<uint32_t>(n * box_rows) * HD * 2);
        }
        __syncwarp();
        const int i = lane / (HD / 64), d = lane % (HD / 64);
        const int page = __shfl_sync(0xffffffffu, ids, (lo + i - (it.key0 >> shift)) & 31);
        if (i < n)
          tma_load_4d(smem + w.k_base + ring.stage * kKeyBytes + d * kHalf * 128 + max(((lo + i) << shift) - key0, 0) * 128, &tm_k,
                      &k_full[ring.stage], d * 64, key0 & ((1 << shift) - 1), it.g, page);
        ring.next();
        ++loads;
      }
      index = next;
      it = next_it;
      ids = next_ids;
    }
    if (!ok) {   // the copies in flight end before the CTA does
      if (lane == 0) timed_out();
      for (int i = 0; i < min(loads, w.k_stages); ++i) {
        if (ring.stage == 0) ring.phase ^= 1;
        ring.stage = (ring.stage == 0 ? w.k_stages : ring.stage) - 1;
        pipe_wait(&k_full[ring.stage], ring.phase);
      }
    }
  } else if (warp == kTeams + 1) {
    // ---------------- MMAs ----------------
    const uint32_t k_desc0 = k_desc(smem_u32(smem + w.k_base)), q_desc0 = k_desc(smem_u32(smem));
    Ring keys(w.k_stages), blocks(w.q_stages);
    int stage = -1;
    uint32_t buf[2] = {0, 0}, s_phase[2] = {0, 0}, t_phase[2] = {0, 0};   // s_phase: a bit per buffer
    bool ok = true;
    for (int r = 0; ok && index_of(r) < n_items; ++r) {
      ok = wait_all(&k_full[keys.stage], keys.phase);
      if (!ok) break;
      int tokens = __shfl_sync(0xffffffffu, descs[keys.stage].tokens, 0);
      const uint32_t halves = __shfl_sync(0xffffffffu, descs[keys.stage].halves, 0);
      int k_stage[2];
      uint32_t k_phase[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        k_stage[h] = keys.stage;
        k_phase[h] = keys.phase;
        if (halves >> h & 1) keys.next();
      }
      if (kTensorKeys) {   // (the desc has been read)
        __syncwarp();
        if (lane < 2 && (halves >> lane & 1)) mbar_arrive(&k_empty[lane ? k_stage[1] : k_stage[0]]);
      }
      for (bool first = true; tokens > 0 && ok; tokens -= w.tokens_per_block, first = false) {
        if (!(halves & 4)) {
          if (stage >= 0 && elect_one()) umma_commit(&q_empty[stage]);
          stage = blocks.stage;
          ok = wait_all(&q_full[stage], blocks.phase);
          blocks.next();
        }
        const int rows = min(tokens, w.tokens_per_block) * a.G;
        const uint32_t id = idesc(std::is_same<T, __half>::value, false, (rows + 31) & ~31);
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          if (!ok || !(halves >> h & 1)) continue;
          if (first && kTensorKeys) {
            ok = wait_all(&t_full[h], t_phase[h]);
            t_phase[h] ^= 1;
          } else if (first) {
            ok = wait_all(&k_full[k_stage[h]], k_phase[h]);
          }
          ok = ok && wait_all(&s_empty[h * 2 + buf[h]], (s_phase[h] >> buf[h] & 1) ^ 1);
          if (!ok) break;
          tc_fence_after();
          const uint32_t d = scores_at(h, buf[h]);
          const uint32_t k0 = k_desc0 + (k_stage[h] * kKeyBytes >> 4), q0 = q_desc0 + (stage * w.q_bytes >> 4);
          const uint32_t q_step = w.q_half >> 4;
          const bool done = tokens <= w.tokens_per_block;   // with these keys
          if (elect_one()) {
#pragma unroll
            for (int k = 0; k < HD / 16; ++k) {
              const uint32_t q = q0 + k / 4 * q_step + (k % 4 * 32 >> 4);
              if constexpr (kTensorKeys) umma_ts(d, tmem + static_cast<uint32_t>(h * 64) + k * 8, q, id, k > 0);
              else umma_ss(d, k0 + ((k / 4 * (kHalf * 128) + k % 4 * 32) >> 4), q, id, k > 0);
            }
            umma_commit(&s_full[h * 2 + buf[h]]);
            if (done && !kTensorKeys) umma_commit(&k_empty[k_stage[h]]);
          }
          __syncwarp();
          s_phase[h] ^= 1u << buf[h];
          if (!kTensorKeys) buf[h] ^= 1;
        }
      }
    }
    if (!ok && lane == 0) timed_out();
  } else {
    // ---------------- query blocks by TMA, with what each row needs beside its scores ----------------
    Ring ring(w.q_stages), rows_at(kRowStages);
    int loads = 0, r = -1, blk = 0;
    Walk item_at(w, totals, seqs);
    LastBlock last;
    Item it;
    it.blocks = 0;
    // the next block; false: none
    auto advance = [&] {
      if (++blk < it.blocks) return true;
      int index;
      while ((index = index_of(++r)) < n_items) {
        it = item_at(index);
        blk = 0;
        if (!last.same(w, it)) return true;
      }
      return false;
    };
    // A lane's rows of a block: their tokens from its first one on, where their lse lies from that of its first row.  One
    // warp's instructions take some five cycles each, so little is left to do per block.
    constexpr int kLaneRows = (kTensorKeys ? kLongBlock : kBlock) / 32;
    const int full = w.tokens_per_block * a.G;
    int token_of[kLaneRows], lse_at[kLaneRows];
#pragma unroll
    for (int i = 0; i < kLaneRows; ++i) {
      const int row = i * 32 + lane;
      token_of[i] = w.by_g.div(row);
      lse_at[i] = token_of[i] * a.H + row - token_of[i] * a.G;
    }
    struct Block {
      int t0, g, at0, rows;
      float l[kLaneRows];
    };
    // what its rows need is loaded a block ahead
    auto fetch = [&](Block& b) {
      const int t = blk * w.tokens_per_block;
      b.t0 = it.t0 + t;
      b.g = it.g * a.G;
      b.at0 = it.at0 + t;
      b.rows = min(it.q1 - b.t0, w.tokens_per_block) * a.G;
      const float* lse = a.lse + static_cast<int64_t>(b.t0) * a.H + b.g;
#pragma unroll
      for (int i = 0; i < kLaneRows; ++i) b.l[i] = i * 32 + lane < b.rows ? lse[lse_at[i]] : -INFINITY;
    };
    bool ok = true, more = advance();
    Block next;
    if (more) fetch(next);
    while (more && ok) {
      const Block b = next;
      more = advance();
      if (more) fetch(next);
      ok = wait_all(&q_empty[ring.stage], ring.phase ^ 1);
      if (!ok) break;
      if (lane == 0) {
        uint8_t* dst = smem + ring.stage * w.q_bytes;
        mbar_arrive_expect_tx(&q_full[ring.stage], static_cast<uint32_t>(full) * HD * 2);
#pragma unroll
        for (int i = 0; i < HD / 64; ++i) tma_load_3d(dst + i * w.q_half, &tm_q, &q_full[ring.stage], i * 64, b.g, b.t0);
      }
      ring.next();
      ++loads;
      const int stage = rows_at.stage;
      ok = wait_all(&row_empty[stage], rows_at.phase ^ 1);
      if (!ok) break;
      bool plain = true;
#pragma unroll
      for (int i = 0; i < kLaneRows; ++i) {
        const int row = i * 32 + lane;
        const bool counts = b.l[i] != -INFINITY;
        row_lse[stage * kLongBlock + row] = counts ? b.l[i] * -1.4426950408889634f : -INFINITY;
        row_at[stage * kLongBlock + row] = counts ? b.at0 + token_of[i] : -1;
        plain = plain && (counts || row >= full);
      }
      plain = __all_sync(0xffffffffu, plain);
      if (lane == 0) plain_block[stage] = plain;
      __syncwarp();
      if (lane == 0) mbar_arrive(&row_full[stage]);
      rows_at.next();
    }
    if (!ok) {
      if (lane == 0) timed_out();
      for (int i = 0; i < min(loads, w.q_stages); ++i) {
        if (ring.stage == 0) ring.phase ^= 1;
        ring.stage = (ring.stage == 0 ? w.q_stages : ring.stage) - 1;
        pipe_wait(&q_full[ring.stage], ring.phase);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kTeams + 1) tmem_dealloc(tmem, 512);
}

namespace {

template <typename T, int HD>
cudaError_t launch_hd(const MassArgs& a, cudaStream_t st, int dev, int n_sm) {
  static std::atomic<uint64_t> done[3];
  MassWork w = {};
  w.a = a;
  w.by_g = FastDiv(static_cast<uint32_t>(a.G));
  const bool single = a.window <= kBlock / a.G;
  const int most_rows = single ? kBlock : kLongBlock;
  w.tokens_per_block = a.window < most_rows / a.G ? a.window : most_rows / a.G;
  w.order = single ? kForward : a.kv.batch <= 32 ? kByLevel : kSnake;
  constexpr uint32_t kKeyBytes = kHalf * HD * 2;
  w.q_half = static_cast<uint32_t>((w.tokens_per_block * a.G + 31) / 32 * 32) * 128;
  w.q_bytes = w.q_half * (HD / 64);
  const uint32_t q_pool = single ? (w.q_bytes <= 16384 ? 32768 : 2 * w.q_bytes) : kPool / 2;
  w.q_stages = static_cast<int>(q_pool / w.q_bytes < kMaxStages ? q_pool / w.q_bytes : kMaxStages);
  w.k_base = q_pool;
  w.k_stages = static_cast<int>((kPool - q_pool) / kKeyBytes < kMaxStages ? (kPool - q_pool) / kKeyBytes : kMaxStages);
  CUtensorMap tm_k, tm_q;
  const int page = 1 << a.kv.page_shift;
  const cuuint64_t dims[3] = {HD, static_cast<cuuint64_t>(a.H), static_cast<cuuint64_t>(a.n_tokens)};
  const cuuint64_t strides[2] = {HD * 2, static_cast<cuuint64_t>(a.n_tokens > 1 ? a.q_stride : int64_t(a.H) * HD) * 2};
  const cuuint32_t box[3] = {64, static_cast<cuuint32_t>(a.G), static_cast<cuuint32_t>(w.tokens_per_block)};
  if (!page_map(&tm_k, a.kv, page < kHalf ? page : kHalf) ||
      !encode_tensor_map(&tm_q, a.kv.fp16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, a.q, dims, strides, box))
    return cudaErrorInvalidValue;
  const int64_t most = (static_cast<int64_t>(a.kv.table_width) * page / kItem + 1) * a.kv.KVH * a.kv.batch;
  const dim3 grid(static_cast<unsigned>(most < n_sm ? most : n_sm));
  auto run = [&](auto* kernel, std::atomic<uint64_t>& done) {
    const cudaError_t e = set_smem(kernel, kSmem, done, dev);
    return e != cudaSuccess ? e : launch(kernel, grid, kThreads, kSmem, st, true, tm_k, tm_q, w);
  };
  if (single) return run(mass_kernel<T, HD, false, true>, done[0]);
  return w.tokens_per_block * a.G % 16 ? run(mass_kernel<T, HD, true, true>, done[1]) : run(mass_kernel<T, HD, true, false>, done[2]);
}

}  // namespace

cudaError_t launch_attention_mass(const MassArgs& a, cudaStream_t st) {
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  if (a.kv.fp16) return a.kv.hd == 128 ? launch_hd<__half, 128>(a, st, dev, n_sm) : launch_hd<__half, 64>(a, st, dev, n_sm);
  return a.kv.hd == 128 ? launch_hd<__nv_bfloat16, 128>(a, st, dev, n_sm) : launch_hd<__nv_bfloat16, 64>(a, st, dev, n_sm);
}

}  // namespace dex
