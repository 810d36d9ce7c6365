// Eviction from a paged K/V cache: for each sequence and K/V head the positions with the largest mass stay, in their
// order.
//
// One cluster of blocks per (sequence, K/V head).  Masses are compared by order-preserving images of their bits; each block
// keeps the images of its share of the positions in shared memory, where they fit.  The smallest that stays is found by
// a histogram over the range that they span, in 2048 bins, summed through distributed shared memory; the bin that it falls
// into mostly has few positions, which go to every block and are ranked by comparing them; where they are many, the
// bin is the next range.  Then the kept positions are listed and their rows move.  In place, position i comes from a position >= i, and
// rows move in rounds of consecutive i: all blocks load a round's rows, meet, and store them.  A later round reads
// positions >= its own i, beyond everything stored so far, so one barrier per round is enough and no copy is needed.
//
// What bounds it: the selection by the latency of its steps (some 15 barriers and passes of 1000-6000 cycles), then the rows by
// HBM, one after the other since all heads select at the same time.  16 prompts of 8 heads x 128 to 2048 positions 54 us, of
// which 29 move 201 MB; 131072 positions of 32 heads to 8192 75 us, 36 of them for 268 MB; 8 sequences of 500 positions of 4 heads
// x 64 to 400 12.7 us.
#include <atomic>

#include "../../include/dex.h"
#include "cluster.cuh"
#include "common.cuh"
#include "kernels.h"

namespace dex {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 4 * kThreads;
constexpr int kMaxCluster = 8;
constexpr int kWarpRows = 8;     // rows that a warp moves in a round, K and V
constexpr int kListed = 2048;    // room for the positions of a bin that are ranked, divided among the blocks
constexpr int kCached = 20480;   // images in a block's shared memory (80 KB, two blocks per SM)
constexpr int kMove = kWarps * kWarpRows * 2 * 256;   // and later the rows on their way
static_assert(kMove <= kCached * 4, "rows in shared memory");

__device__ __forceinline__ uint32_t mass_key(float m) { return m != m ? 0u : ordered_key(m); }   // NaN below -inf

struct alignas(16) EvictShared {
  uint32_t hist[2][kBins];
  uint32_t list[kListed];              // images, block r's from r * kListed / blocks on
  uint32_t flat[kListed / 2];          // the same without gaps
  uint8_t list_warp[kListed];          // the warp whose run holds one of this block's
  uint32_t warp_a[kWarps], warp_b[kWarps];
  uint64_t totals[4][kMaxCluster];     // of every block of the cluster, written by each of them
  uint4 found;                         // bin, positions before it, positions in it: written by the block that finds it
  uint32_t cut, quota;                 // the smallest image that stays and how many equal to it do, likewise
  uint32_t listed;
  uint64_t loaded[kWarps];             // mbarriers of the warps' rows
};

// 1-D bulk copy shared -> global, of the thread's bulk group.
__device__ __forceinline__ void bulk_store_1d(void* dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(reinterpret_cast<uint64_t>(dst)), "r"(smem_u32(src)), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

}  // namespace

template <int HD>
__global__ void __launch_bounds__(kThreads, 2) evict_kernel(const __grid_constant__ EvictArgs a, int cached) {
  extern __shared__ __align__(16) uint8_t smem[];
  EvictShared& sh = *reinterpret_cast<EvictShared*>(smem);
  uint32_t* keys = reinterpret_cast<uint32_t*>(smem + sizeof(EvictShared));
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (lane == 0) mbar_init(&sh.loaded[warp], 1);
  fence_mbar_init();
  const uint32_t rank = cluster_rank(), n_cta = cluster_size();
  cluster_started_arrive();
  griddep_wait();
  griddep_launch_dependents();
  const int chain = blockIdx.x / n_cta, b = chain / a.kv.KVH, g = chain % a.kv.KVH;
  const int len = a.seq_len[b], shift = a.kv.page_shift;
  int32_t* kept = a.kept + static_cast<int64_t>(chain) * a.keep;
  const bool bad_len = len < 0 || len > (static_cast<int64_t>(a.kv.table_width) << shift);
  const int now = bad_len ? 0 : min(len, a.keep);
  if (rank == 0 && tid == 0 && g == 0) {
    a.new_len[b] = bad_len ? len : now;
    if (bad_len && a.status) atomicOr(a.status, DEX_ATTN_BAD_RANGE);
  }
  const int step = static_cast<int>(n_cta) * kThreads, self = static_cast<int>(rank) * kThreads + tid;
  const float* mass = a.mass + static_cast<int64_t>(chain) * a.mass_stride;
  for (int64_t i = static_cast<int64_t>(now) + self; i < a.keep; i += step) kept[i] = -1;
  cluster_started_wait();
  if (bad_len) return;   // the whole cluster

  if (len <= a.keep) {
    for (int64_t i = self; i < now; i += step) kept[i] = static_cast<int>(i);
  } else {
    for (int64_t i = self; i < a.first; i += step) kept[i] = static_cast<int>(i);
    for (int64_t i = self; i < a.recent; i += step) kept[a.keep - a.recent + i] = static_cast<int>(len - a.recent + i);
    // candidates [first, len - recent), a run of them per warp
    const int n = len - a.recent - a.first;
    const uint32_t want = static_cast<uint32_t>(a.keep - a.first - a.recent);
    const int per_warp = static_cast<int>((static_cast<uint32_t>(n) + n_cta * kThreads - 1) / (n_cta * kThreads)) * 32;
    const int64_t w_lo = (static_cast<int64_t>(rank) * kWarps + warp) * per_warp;
    const int lo = a.first + static_cast<int>(w_lo < n ? w_lo : n);
    const int hi = a.first + static_cast<int>(w_lo + per_warp < n ? w_lo + per_warp : n);
    const bool in_shared = per_warp <= cached / kWarps;
    uint32_t* run = keys + warp * per_warp;   // images of lo .. hi - 1
    // f(image) of the lane's part of the run, in no order
    auto each = [&](auto f) {
      const int n_run = hi - lo;
      if (in_shared) {
        int i = 4 * lane;
#pragma unroll 2
        for (; i + 3 < n_run; i += 128) {
          const uint4 k = *reinterpret_cast<const uint4*>(run + i);
          f(k.x);
          f(k.y);
          f(k.z);
          f(k.w);
        }
        for (int e = i; e < min(i + 4, n_run); ++e) f(run[e]);
      } else {
#pragma unroll 4
        for (int i = lane; i < n_run; i += 32) f(mass_key(mass[lo + i]));
      }
    };
    // positions without any weight would spread the range: they and what is below count with the lowest bin at first
    constexpr uint32_t kZeroKey = 0x80000000u;
    uint32_t low = 0xffffffffu, high = 0;
#pragma unroll 16
    for (int i = lo + lane; i < hi; i += 32) {
      const uint32_t key = mass_key(mass[i]);
      if (in_shared) run[i - lo] = key;
      if (key > kZeroKey) low = min(low, key);
      high = max(high, key);
    }
    low = __reduce_min_sync(0xffffffffu, low);
    high = __reduce_max_sync(0xffffffffu, high);
    if (lane == 0) {
      sh.warp_a[warp] = low;
      sh.warp_b[warp] = high;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      low = min(low, sh.warp_a[w]);
      high = max(high, sh.warp_b[w]);
    }
    int n_exchange = 0;
    auto exchange = [&](uint64_t v) {   // v of every block, in sh.totals[slot]
      const int slot = n_exchange++ & 3;
      if (tid < static_cast<int>(n_cta)) st_cluster_u64(map_shared(&sh.totals[slot][rank], tid), v);
      cluster_sync();
      return slot;
    };
    {
      const int slot = exchange(static_cast<uint64_t>(high) << 32 | low);
      for (uint32_t r = 0; r < n_cta; ++r) {
        low = min(low, static_cast<uint32_t>(sh.totals[slot][r]));
        high = max(high, static_cast<uint32_t>(sh.totals[slot][r] >> 32));
      }
    }
    low = min(low, high);
    bool open = true;   // smaller ones than low count in the lowest bin
    // the smallest image that stays lies in [low, high] (open: or below), `above` positions are larger than high
    uint32_t cut = 0xffffffffu, quota = 0, above = 0, gt = 0;
    int n_hist = 0;
    bool done = want == 0, counted = false;
    while (!done) {
      const uint32_t span = high - low;
      int down = 0;
      while ((span >> down) >= static_cast<uint32_t>(kBins)) ++down;
      uint32_t* h = sh.hist[n_hist++ & 1];
      *reinterpret_cast<uint4*>(&h[4 * tid]) = make_uint4(0, 0, 0, 0);
      if (tid == 0) sh.listed = 0;
      __syncthreads();
      each([&](uint32_t key) {
        if (key <= high && (open || key >= low)) red_shared(&h[key < low ? kBins - 1 : (high - key) >> down], 1u);   // from the top
      });
      cluster_sync();
      // each block sums its part of the bins over the cluster (all of it in every block would be eight times the traffic
      // between SMs: 7000 cycles of a cluster of eight instead of 3000)
      const int part = kBins / 4 / static_cast<int>(n_cta);   // of four bins, in threads
      uint4 c = make_uint4(0, 0, 0, 0);
      if (tid < part)
#pragma unroll
        for (int r = 0; r < kMaxCluster; ++r)
          if (r < static_cast<int>(n_cta)) {
            const uint4 t = ld_cluster_v4(map_shared(&h[4 * (static_cast<int>(rank) * part + tid)], r));
            c.x += t.x;
            c.y += t.y;
            c.z += t.z;
            c.w += t.w;
          }
      const uint32_t own = c.x + c.y + c.z + c.w;
      uint32_t incl = own, total = 0;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) sh.warp_a[warp] = incl;
      __syncthreads();
      uint32_t base = above + incl - own;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        const uint32_t t = sh.warp_a[w];
        if (w < warp) base += t;
        total += t;
      }
      const int sums = exchange(total);
      for (uint32_t r = 0; r < rank; ++r) base += static_cast<uint32_t>(sh.totals[sums][r]);
      const uint32_t cs[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        if (base < want && base + cs[k] >= want)
          for (uint32_t r = 0; r < n_cta; ++r)
            st_cluster_v4(map_shared(&sh.found, r), make_uint4(4 * (static_cast<int>(rank) * part + tid) + k, base, cs[k], 0));
        base += cs[k];
      }
      cluster_sync();
      const uint32_t bin = sh.found.x, count = sh.found.z;
      above = sh.found.y;
      const bool rest = open && bin == kBins - 1;
      high = rest && (span >> down) < static_cast<uint32_t>(kBins - 1) ? low - 1 : high - (bin << down);
      low = rest ? 0 : max(low, high - min(high, (1u << down) - 1));
      open = false;
      if (rest) continue;
      if (down == 0) {   // one value: as many of them as it takes
        cut = high;
        quota = want - above;
        break;
      }
      const uint32_t room = kListed / n_cta;
      if (count > static_cast<uint32_t>(kListed) / 2) continue;
      // few positions: their images to every block (as many as a block has room for: else the next range); what is larger
      // than they are is counted on the way
      auto list = [&](uint32_t key) {
        const uint32_t at = atom_shared(&sh.listed, 1u);
        if (at < room) {
          sh.list_warp[at] = static_cast<uint8_t>(warp);
          for (uint32_t r = 0; r < n_cta; ++r) st_cluster_u32(map_shared(&sh.list[rank * room + at], r), key);
        }
      };
      gt = 0;
      uint32_t hits = 0, hit = 0;   // a lane's last one waits for the end, so that most go together
      each([&](uint32_t key) {
        gt += key > high;
        if (key >= low && key <= high) {
          if (hits++) list(hit);
          hit = key;
        }
      });
      if (hits) list(hit);
      gt = __reduce_add_sync(0xffffffffu, gt);
      if (lane == 0) {
        sh.warp_a[warp] = gt;
        sh.warp_b[warp] = 0;
      }
      __syncthreads();
      const int slot = exchange(sh.listed);
      bool fits = true;
      for (uint32_t r = 0; r < n_cta; ++r) fits = fits && sh.totals[slot][r] <= room;
      if (!fits) continue;
      uint32_t ahead = 0, n_all = 0;
      for (uint32_t r = 0; r < n_cta; ++r) {
        const uint32_t m = static_cast<uint32_t>(sh.totals[slot][r]);
        for (uint32_t j = tid; j < m; j += kThreads) sh.flat[n_all + j] = sh.list[r * room + j];
        if (r < rank) ahead += m;
        n_all += m;
      }
      __syncthreads();
      // a warp takes one of this block's at a time, its lanes compare it with all
      for (uint32_t i = warp; i < sh.listed; i += kWarps) {
        const uint32_t key = sh.flat[ahead + i];
        uint32_t larger = 0, equal = 0;
#pragma unroll 4
        for (uint32_t j = lane; j < n_all; j += 32) {
          const uint32_t o = sh.flat[j];
          larger += o > key;
          equal += o == key;
        }
        larger = __reduce_add_sync(0xffffffffu, larger);
        equal = __reduce_add_sync(0xffffffffu, equal);
        if (above + larger < want && above + larger + equal >= want && lane < static_cast<int>(n_cta)) {   // the same for all equal ones
          st_cluster_u32(map_shared(&sh.cut, lane), key);
          st_cluster_u32(map_shared(&sh.quota, lane), want - above - larger);
        }
      }
      cluster_sync();
      cut = sh.cut;
      quota = sh.quota;
      for (uint32_t i = tid; i < sh.listed; i += kThreads) {
        const uint32_t key = sh.list[rank * room + i];
        if (key > cut) atomicAdd(&sh.warp_a[sh.list_warp[i]], 1u);
        if (key == cut) atomicAdd(&sh.warp_b[sh.list_warp[i]], 1u);
      }
      done = counted = true;
    }
    // how many stay before this warp's run
    if (!counted) {
      uint32_t more = 0, equal = 0;
      each([&](uint32_t key) {
        more += key > cut;
        equal += key == cut;
      });
      more = __reduce_add_sync(0xffffffffu, more);
      equal = __reduce_add_sync(0xffffffffu, equal);
      __syncthreads();
      if (lane == 0) {
        sh.warp_a[warp] = more;
        sh.warp_b[warp] = equal;
      }
    }
    __syncthreads();
    uint32_t all_gt = 0, all_eq = 0, eq = 0;
    gt = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) {
        gt += sh.warp_a[w];
        eq += sh.warp_b[w];
      }
      all_gt += sh.warp_a[w];
      all_eq += sh.warp_b[w];
    }
    const int slot = exchange(static_cast<uint64_t>(all_eq) << 32 | all_gt);
    uint32_t equal = 0;
    for (uint32_t r = 0; r < n_cta; ++r) {
      const uint32_t x = static_cast<uint32_t>(sh.totals[slot][r]), y = static_cast<uint32_t>(sh.totals[slot][r] >> 32);
      if (r < rank) {
        gt += x;
        eq += y;
      }
      equal += y;
    }
    const uint32_t below = (1u << lane) - 1;
    if (in_shared && equal <= quota) {   // all that equal the smallest stay: one comparison
      int32_t* to = kept + a.first + gt + eq;
#pragma unroll 4
      for (int i = 0; i < hi - lo; i += 32) {
        const bool stays = i + lane < hi - lo && run[i + lane] >= cut;
        const uint32_t bits = __ballot_sync(0xffffffffu, stays);
        if (stays) to[__popc(bits & below)] = lo + i + lane;
        to += __popc(bits);
      }
    } else {
      for (int i = lo; i < hi; i += 32) {
        const bool in = i + lane < hi;
        const uint32_t key = in ? (in_shared ? run[i + lane - lo] : mass_key(mass[i + lane])) : 0u;
        const uint32_t is_gt = __ballot_sync(0xffffffffu, in && key > cut), is_eq = __ballot_sync(0xffffffffu, in && key == cut);
        const uint32_t e = eq + __popc(is_eq & below);
        if (in && (key > cut || (key == cut && e < quota))) kept[a.first + gt + __popc(is_gt & below) + min(e, quota)] = i + lane;
        gt += __popc(is_gt);
        eq += __popc(is_eq);
      }
    }
  }
  cluster_sync();   // the list

  // Rounds of rows: a lane takes the K or the V of one row, by bulk copies through shared memory.  (With 16-byte loads
  // and stores through registers instead, half the time goes into addresses: 16 prompts to 2048 positions 62 us.)
  constexpr uint32_t kPiece = HD * 2;
  constexpr int kRound = kWarps * kWarpRows;
  const int ps = 1 << shift, which = lane & 1;
  const int32_t* table = a.kv.table + static_cast<int64_t>(b) * a.kv.table_stride;
  const int32_t* out_table = a.out_table + static_cast<int64_t>(b) * a.out_table_stride;
  const bool in_place = a.out_table == a.kv.table;
  // (masses in place: their readers have to be through as well)
  const bool meet = in_place || a.mass_out == a.mass;
  uint8_t* pages = static_cast<uint8_t*>(a.kv.pages) + (static_cast<int64_t>(which) * a.kv.KVH + g) * ps * kPiece;
  const int64_t page_bytes = a.kv.page_stride * 2;
  uint8_t* slot = smem + sizeof(EvictShared) + (warp * 2 * kWarpRows + lane) * kPiece;
  float* mass_out = a.mass_out ? a.mass_out + static_cast<int64_t>(chain) * a.mass_out_stride : nullptr;
  const int64_t i0 = static_cast<int64_t>(a.first) + static_cast<int64_t>(rank) * kRound + warp * kWarpRows + (lane >> 1);
  // a row's way, found a round ahead: positions and pages are loads that wait for one another
  struct Way {
    int src, page, dst;   // dst -2: the row stays where it is
    float mass;
  };
  auto way_of = [&](int64_t i) {
    Way w{-1, -1, -2, 0.0f};
    if (lane >= 2 * kWarpRows || i >= now) return w;
    w.src = __ldcg(&kept[i]);
    if (which == 0 && mass_out) w.mass = __ldcg(&mass[w.src]);
    if (in_place && w.src == i) return w;
    w.page = table[w.src >> shift];
    const int64_t entry = i >> shift;
    w.dst = entry < (a.out_positions >> shift) ? out_table[entry] : -1;
    if (w.dst < 0 || w.dst >= a.kv.n_pages) w.dst = -1;
    if (w.page < 0 || w.page >= a.kv.n_pages) w.page = -1;
    return w;
  };
  uint32_t phase = 0;
  Way way = way_of(i0);
  fence_proxy_async_smem();   // the images are read before the rows overwrite them
  __syncthreads();
  for (int64_t r0 = a.first, i = i0; r0 < now; r0 += kRound * n_cta, i += kRound * n_cta) {
    bool move = way.dst >= 0;
    const bool load = move && way.page >= 0;
    const uint32_t loads = __popc(__ballot_sync(0xffffffffu, load));
    if (lane == 0 && loads) mbar_arrive_expect_tx(&sh.loaded[warp], loads * kPiece);
    __syncwarp();
    if (load) {
      bulk_load_1d(slot, pages + way.page * page_bytes + (way.src & (ps - 1)) * static_cast<int64_t>(kPiece), kPiece, &sh.loaded[warp]);
    } else if (move) {   // NaN in both types
      for (uint32_t k = 0; k < kPiece / 16; ++k) reinterpret_cast<uint4*>(slot)[k] = make_uint4(0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu, 0x7fff7fffu);
      fence_proxy_async_smem();
    }
    if (way.src >= 0 && way.dst != -2 && (way.dst < 0 || way.page < 0) && a.status) atomicOr(a.status, DEX_ATTN_BAD_PAGE);
    const Way next = way_of(i + kRound * n_cta);
    if (loads) {
      if (!mbar_wait(&sh.loaded[warp], phase, nullptr, 0)) {
        move = false;
        if (a.status) atomicOr(a.status, DEX_ATTN_TIMEOUT);
      }
      phase ^= 1;
    }
    __syncwarp();
    if (meet) cluster_sync();
    if (move) bulk_store_1d(pages + way.dst * page_bytes + (i & (ps - 1)) * static_cast<int64_t>(kPiece), slot, kPiece);
    bulk_commit();
    if (which == 0 && way.src >= 0 && mass_out) mass_out[i] = way.mass;
    bulk_wait_read();
    __syncwarp();
    way = next;
  }
  bulk_wait();
  // masses behind the last round's: every block has read what it needs
  if (mass_out)
    for (int64_t i = static_cast<int64_t>(max(now, a.first)) + self; i < len; i += step) mass_out[i] = 0.0f;
}

namespace {

template <int HD>
cudaError_t launch(const EvictArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // Blocks of a cluster: as many as two per SM allow, each with 2048 positions or more of a full table or a round of rows.
  const int64_t chains = static_cast<int64_t>(a.kv.batch) * a.kv.KVH, positions = static_cast<int64_t>(a.kv.table_width) << a.kv.page_shift;
  unsigned n_cta = 1;
  while (n_cta < kMaxCluster && chains * n_cta * 2 <= 2 * n_sm && (positions >= int64_t(4096) * n_cta || a.keep > kWarps * kWarpRows * static_cast<int>(n_cta)))
    n_cta *= 2;
  const int64_t share = (positions + n_cta * kThreads - 1) / (n_cta * kThreads) * kThreads;
  const int cached = static_cast<int>(share < kMove / 4 ? kMove / 4 : share < kCached ? share : kCached);
  if (dev >= 64 || !(done.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(evict_kernel<HD>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(sizeof(EvictShared) + kCached * 4));
    if (e != cudaSuccess) return e;
    if (dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(chains) * n_cta);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = sizeof(EvictShared) + static_cast<size_t>(cached) * 4;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = n_cta;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, evict_kernel<HD>, a, cached);
}

}  // namespace

cudaError_t launch_evict(const EvictArgs& a, cudaStream_t st) { return a.kv.hd == 128 ? launch<128>(a, st) : launch<64>(a, st); }

}  // namespace dex
