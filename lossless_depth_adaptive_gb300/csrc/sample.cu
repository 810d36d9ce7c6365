// Sampling a token from a row of logits: temperature, top-k, top-p, min-p, then the first token up to which more
// than u of the remaining mass lies.
//
// One cluster of blocks per row, each with a slice of the row in shared memory; logits are read once.  Weights
// are 43-bit fractions of the largest (weight_of), so masses are exact integer sums: no order of summation,
// number of blocks or atomic changes a token.  Each is off by up to two units of 2^-43, and one below half a unit is nothing, so the border
// between two tokens of a row of V is off by at most 2 V units (2^-24 of the largest weight for the longest row; some sqrt(V) where
// errors fall both ways).
//
// No limit sorts the row.  What top-k or top-p cuts off begins at one token, the last that stays in the order of
// descending logits (equal ones: ascending ids), and everything else is a comparison with it.  It is found among candidates: few
// tokens that contain it, sent to every block, each block ranking its own among all, a comparison per pair.
//  * A small top-k: a thread has the largest of its part of the slice anyway, and the k-th largest of these maxima is at
//    most the k-th largest logit; a histogram of the maxima in eighths of an octave gives a threshold with some more than k tokens
//    above it.  They are all that matters from there on, so the first block finishes the row with them.  So are those of a
//    small nucleus, given the mass of the row.
//  * Another top-p, and a large top-k: a histogram of masses (counts) over the row in 1/22 octaves, summed through distributed
//    shared memory, gives the bin that holds the token; its tokens are the candidates.
// Masses of the whole row are first summed from rough weights, good to 2^-18 of themselves; where the borders that decide the row are not clear of what those sums may be off by, it is done again with exact weights.
// Where the candidates are too many (equal logits, mostly), bits of the order-preserving images of the bin's logits are
// counted, ten at a time, and then the ids.
//
// What bounds it.  Few rows: latency, some 25 steps of 500-3000 cycles (cluster barriers 700, a histogram's sums over the
// cluster 4000), many of them code that runs once or twice: 8 rows of 32000 fp32, top-p 19.2 us (31 where a row takes exact weights, one call
// of 27); 15 rows of 128256 fp16, min-p 13.1; 64 rows of 151936 bf16, top-k
// 50 and top-p 16.8.  Many rows: the issue of instructions between barriers (two blocks per SM; 49 % of the issue slots, HBM
// 11 %): 256 rows of 151936 fp32 greedy 45 us, top-k 50 93, temperature alone 162, top-p at temperature 0.5 170, where most
// rows are so flat that it takes exact weights 440; settings of their own 178.
#include <math.h>

#include <atomic>

#include <cuda_fp16.h>

#include "../../include/dex.h"
#include "cluster.cuh"
#include "common.cuh"
#include "kernels.h"
#include "sample_weight.h"

namespace dex {

namespace {

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kBins = 2 * kThreads;    // of a histogram over the row
constexpr int kMaxCluster = 8;
constexpr float kZeroOctaves = 45.0f;  // weights this far below the largest are zero
constexpr int kMaxBins = kThreads;     // of the histogram of maxima: an eighth of an octave each
constexpr int kZeroBin = 8 * 45 + 8;   // its bins from here on hold zero weights
constexpr int kFlat = kThreads;        // candidates of a row
constexpr int kListed = 2 * kFlat;     // room for them, divided among its blocks
constexpr int kPerWarp = 64;           // candidates of a warp's run
constexpr int kMostK = 256;            // top-k by maxima up to here
constexpr uint32_t kNucleus = 128;     // and top-p alone, if the nucleus lies among the tokens above this many maxima

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float from_key(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k); }
template <typename T> __device__ __forceinline__ T minus_inf();
template <> __device__ __forceinline__ float minus_inf<float>() { return -INFINITY; }
template <> __device__ __forceinline__ __nv_bfloat16 minus_inf<__nv_bfloat16>() { return __ushort_as_bfloat16(0xFF80); }
template <> __device__ __forceinline__ __half minus_inf<__half>() { return __ushort_as_half(0xFC00); }

template <typename T> __device__ __forceinline__ T to_nan();
template <> __device__ __forceinline__ float to_nan<float>() { return __int_as_float(0x7fffffff); }
template <> __device__ __forceinline__ __nv_bfloat16 to_nan<__nv_bfloat16>() { return __ushort_as_bfloat16(0x7fff); }
template <> __device__ __forceinline__ __half to_nan<__half>() { return __ushort_as_half(0x7fff); }

struct alignas(16) Candidate {
  uint32_t key, id;
  uint64_t w;
};
struct alignas(16) Rank {
  uint64_t before;   // mass of the larger ones
  uint32_t rank, pad;
};

// What shares memory is never in use at the same time on any block: a histogram is read by the others before the
// barrier of the lists, candidates are put in one row after it; a warp's finds go to the lists before it, ranks arrive after it.
struct alignas(16) Shared {
  Candidate list[kListed];       // block r's from r * kListed / blocks on
  union {
    uint32_t hist[2][kBins];     // lower and upper words
    Candidate flat[kFlat];       // the candidates of all blocks, in the order of their ids
  };
  union {
    struct {
      float x;
      int id;
    } finds[kWarps][kPerWarp];
    Rank ranks[kFlat];           // in the first block
  };
  uint32_t maxima[kMaxBins];
  uint64_t warp_sum[kWarps];
  uint32_t warp_count[kWarps];
  uint64_t totals[4][kMaxCluster];   // of every block of the cluster, written by each of them
  uint32_t counts[kMaxCluster];      // candidates of every block, kOverflow: too many
  uint64_t found[4];
  uint64_t cut;                      // key and id of the last token that stays, written by the block that found it
  uint64_t loaded[kWarps];           // mbarriers of the warps' runs
  Pair table[kWeightTable];
};
constexpr uint32_t kOverflow = 1u << 20;
constexpr size_t kHead = (sizeof(Shared) + 15) / 16 * 16;
constexpr size_t kMostBytes = 227 * 1024;
static_assert(kHead + (1 << 18) / kMaxCluster * 4 + 16 <= kMostBytes, "a slice of the longest row");

template <typename T>
__global__ void __launch_bounds__(kThreads, 2) sample_kernel(const __grid_constant__ SampleArgs a, int slice) {
  extern __shared__ __align__(16) uint8_t smem[];
  Shared& sh = *reinterpret_cast<Shared*>(smem);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const uint32_t rank = cluster_rank(), n_cta = cluster_size();
  const int row = blockIdx.x / n_cta;
  const int v0 = static_cast<int>(rank) * slice, count = min(slice, max(0, a.vocab - v0));
  // a warp's run of the slice, in the order of the ids: run + 32 s + lane
  const int run = warp * (slice / kWarps), steps = slice / kThreads;

  // The slice lies in shared memory with its address's remainder by 16, so that a run's inner part is one bulk copy.
  const T* src = static_cast<const T*>(a.logits) + row * a.logits_stride + v0;
  T* xs = reinterpret_cast<T*>(smem + kHead + (reinterpret_cast<uintptr_t>(src) & 15));
  if (lane == 0) mbar_init(&sh.loaded[warp], 1);
  fence_mbar_init();
  __syncwarp();
  cluster_started_arrive();
  griddep_wait();
  griddep_launch_dependents();
  {
    const int lo = min(run, count), hi = min(run + slice / kWarps, count);
    const uintptr_t p0 = reinterpret_cast<uintptr_t>(src + lo), p1 = reinterpret_cast<uintptr_t>(src + hi);
    const uintptr_t in0 = (p0 + 15) & ~uintptr_t(15), in1 = p1 & ~uintptr_t(15);
    const bool bulk = in1 > in0;
    const int first = bulk ? static_cast<int>((in0 - p0) / sizeof(T)) : hi - lo, end = bulk ? static_cast<int>((p1 - in1) / sizeof(T)) : 0;
    if (bulk && lane == 0) {
      mbar_arrive_expect_tx(&sh.loaded[warp], static_cast<uint32_t>(in1 - in0));
      bulk_load_1d(xs + lo + first, reinterpret_cast<const void*>(in0), static_cast<uint32_t>(in1 - in0), &sh.loaded[warp]);
    }
    if (lane < first) xs[lo + lane] = src[lo + lane];          // (16 bytes and less: no more elements than lanes)
    if (lane < end) xs[hi - end + lane] = src[hi - end + lane];
    for (int i = max(run, count) + lane; i < run + slice / kWarps; i += 32) xs[i] = minus_inf<T>();
    if (tid < kWeightTable) sh.table[tid] = pair_of(weight_table_entry(tid));
    sh.maxima[tid] = 0;
    if (bulk && !mbar_wait(&sh.loaded[warp], 0, nullptr, 0)) xs[lo] = to_nan<T>();   // (never: the row gets no token)
    __syncwarp();
  }
  const float temp = a.temperature ? a.temperature[row] : a.temperature_all;
  const float top_p = a.top_p ? a.top_p[row] : a.top_p_all, min_p = a.min_p ? a.min_p[row] : a.min_p_all;
  int top_k = a.top_k ? a.top_k[row] : a.top_k_all;
  if (top_k >= a.vocab || top_k < 0) top_k = 0;
  const float u = a.u[row];
  if (a.n_exclude > 0) {
    __syncthreads();
    for (int i = tid; i < a.n_exclude; i += kThreads) {
      const int64_t at = static_cast<int64_t>(a.exclude[row * a.exclude_stride + i]) - v0;
      if (at >= 0 && at < count) xs[at] = minus_inf<T>();
    }
    __syncthreads();
  }
  auto x_at = [&](int s) { return to_f32(xs[run + 32 * s + lane]) + 0.0f; };   // -0 is 0
  auto id_at = [&](int s) { return v0 + run + 32 * s + lane; };

  int n_exchange = 0;
  // v of every block, in sh.totals[n_exchange]; the value is the block's thread 0's
  auto exchange = [&](uint64_t v) {
    const int slot = n_exchange++ & 3;
    if (tid < static_cast<int>(n_cta)) st_cluster_u64(map_shared(&sh.totals[slot][rank], tid), v);
    cluster_sync();
    return slot;
  };
  auto block_sum = [&](uint64_t v) {   // the same in every thread
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    __syncthreads();
    if (lane == 0) sh.warp_sum[warp] = v;
    __syncthreads();
    uint64_t t = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) t += sh.warp_sum[w];
    return t;
  };
  auto warp_scan = [&](uint64_t v) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint64_t t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    return v;
  };
  // Sum of v over the threads of all blocks, the part of the blocks before this one in `before`; warp_sum has the warps'.
  auto total_of = [&](uint64_t v, uint64_t& before) {
    const int slot = exchange(block_sum(v));
    uint64_t all = 0;
    before = 0;
    for (uint32_t r = 0; r < n_cta; ++r) {
      const uint64_t t = sh.totals[slot][r];
      if (r < rank) before += t;
      all += t;
    }
    return all;
  };
  // Sum of measure(x, id) over the row, the part of the blocks before this one in `before`; warp_sum has the warps'.
  auto sums = [&](auto measure, uint64_t& before) {
    uint64_t v = 0;
    for (int s = 0; s < steps; ++s) v += measure(x_at(s), id_at(s));
    return total_of(v, before);
  };
  // The lowest id up to which measure adds up to target, given what sums() left: in the one warp that holds it, else -1 (-2: not even
  // there).  (before becomes the sum up to it, without it)
  auto locate = [&](auto measure, uint64_t& before, uint64_t target) {
    for (int w = 0; w < warp; ++w) before += sh.warp_sum[w];
    if (!(before < target && before + sh.warp_sum[warp] >= target)) return -1;
    // a lane adds up `steps` consecutive ones, then the warp goes through those of the lane that holds it
    uint64_t v = 0;
    const int part0 = run + lane * steps;
#pragma unroll 4
    for (int s = 0; s < steps; ++s) v += measure(to_f32(xs[part0 + s]) + 0.0f, v0 + part0 + s);
    const uint64_t upto = before + warp_scan(v);
    const uint32_t owners = __ballot_sync(0xffffffffu, upto >= target);
    if (owners == 0) return -2;   // (sums of rough weights differ with the order)
    const int owner = __ffs(owners) - 1;
    before = __shfl_sync(0xffffffffu, upto - v, owner);
    const int from = run + owner * steps;
    for (int s = 0; s < steps; s += 32) {
      const uint64_t m = s + lane < steps ? measure(to_f32(xs[from + s + lane]) + 0.0f, v0 + from + s + lane) : 0, incl = warp_scan(m);
      const uint32_t hit = __ballot_sync(0xffffffffu, before + incl >= target);
      if (hit) {
        before += __shfl_sync(0xffffffffu, incl - m, __ffs(hit) - 1);
        return v0 + from + s + __ffs(hit) - 1;
      }
      before += __shfl_sync(0xffffffffu, incl, 31);
    }
    return -2;
  };
  auto answer = [&](int id, float logprob) {
    a.tokens[row] = id;
    if (a.logprob) a.logprob[row] = logprob;
  };
  // ---- the largest logit; a row with NaN or +inf has no answer
  float most = -INFINITY;   // of the thread's
  bool bad = false;
  auto look = [&](float x, int) {
    bad |= !(x < INFINITY);
    most = fmaxf(most, x);
  };
  const bool aligned = (reinterpret_cast<uintptr_t>(src) & 15) == 0;   // 16 bytes at a time, in another order
  constexpr int kVec = 16 / sizeof(T);
  const int wide = aligned ? slice / kWarps / (32 * kVec) : 0;
  // f(x, id) of the lane's part of the run, in no order
  auto each = [&](auto f) {
#pragma unroll 2
    for (int s = 0; s < wide; ++s) {
      const int i = run + (32 * s + lane) * kVec;
      const uint4 v = *reinterpret_cast<const uint4*>(xs + i);
      const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int k = 0; k < kVec; ++k) f(to_f32(e[k]) + 0.0f, v0 + i + k);
    }
#pragma unroll 4
    for (int s = wide * kVec; s < steps; ++s) f(x_at(s), id_at(s));
  };
  each(look);
  {
    const float m = warp_max(most);
    if (lane == 0) sh.warp_sum[warp] = ordered_key(m);
  }
  bad = __syncthreads_or(bad);
  uint64_t best = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) best = max(best, sh.warp_sum[w]);
  {
    cluster_started_wait();
    const int slot = exchange(bad ? ~0ull : best);
    for (uint32_t r = 0; r < n_cta; ++r) best = max(best, sh.totals[slot][r]);
  }
  const float top = from_key(static_cast<uint32_t>(best));
  if (best == ~0ull || top == -INFINITY || !(temp >= 0.0f && temp < INFINITY) || top_p != top_p || min_p != min_p || u != u) {
    if (rank == 0 && tid == 0) answer(-1, __int_as_float(0x7fffffff));
    return;   // (nothing of another block is read after an exchange)
  }
  if (temp == 0.0f || top_k == 1 || top_p <= 0.0f) {
    uint32_t id = 0xffffffffu;
    if (__any_sync(0xffffffffu, most == top))   // (the thread's largest is of another part of the run than x_at's)
      for (int s = steps - 1; s >= 0; --s)
        if (x_at(s) == top) id = id_at(s);
    id = __reduce_min_sync(0xffffffffu, id);
    if (lane == 0) sh.warp_count[warp] = id;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) id = min(id, sh.warp_count[w]);
    const int slot = exchange(id);
    for (uint32_t r = 0; r < n_cta; ++r) id = min(id, static_cast<uint32_t>(sh.totals[slot][r]));
    if (rank == 0 && tid == 0) answer(static_cast<int>(id), 0.0f);
    return;
  }

  // Hot rows (their weights are mostly one) are weighed exactly at once: rough weights have no room to scale logits, and below
  // -3e38 they cannot tell -inf from a logit that counts.
  const float down = temp >= kHot ? kHotScale : 1.0f;
  const Pair c = octaves_per_unit(temp * down);
  const float per_unit = c.hi * down;   // octaves
  const bool rough = temp < kHot && c.hi < INFINITY;
  auto weight = [&](float x) { return weight_of(x, top, c, sh.table, down); };
  // The log of the share that a token of weight w has of the mass.  What it is drawn by are whole units of 2^-43; the share of one that
  // is not most of the mass goes by its logit.
  auto share_of = [&](float x, uint64_t w, uint64_t mass) {
    if (2 * w > mass) return log1pf(-(static_cast<float>(mass - w) / static_cast<float>(mass)));
    return log_share(x == top ? Pair{0.0f, 0.0f} : octaves_of(x, top, c, down), mass);
  };
  const float far = fmaxf(-128.0f / per_unit, -3.0e38f);
  auto near = [&](float x) { return weight_near(x, top, c, far); };
  auto near_units = [&](float x) { return in_units(near(x)); };
  auto rough_sum = [&] {   // of the thread's, four at a time as floats
    uint64_t sum = 0;
    float some = 0.0f;
    int n = 0;
    each([&](float x, int) {
      some += near(x);
      if ((++n & 3) == 0) {
        sum += in_units(some);
        some = 0.0f;
      }
    });
    return sum + in_units(some);
  };
  constexpr float kTwo43 = 8796093022208.0f, kTwo64 = 18446744073709551616.0f;
  const uint64_t least = static_cast<uint64_t>(ceilf(fminf(fmaxf(min_p, 0.0f), 1.0f) * kTwo43));
  const uint64_t part = fmaxf(u, 0.0f) >= 1.0f ? ~0ull : static_cast<uint64_t>(fmaxf(u, 0.0f) * kTwo64);   // u 2^64
  // less than top_p of the mass before a token: the sum up to the last that stays reaches the smallest integer not less than that
  const uint64_t p64 = top_p < 1.0f ? static_cast<uint64_t>(top_p * kTwo64) : 0;
  auto nucleus = [&](uint64_t mass) {
    const uint64_t t = __umul64hi(p64, mass) + (p64 * mass != 0);
    return t < 1 ? uint64_t(1) : t > mass ? mass : t;
  };
  auto scan32 = [&](uint32_t v) {   // inclusive
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t t = __shfl_up_sync(0xffffffffu, v, o);
      if (lane >= o) v += t;
    }
    return v;
  };

  // The tokens for which is(x) holds go to every block, in the order of their ids, with measure(x, id).  False: too many.
  // skip: whether the warp has none.
  uint32_t all, own, ahead;   // candidates of all blocks, of this one, of the blocks before it
  auto collect = [&](bool skip, auto is, auto measure) {
    uint32_t mine = 0;
    for (int s = 0; s < (skip ? 0 : wide); ++s) {   // 16 bytes at a time: mostly there is nothing
      const int i = run + (32 * s + lane) * kVec;
      const uint4 v = *reinterpret_cast<const uint4*>(xs + i);
      const T* e = reinterpret_cast<const T*>(&v);
      uint32_t hits = 0;
#pragma unroll
      for (int k = 0; k < kVec; ++k) hits |= static_cast<uint32_t>(is(to_f32(e[k]) + 0.0f, v0 + i + k)) << k;
      if (!__any_sync(0xffffffffu, hits != 0)) continue;
      const uint32_t n = __popc(hits);
      uint32_t at = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const uint32_t t = __shfl_up_sync(0xffffffffu, at, o);
        if (lane >= o) at += t;
      }
      const uint32_t all_hits = __shfl_sync(0xffffffffu, at, 31);
      at += mine - n;
#pragma unroll
      for (int k = 0; k < kVec; ++k)
        if (hits >> k & 1) {
          if (at < kPerWarp) {
            sh.finds[warp][at].x = to_f32(e[k]) + 0.0f;
            sh.finds[warp][at].id = v0 + i + k;
          }
          ++at;
        }
      mine += all_hits;
    }
    if (!skip)
#pragma unroll 4
      for (int s = wide * kVec; s < steps; ++s) {
        const float x = x_at(s);
        const bool it = is(x, id_at(s));
        const uint32_t b = __ballot_sync(0xffffffffu, it);
        if (b) {
          const uint32_t at = mine + __popc(b & ((1u << lane) - 1));
          if (it && at < kPerWarp) {
            sh.finds[warp][at].x = x;
            sh.finds[warp][at].id = id_at(s);
          }
          mine += __popc(b);
        }
      }
    if (lane == 0) sh.warp_count[warp] = mine;
    const bool over = __syncthreads_or(mine > kPerWarp);
    uint32_t first = 0;
    own = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint32_t n = sh.warp_count[w];
      if (w < warp) first += n;
      own += n;
    }
    const uint32_t room = kListed / n_cta;
    if (!over && own <= room) {
      for (uint32_t i = lane; i < mine; i += 32) {
        const float x = sh.finds[warp][i].x;
        const int id = sh.finds[warp][i].id;
        const uint64_t m = measure(x, id);
        const uint4 v = make_uint4(ordered_key(x), static_cast<uint32_t>(id), static_cast<uint32_t>(m), static_cast<uint32_t>(m >> 32));
        for (uint32_t r = 0; r < n_cta; ++r) st_cluster_v4(map_shared(&sh.list[rank * room + first + i], r), v);
      }
    }
    if (tid < static_cast<int>(n_cta)) st_cluster_u32(map_shared(&sh.counts[rank], tid), over || own > room ? kOverflow : own);
    cluster_sync();
    all = 0;
    ahead = 0;
    uint32_t at = 0, from = 0;   // of candidate tid, in the lists
    for (uint32_t r = 0; r < n_cta; ++r) {
      const uint32_t n = sh.counts[r];
      if (static_cast<uint32_t>(tid) >= all) {
        from = r * room;
        at = tid - all;
      }
      if (r < rank) ahead += n;
      all += n;
    }
    if (all > kFlat) return false;
    if (static_cast<uint32_t>(tid) < all) sh.flat[tid] = sh.list[from + at];
    __syncthreads();
    return true;
  };
  // Of this block's candidate i: how many are larger, and the sum of their measures.  The whole warp, a part per lane.
  auto rank_of = [&](const Candidate& me) {
    uint32_t larger = 0;
    uint64_t w = 0;
#pragma unroll 4
    for (uint32_t j = lane; j < all; j += 32) {
      const Candidate o = sh.flat[j];
      if (o.key > me.key || (o.key == me.key && o.id < me.id)) {
        ++larger;
        w += o.w;
      }
    }
    // (a lane's sum is below 2^48)
    const uint64_t lo = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(w) & 0xffffffu), hi = __reduce_add_sync(0xffffffffu, static_cast<uint32_t>(w >> 24));
    return Rank{lo + (hi << 24), __reduce_add_sync(0xffffffffu, larger), 0};
  };

  float cut = -INFINITY;   // a token stays where its logit and id are not behind these
  int last = a.vocab;

  // ---- few tokens that matter: the first block finishes the row
  // The nucleus of most rows is small.  Looked for here where a thread has 16 logits and more.  In us, so and by the histogram alone, at
  // temperature 0.5, where nuclei are small in most rows, and at 1, where they are not: 256 rows of 151936 fp32 171 and 254, 441 and 463; 256 of 50257 74
  // and 104, 154 and 153; 8 rows of 65536 (16 per thread) 13 and 22, 50 and 46; 64 rows of 151936 bf16 64 and 55, 170 and 161.  With fewer logits per
  // thread most is gained and lost: 8 rows of 50257 (13) 13 and 21, 44 and 41; 8 of 32000 (8) 12.5 and 18.9, 26 and 21.
  const bool few_p = top_k == 0 && top_p < 1.0f && rough && steps >= 16;
  const bool by_maxima = few_p || (top_k > 0 && top_k <= kMostK);
  if (by_maxima || (top_k == 0 && top_p >= 1.0f && least > 0)) {
    uint64_t row_mass = 0;   // few_p: of the whole row, roughly
    bool worth = true;
    int threshold;   // (products with per_unit in an order in which none overflows before it is compared)
    if (by_maxima) {
      const int b = most == top ? 0 : static_cast<int>(fminf(mul_rn(sub_rn(top, most), per_unit) * 8.0f, kMaxBins - 1.0f));
      red_shared(&sh.maxima[b], 1u);
      if (few_p) {
        uint64_t before;
        row_mass = total_of(rough_sum(), before);
      } else {
        cluster_sync();
      }
      uint32_t n = 0;
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < static_cast<int>(n_cta)) n += ld_cluster_u32(map_shared(&sh.maxima[tid], r));
      uint32_t incl = scan32(n);
      if (lane == 31) sh.warp_count[warp] = incl;
      if (tid == 0) sh.found[0] = kZeroBin;
      __syncthreads();
      for (int w = 0; w < warp; ++w) incl += sh.warp_count[w];
      const uint32_t need = few_p ? kNucleus : static_cast<uint32_t>(top_k);
      if (incl - n < need && incl >= need) sh.found[0] = min(tid, kZeroBin);
      __syncthreads();
      threshold = static_cast<int>(sh.found[0]) + 1;
      if (few_p) {   // a nucleus that these maxima do not come near (their weights, about, in units of 2^-20) is not looked for here
        const float about = tid < threshold ? static_cast<float>(n) * exp2_fast(-0.125f * static_cast<float>(tid)) : 0.0f;
        const uint64_t held = block_sum(static_cast<uint64_t>(about * 1048576.0f));
        worth = held + (held >> 2) >= nucleus(row_mass) >> (kWeightBits - 20);
      }
    } else {   // weights of min_p and more, and some others
      threshold = static_cast<int>(fminf(8.0f * (1.0f - log2f(fminf(min_p, 1.0f))), static_cast<float>(kZeroBin)));
    }
    // as a logit, somewhat lower than it need be (where weights have no room: the largest alone; where all have: all)
    const float far = static_cast<float>(threshold) * 0.125f / per_unit;
    const float from = top - far - (fabsf(top) + far) * 1e-6f;
    bool few = worth && collect(!__any_sync(0xffffffffu, most >= from), [&](float x, int) { return x >= from; }, [&](float x, int) { return weight(x); });
    uint64_t end = 0, off = 0;   // few_p: the nucleus ends where the mass before a token reaches `end`, which may be that much off
    if (few && few_p) {
      const uint64_t held = block_sum(static_cast<uint32_t>(tid) < all ? sh.flat[tid].w : 0);
      end = nucleus(row_mass);
      off = rough_slack(held, (threshold + 2) * 0.125f) + rough_slack(row_mass - min(row_mass, held), kZeroOctaves);
      few = held >= end + off;   // else it is not all here
    }
    if (few) {
      if (by_maxima) {
        bool unsure = false;
        for (uint32_t i = warp; i < own; i += kWarps) {
          const Rank k = rank_of(sh.flat[ahead + i]);
          unsure |= few_p && k.rank > 0 && k.before + off >= end && k.before < end + off;
          if (lane == 0)
            st_cluster_v4(map_shared(&sh.ranks[ahead + i], 0), make_uint4(static_cast<uint32_t>(k.before), static_cast<uint32_t>(k.before >> 32), k.rank, 0));
        }
        if (few_p) {
          const uint32_t any = __syncthreads_or(unsure);
          const int slot = exchange(any);
          for (uint32_t r = 0; r < n_cta; ++r) few = few && !sh.totals[slot][r];
        } else {
          cluster_sync();
        }
      }
    }
    if (few) {
      if (rank != 0) return;
      uint64_t w = static_cast<uint32_t>(tid) < all ? sh.flat[tid].w : 0;
      if (by_maxima) {
        const Rank k = sh.ranks[tid];
        if (top_k > 0 && k.rank >= static_cast<uint32_t>(top_k)) w = 0;
        if (top_p < 1.0f && !few_p) end = nucleus(block_sum(w));   // (the same for all threads: they meet in block_sum)
        if (top_p < 1.0f && k.rank > 0 && k.before >= end) w = 0;
      }
      if (w < least) w = 0;
      uint64_t incl = warp_scan(w), mass = 0;
      __syncthreads();
      if (lane == 31) sh.warp_sum[warp] = incl;
      __syncthreads();
#pragma unroll
      for (int v = 0; v < kWarps; ++v) {
        const uint64_t t = sh.warp_sum[v];
        if (v < warp) incl += t;
        mass += t;
      }
      const uint64_t target = __umul64hi(part, mass) + 1;   // more than u of the mass
      if (incl - w < target && incl >= target) answer(static_cast<int>(sh.flat[tid].id), share_of(from_key(sh.flat[tid].key), w, mass));
      return;
    }
    if (!few_p) cut = from;   // what is lower has no chance
  }

  // ---- over the whole row
  auto in_cut = [&](float x, int id) { return x > cut || (x == cut && id <= last); };
  // Where a logit lies below the largest: in steps of 1 / (22 kBins) octave, the bin and in its lower digits the bin's own bins.
  constexpr int kFineBits = 10;
  static_assert(kBins == 1 << kFineBits, "digits");
  constexpr float kPerOctave = kBins * ((kBins - 1) / kZeroOctaves);
  auto fine = [&](float x) {   // (starts as weight_near does)
    const float y = mul_rn(fmaxf(sub_rn(x, top), far), per_unit);
    return x == top ? 0 : static_cast<int>(fminf(mul_rn(y, -kPerOctave), kBins * kBins - 1.0f));
  };
  // Sums of measure by bins (bin_of: -1 for none) over the row; returns the total, and the bin in which the running sum plus `above`
  // reaches target(total); above grows by what is before it, in_bin is what is in it.
  uint64_t in_bin, in_all;
  auto histogram = [&](auto bin_of, auto measure, auto target_of, uint64_t& above, int& bin) {
    *reinterpret_cast<uint2*>(&sh.hist[0][2 * tid]) = make_uint2(0, 0);
    *reinterpret_cast<uint2*>(&sh.hist[1][2 * tid]) = make_uint2(0, 0);
    __syncthreads();
    each([&](float x, int id) {
      const uint64_t m = measure(x, id);
      const int o = m ? bin_of(x) : -1;
      if (o >= 0) {   // a 64-bit sum in two words, with the carry
        const uint32_t lo = static_cast<uint32_t>(m), old = atom_shared(&sh.hist[0][o], lo);
        const uint32_t carry = static_cast<uint32_t>(m >> 32) + (old + lo < old);
        if (carry) red_shared(&sh.hist[1][o], carry);
      }
    });
    cluster_sync();
    // each block sums its part of the bins over the cluster
    const int part = kBins / 2 / static_cast<int>(n_cta), first = 2 * (static_cast<int>(rank) * part + tid);
    ulonglong2 n = make_ulonglong2(0, 0);   // of the thread's two bins
    if (tid < part)
#pragma unroll
      for (int r = 0; r < kMaxCluster; ++r)
        if (r < static_cast<int>(n_cta)) {
          const uint2 lo = ld_cluster_v2(map_shared(&sh.hist[0][first], r)), hi = ld_cluster_v2(map_shared(&sh.hist[1][first], r));
          n.x += static_cast<uint64_t>(hi.x) << 32 | lo.x;
          n.y += static_cast<uint64_t>(hi.y) << 32 | lo.y;
        }
    uint64_t incl = warp_scan(n.x + n.y), total = 0;
    if (lane == 31) sh.warp_sum[warp] = incl;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const uint64_t t = sh.warp_sum[w];
      if (w < warp) incl += t;
      total += t;
    }
    if (tid == 0) sh.found[0] = kBins;   // (read by nobody between the barriers here)
    const int slot = exchange(total);
    total = 0;
    for (uint32_t r = 0; r < n_cta; ++r) {
      const uint64_t t = sh.totals[slot][r];
      if (r < rank) incl += t;
      total += t;
    }
    in_all = total;
    const uint64_t target = target_of(total), b2 = above + incl, b1 = b2 - n.y, b0 = b1 - n.x;
    const bool in_x = b0 < target && b1 >= target, in_y = b1 < target && b2 >= target;
    if (in_x || in_y)
      for (uint32_t r = 0; r < n_cta; ++r) {
        st_cluster_u64(map_shared(&sh.found[0], r), first + in_y);
        st_cluster_u64(map_shared(&sh.found[1], r), in_y ? b1 : b0);
        st_cluster_u64(map_shared(&sh.found[2], r), in_y ? n.y : n.x);
      }
    cluster_sync();
    bin = static_cast<int>(sh.found[0]);
    above = sh.found[1];
    in_bin = sh.found[2];
    return target;
  };
  // Moves the cut to where the measure of what stays, largest first, reaches target_of(its total).  rough_of: what is summed over the
  // row; unless that is exact too, false where it does not tell.
  float depth = kZeroOctaves;   // of the cut, in octaves
  auto select = [&](auto rough_of, auto measure, auto target_of, bool exact) {
    uint64_t above = 0;
    int bin;
    auto of_cut = [&](float x, int id) { return in_cut(x, id) ? measure(x) : uint64_t(0); };
    auto sum_of = [&](float x, int id) { return in_cut(x, id) ? rough_of(x) : uint64_t(0); };
    const uint64_t target = histogram([&](float x) { return fine(x) >> kFineBits; }, sum_of, target_of, above, bin), sum = in_all;
    if (bin >= kBins - 1) return exact;   // among the zero weights, or not at all: nothing is cut
    int low = bin << kFineBits, high = low + kBins - 1;
    // logits between which these are, and not much more (a cheaper question than fine)
    auto down_by = [&](float steps) { return steps * (1.0f / kPerOctave) / per_unit; };   // (a single step may be too small for a float)
    float x_low, x_high;
    auto limits = [&] {
      const float wide = 1e-6f * (fabsf(top) + down_by(high));
      x_low = down_by(1.0f) < 1e30f ? top - down_by(high + 2) - wide : -INFINITY;
      x_high = down_by(1.0f) < 1e30f ? top - down_by(low - 2) + wide : INFINITY;
    };
    const uint64_t middle = rough_of(top - down_by((bin + 0.5f) * kBins));   // the weight of the bin's tokens, about
    depth = (high + 1) / kPerOctave;
    // (the target is at most as much off as the sum that it is a part of)
    if (!exact && middle < 2 * (2 * rough_slack(above, depth) + rough_slack(sum - above, kZeroOctaves))) return false;   // it would hardly tell
    if (in_bin > (kFlat / 2) * middle) {   // many tokens: the bin's own bins
      cluster_sync();   // (the histogram's own barriers would do)
      limits();
      histogram(
          [&](float x) {
            const int f = fine(x);
            return f >> kFineBits == bin ? f & (kBins - 1) : -1;
          },
          [&](float x, int id) { return x >= x_low && x <= x_high ? sum_of(x, id) : uint64_t(0); }, [&](uint64_t) { return target; }, above, high);
      if (high >= kBins) return false;   // (only with rough sums)
      low = high += low;
    }
    if (tid == 0) sh.cut = 0;
    constexpr uint32_t kSure = 0x80000000u;
    limits();
    auto there = [&](float x, int id) {
      if (!(x >= x_low && x <= x_high)) return false;
      const int f = fine(x);
      return f >= low && f <= high && in_cut(x, id);
    };
    if (collect(false, there, of_cut)) {
      const uint64_t off = exact ? 0 : 2 * rough_slack(above, depth) + rough_slack(sum - above, kZeroOctaves);
      for (uint32_t i = warp; i < own; i += kWarps) {
        const Candidate me = sh.flat[ahead + i];
        const uint64_t to = above + rank_of(me).before;
        if (lane < static_cast<int>(n_cta) && to + off < target && to + me.w >= target + off)
          st_cluster_u64(map_shared(&sh.cut, lane), static_cast<uint64_t>(me.key) << 32 | me.id | kSure);
      }
      cluster_sync();
      const uint64_t found = sh.cut;
      cluster_sync();   // (before the next one is written)
      if (!(found & kSure)) return false;
      cut = from_key(static_cast<uint32_t>(found >> 32));
      last = static_cast<int>(static_cast<uint32_t>(found) & ~kSure);
      return true;
    }
    if (!exact) return false;
    uint32_t prefix = 0, mask = 0;
    for (int pass = 0; pass < 4; ++pass) {
      const int at = pass < 3 ? 22 - 10 * pass : 0, ones = pass < 3 ? 1023 : 3;
      cluster_sync();   // (as above)
      int digit;
      histogram(
          [&](float x) {
            const uint32_t key = ordered_key(x);
            return fine(x) >= low && fine(x) <= high && (key & mask) == prefix ? ones - static_cast<int>(key >> at & ones) : -1;
          },
          [&](float x, int id) { return x >= x_low && x <= x_high ? of_cut(x, id) : uint64_t(0); }, [&](uint64_t) { return target; }, above, digit);
      prefix |= static_cast<uint32_t>(ones - digit) << at;
      mask |= static_cast<uint32_t>(ones) << at;
    }
    // equal logits: as many of them as it takes, by their ids
    auto equal = [&](float x, int id) { return ordered_key(x) == prefix ? of_cut(x, id) : uint64_t(0); };
    uint64_t before;
    sums(equal, before);
    const int id = locate(equal, before, target - above);
    if (id >= 0 && lane < static_cast<int>(n_cta)) st_cluster_u64(map_shared(&sh.cut, lane), id);
    cluster_sync();
    cut = from_key(prefix);
    last = static_cast<int>(sh.cut);
    cluster_sync();
    return true;
  };
  // The token among what stays; false where rough weights do not tell.  Its log-probability may go by a mass of rough weights: off by
  // each one's 2^-21 and by 2^-24 ln 2 per octave, of which the tokens of a row lie, by their shares, at most log2(vocab) <= 18
  // below the largest (else their entropy would be more than that), so by 2^-19.6; a float's step at a log of -16 is 2^-19.
  auto finish = [&](auto units_of, bool exact) {
    auto enough = [&](float x, uint64_t w) {   // min-p
      if (least == 0) return w;
      const uint64_t off = (w >> 18) + 4;
      if (w + off < least) return uint64_t(0);
      return w > least + off || weight(x) >= least ? w : uint64_t(0);
    };
    auto stays = [&](float x, int id) { return in_cut(x, id) ? enough(x, units_of(x)) : uint64_t(0); };
    uint64_t mine = 0;
    if (cut == -INFINITY && least == 0) {
      if (exact) {
        each([&](float x, int) { mine += units_of(x); });
      } else {
        mine = rough_sum();
      }
    } else {   // few of many: a warp puts them side by side and weighs 32 at a time
      float* x_of = &sh.finds[warp][0].x;   // 128 of them
      uint32_t n = 0;
#pragma unroll 4
      for (int s = 0; s < steps; ++s) {
        const float x = x_at(s);
        const bool is = in_cut(x, id_at(s));
        const uint32_t b = __ballot_sync(0xffffffffu, is);
        if (b == 0) continue;
        if (is) x_of[n + __popc(b & ((1u << lane) - 1))] = x;
        n += __popc(b);
        if (n >= 32) {
          __syncwarp();
          const float x0 = x_of[lane], next = x_of[32 + lane];
          mine += enough(x0, units_of(x0));
          __syncwarp();
          x_of[lane] = next;
          n -= 32;
        }
      }
      __syncwarp();
      if (lane < static_cast<int>(n)) mine += enough(x_of[lane], units_of(x_of[lane]));
      __syncwarp();
    }
    uint64_t before;
    const uint64_t mass = total_of(mine, before), target = __umul64hi(part, mass) + 1;   // more than u of the mass
    const int id = locate(stays, before, target);
    bool sure = id != -2;
    if (id >= 0) {
      const float x = to_f32(xs[id - v0]) + 0.0f;
      const uint64_t w = stays(x, id), off = exact ? 0 : rough_slack(mass, depth) + rough_slack(before, depth);
      sure = exact || (before + off < target && before + w >= target + off);
      if (sure && lane == 0) answer(id, share_of(x, weight(x), mass));
    }
    if (exact) return true;
    const uint32_t unsure = __syncthreads_or(!sure);
    const int slot = exchange(unsure);
    for (uint32_t r = 0; r < n_cta; ++r)
      if (sh.totals[slot][r]) return false;
    return true;
  };
  if (top_k > 0) {
    auto one = [](float) { return uint64_t(1); };
    select(one, one, [&](uint64_t) { return static_cast<uint64_t>(top_k); }, true);
  }
  const float cut_k = cut;
  const int last_k = last;
  // (also with few logits per thread: 8 rows of 32000 with top-p 19 us, weighed exactly at once 20.5 when this came in)
  if (rough && (top_p >= 1.0f || select(near_units, weight, nucleus, false)) && finish(near_units, false)) return;
  cut = cut_k;
  last = last_k;
  if (top_p < 1.0f) select(weight, weight, nucleus, true);
  finish(weight, true);
}

template <typename T>
cudaError_t launch(const SampleArgs& a, cudaStream_t st) {
  static std::atomic<uint64_t> done{0};   // devices where the kernel may have the shared memory of the longest row
  int dev = 0, n_sm = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e == cudaSuccess) e = cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev);
  if (e != cudaSuccess) return e;
  // Blocks of a row.  Few rows: eight, for the latency (8 rows of 32000 fp32 with top-p 19 us, with four 25.5; 8 rows of 151936, flat, 73 and
  // 116).  Where eight would not all be resident at two blocks per SM, four, if two of those fit an SM (64 rows of 151936 bf16 with top-k 16.9 us, with
  // eight 26; 256 rows of 32000 fp32 with top-p 61 and 146).  Else eight: with four there is one block per SM (256 rows of 151936 fp32, temperature
  // alone 161 us, with four 204; settings of their own 190 and 229; top-k 50 93 and 90).
  const auto bytes_of = [&](int n) { return kHead + static_cast<size_t>((a.vocab + n * kThreads - 1) / (n * kThreads) * kThreads) * sizeof(T) + 16; };
  const unsigned n_cta = a.n_rows * 8 > 2 * n_sm && bytes_of(4) <= 112 * 1024 ? 4 : 8;
  const int slice = (a.vocab + static_cast<int>(n_cta) * kThreads - 1) / (static_cast<int>(n_cta) * kThreads) * kThreads;
  const size_t bytes = kHead + static_cast<size_t>(slice) * sizeof(T) + 16;
  if (dev >= 64 || !(done.load(std::memory_order_relaxed) >> dev & 1)) {
    e = cudaFuncSetAttribute(sample_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMostBytes));
    if (e != cudaSuccess) return e;
    if (dev < 64) done.fetch_or(uint64_t(1) << dev, std::memory_order_relaxed);
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>(a.n_rows) * n_cta);
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = bytes;
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
  return cudaLaunchKernelEx(&cfg, sample_kernel<T>, a, slice);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs& a, cudaStream_t st) {
  if (a.dtype == DEX_DT_FP32) return launch<float>(a, st);
  return a.dtype == DEX_DT_FP16 ? launch<__half>(a, st) : launch<__nv_bfloat16>(a, st);
}

}  // namespace dex

extern "C" int dex_sample(const dex_sample_args* a, void* stream) {
  if (!a || a->n_rows < 0 || a->n_rows > (1 << 20) || a->vocab < 1 || a->vocab > (1 << 18) || a->dtype < DEX_DT_BF16 ||
      a->dtype > DEX_DT_FP32 || a->n_exclude < 0 || a->n_exclude > 1024)
    return DEX_EINVAL;
  if (!a->temperature && !(a->temperature_all >= 0.0f && a->temperature_all < INFINITY)) return DEX_EINVAL;
  if (!a->top_k && a->top_k_all < 0) return DEX_EINVAL;
  if (!a->top_p && !(a->top_p_all > 0.0f && a->top_p_all <= 1.0f)) return DEX_EINVAL;
  if (!a->min_p && !(a->min_p_all >= 0.0f && a->min_p_all <= 1.0f)) return DEX_EINVAL;
  if (a->n_rows == 0) return DEX_OK;
  const uintptr_t size = a->dtype == DEX_DT_FP32 ? 4 : 2;
  if (!a->logits || reinterpret_cast<uintptr_t>(a->logits) % size || !a->u || !a->tokens ||
      (a->n_exclude > 0 && (!a->exclude || a->exclude_stride < a->n_exclude)))
    return DEX_EINVAL;
  dex::SampleArgs d = {};
  d.logits = a->logits;
  d.logits_stride = a->logits_stride;
  d.u = a->u;
  d.temperature = a->temperature;
  d.top_k = a->top_k;
  d.top_p = a->top_p;
  d.min_p = a->min_p;
  d.temperature_all = a->temperature_all;
  d.top_k_all = a->top_k_all;
  d.top_p_all = a->top_p_all;
  d.min_p_all = a->min_p_all;
  d.exclude = a->exclude;
  d.exclude_stride = a->exclude_stride;
  d.n_exclude = a->n_exclude;
  d.n_rows = a->n_rows;
  d.vocab = a->vocab;
  d.dtype = a->dtype;
  d.tokens = a->tokens;
  d.logprob = a->logprob;
  return dex::launch_sample(d, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DEX_OK : DEX_ECUDA;
}
