// Paged K/V cache: the append kernel (rotary positions applied on the way) and the C entry
// points of the cache (include/dex.h, "paged K/V cache").
#include <math.h>

#include "../../include/dex.h"
#include "common.cuh"
#include "kernels.h"
#include "rope_angle.h"

namespace dex {

namespace {

constexpr int kAppendWarps = 4;   // of a block

__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ void from_f32(__nv_bfloat16& y, float x) { y = __float2bfloat16_rn(x); }
__device__ __forceinline__ void from_f32(__half& y, float x) { y = __float2half_rn(x); }

// Eight consecutive elements as loaded (16 bytes of a 16-bit type, 32 of fp32).  Nothing goes through the
// read-only path: the kernel can be resident before the one that writes its inputs ends.
template <typename T>
struct alignas(16) Vec8 {
  T v[8];
};
template <typename T>
__device__ __forceinline__ Vec8<T> load8(const T* p) {
  Vec8<T> r;
  const uint4* s = reinterpret_cast<const uint4*>(p);
  uint4* d = reinterpret_cast<uint4*>(&r);
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(r) / 16); ++i) d[i] = __ldcg(s + i);
  return r;
}

}  // namespace

// A warp takes one token, or `rows` of its head rows when there are few tokens.  An item is eight pairs
// (x_j, x_{j + HD/2}), j = 8c .. 8c+7, of one head row of q, k or v: two 16-byte loads and two
// 16-byte stores of a 16-bit type.  A lane keeps its c, hence its eight (cos, sin), and walks the rows;
// the first are loaded before the token's table entry is known.  Warps share nothing, so there is no
// block barrier.  Bound by memory: 13498 tokens of 32 + 2 x 8 heads x 128 (332 MB) take 57 us, 5.8 TB/s.
// That takes warps more than loads per warp: 32 of 64 registers per SM with one item each 58 us, with two
// 66 us; 24 warps with two to four items 80 us, 40 warps (48 registers, spills) 70 us.
//
// Angle: the turn of pair j at position r is r * theta^(-2j/HD) / 2 pi.  With the turn of position
// 1 as a 64-bit fixed-point fraction, r times it modulo 2^64 is the fraction of a turn left after
// whole turns, exactly -- an fp32 product r * frequency would be off by 2^-24 r radians (0.06 at
// r = 10^6).  Its upper 32 bits as a signed number are half-turns in units of 2^-31.  theta^(-2j/HD)
// is the product of the powers theta^(-2 2^b / HD) over the bits b of j, each a 64-bit fraction: at position 2^31
// the turn is off by at most 2^-27, and what is left of the error is that of fp32 (2^-21.4 of a row's value).
template <typename CT, typename IT, int HD>
__global__ void __launch_bounds__(32 * kAppendWarps, 8) paged_append_kernel(const __grid_constant__ AppendArgs a, int rows) {
  constexpr int kItems = HD / 16, kStep = 32 / kItems;   // items per head row, rows of one pass of the warp
  __shared__ __align__(16) float2 cs[kAppendWarps][HD / 2];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = lane % kItems;
  const int t = blockIdx.x * kAppendWarps + warp;
  griddep_wait();
  griddep_launch_dependents();
  if (t >= a.n_tokens) return;
  const int end = min((blockIdx.y + 1) * rows, a.H + 2 * a.kv.KVH), v_row0 = a.H + a.kv.KVH;
  const IT* q = static_cast<const IT*>(a.q) + t * a.q_stride + 8 * c;
  const IT* k = static_cast<const IT*>(a.k) + t * a.k_stride + 8 * c;
  const IT* v = static_cast<const IT*>(a.v) + t * a.v_stride + 8 * c;

  Vec8<IT> lo, hi;
  auto load_item = [&](int row) {
    const IT* src = row < a.H ? q + row * HD : row < v_row0 ? k + (row - a.H) * HD : v + (row - v_row0) * HD;
    lo = load8(src);
    hi = load8(src + HD / 2);
  };
  const int first = blockIdx.y * rows + lane / kItems;
  if (first < end) load_item(first);

  const int seq = a.seq[t], pos = a.pos[t], pidx = pos >> a.kv.page_shift;
  bool ok = seq >= 0 && seq < a.kv.batch && pos >= 0 && pidx < a.kv.table_width;
  int page = -1;
  if (ok) {
    page = a.kv.table[static_cast<int64_t>(seq) * a.kv.table_stride + pidx];
    ok = page >= 0 && page < a.kv.n_pages;
  }
  if (!ok) {
    if (seq != -1 && a.rejected && lane == 0 && blockIdx.y == 0) atomicAdd(a.rejected, 1);
    return;
  }
  float4 w[4];   // (cos, sin) of the lane's eight pairs
  if (a.rotate) {
    const int rpos = a.rope_pos ? a.rope_pos[t] : pos;
    for (int j = lane; j < HD / 2; j += 32) {
      uint64_t turn = a.turn;
#pragma unroll
      for (int b = 0; b < 6; ++b)
        if (j >> b & 1) turn = __umul64hi(turn, a.power[b]);
      turn *= static_cast<uint64_t>(static_cast<int64_t>(rpos));
      float s, co;
      sincospif(static_cast<float>(static_cast<int32_t>(turn >> 32)) * 4.656612873077393e-10f, &s, &co);   // 2^-31
      cs[warp][j] = make_float2(co, s);
    }
    __syncwarp();
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = *reinterpret_cast<const float4*>(&cs[warp][8 * c + 2 * i]);
  }

  const int page_size = 1 << a.kv.page_shift, head_stride = page_size * HD;
  CT* q_out = static_cast<CT*>(a.q_out) + t * a.q_out_stride + 8 * c;
  CT* kv_out = static_cast<CT*>(a.kv.pages) + page * a.kv.page_stride + (pos & (page_size - 1)) * HD + 8 * c;
  for (int row = first; row < end; row += kStep) {
    if (row != first) load_item(row);
    Vec8<CT> x, y;
    if (a.rotate && row < v_row0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p0 = to_f32(lo.v[2 * i]), r0 = to_f32(hi.v[2 * i]);
        const float p1 = to_f32(lo.v[2 * i + 1]), r1 = to_f32(hi.v[2 * i + 1]);
        from_f32(x.v[2 * i], p0 * w[i].x - r0 * w[i].y);
        from_f32(y.v[2 * i], r0 * w[i].x + p0 * w[i].y);
        from_f32(x.v[2 * i + 1], p1 * w[i].z - r1 * w[i].w);
        from_f32(y.v[2 * i + 1], r1 * w[i].z + p1 * w[i].w);
      }
    } else if constexpr (sizeof(IT) == 2) {
      x = *reinterpret_cast<const Vec8<CT>*>(&lo);
      y = *reinterpret_cast<const Vec8<CT>*>(&hi);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        from_f32(x.v[i], to_f32(lo.v[i]));
        from_f32(y.v[i], to_f32(hi.v[i]));
      }
    }
    // the V heads of a page follow its K heads
    CT* dst = row < a.H ? q_out + row * HD : kv_out + static_cast<int64_t>(row - a.H) * head_stride;
    *reinterpret_cast<uint4*>(dst) = *reinterpret_cast<const uint4*>(&x);
    *reinterpret_cast<uint4*>(dst + HD / 2) = *reinterpret_cast<const uint4*>(&y);
  }
}

template <typename CT, typename IT, int HD>
static cudaError_t launch_append(const AppendArgs& a, cudaStream_t st) {
  // A warp per token once that gives every SM 16 warps (13498 tokens: 57 us, with 24 rows per warp, which
  // computes the angles twice, 60 us); eight rows per warp below, where latency counts (eight tokens of 48
  // rows: 3.0 us, with 16 rows 3.7 us).
  const int n_rows = a.H + 2 * a.kv.KVH, rows = a.n_tokens >= 16 * 152 ? n_rows : 8;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(static_cast<unsigned>((a.n_tokens + kAppendWarps - 1) / kAppendWarps),
                     static_cast<unsigned>((n_rows + rows - 1) / rows));
  cfg.blockDim = dim3(32 * kAppendWarps);
  cfg.stream = st;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, paged_append_kernel<CT, IT, HD>, a, rows);
}
template <typename CT>
static cudaError_t launch_append_in(const AppendArgs& a, cudaStream_t st) {
  if (a.in_fp32) return a.kv.hd == 128 ? launch_append<CT, float, 128>(a, st) : launch_append<CT, float, 64>(a, st);
  return a.kv.hd == 128 ? launch_append<CT, CT, 128>(a, st) : launch_append<CT, CT, 64>(a, st);
}

cudaError_t launch_paged_append(const AppendArgs& a, cudaStream_t st) {
  return a.kv.fp16 ? launch_append_in<__half>(a, st) : launch_append_in<__nv_bfloat16>(a, st);
}

}  // namespace dex

namespace {

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Positions of a sequence and tokens of a call: a tile beyond the last one still counts in 31 bits, and so do the
// rows of 128 query heads.
constexpr int64_t kMaxPositions = (int64_t(1) << 31) - 512;
constexpr int kMaxTokens = 1 << 23;

// Checks a cache description and fills the kernels' form of it.
int paged_kv(const dex_paged_kv* kv, dex::PagedKv* out) {
  if (!kv || (kv->head_dim != 64 && kv->head_dim != 128) || kv->n_pages < 1 || kv->n_kv_heads < 1 ||
      kv->n_kv_heads > 1024 || kv->batch < 1 || kv->batch > 1024 || kv->table_width < 1 ||
      kv->table_stride < kv->table_width || (kv->dtype != DEX_DT_BF16 && kv->dtype != DEX_DT_FP16))
    return DEX_EINVAL;
  int shift = 4;
  while (shift < 8 && (1 << shift) != kv->page_size) ++shift;
  if ((1 << shift) != kv->page_size) return DEX_EINVAL;
  if (static_cast<int64_t>(kv->table_width) * kv->page_size > kMaxPositions) return DEX_EINVAL;
  const int64_t page_elems = int64_t(2) * kv->n_kv_heads * kv->page_size * kv->head_dim;
  if (kv->page_stride < page_elems || kv->page_stride % 8 || kv->page_stride >= (int64_t(1) << 39)) return DEX_EINVAL;
  out->pages = kv->pages;
  out->table = kv->table;
  out->page_stride = kv->page_stride;
  out->n_pages = kv->n_pages;
  out->page_shift = shift;
  out->KVH = kv->n_kv_heads;
  out->hd = kv->head_dim;
  out->batch = kv->batch;
  out->table_width = kv->table_width;
  out->table_stride = kv->table_stride;
  out->fp16 = kv->dtype == DEX_DT_FP16;
  return DEX_OK;
}

}  // namespace

extern "C" int dex_paged_append(const dex_paged_kv* kv, const dex_append_args* a, int32_t* rejected, void* stream) {
  dex::AppendArgs d = {};
  const int rc = paged_kv(kv, &d.kv);
  if (rc) return rc;
  if (!a || a->n_tokens < 0 || a->n_tokens > kMaxTokens || !kv->pages || !kv->table || !aligned16(kv->pages)) return DEX_EINVAL;
  if (a->in_dtype != kv->dtype && a->in_dtype != DEX_DT_FP32) return DEX_EINVAL;
  if (!(a->rope_theta == 0.0f || (a->rope_theta >= 1.0f && a->rope_theta < INFINITY))) return DEX_EINVAL;
  const int64_t vec = a->in_dtype == DEX_DT_FP32 ? 4 : 8;   // elements in 16 bytes
  if (a->n_tokens > 0) {
    if (!a->k || !a->v || !a->seq || !a->pos || !aligned16(a->k) || !aligned16(a->v) || a->k_stride % vec ||
        a->v_stride % vec || (a->q == nullptr) != (a->q_out == nullptr))
      return DEX_EINVAL;
    if (a->q && (a->n_heads < 1 || a->n_heads > 131072 - 2 * kv->n_kv_heads || !aligned16(a->q) || !aligned16(a->q_out) || a->q_stride % vec ||
                 a->q_out_stride % 8 ||
                 (a->n_tokens > 1 && a->q_out_stride < static_cast<int64_t>(a->n_heads) * kv->head_dim)))
      return DEX_EINVAL;
    if (a->q && a->q == a->q_out && (a->in_dtype != kv->dtype || a->q_stride != a->q_out_stride)) return DEX_EINVAL;
  }
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  if (rejected && cudaMemsetAsync(rejected, 0, sizeof(int32_t), st) != cudaSuccess) return DEX_ECUDA;
  if (a->n_tokens == 0) return DEX_OK;
  d.q = a->q;
  d.k = a->k;
  d.v = a->v;
  d.q_out = a->q_out;
  d.q_stride = a->q_stride;
  d.k_stride = a->k_stride;
  d.v_stride = a->v_stride;
  d.q_out_stride = a->q_out_stride;
  d.seq = a->seq;
  d.pos = a->pos;
  d.rope_pos = a->rope_pos;
  d.n_tokens = a->n_tokens;
  d.H = a->q ? a->n_heads : 0;
  d.in_fp32 = a->in_dtype == DEX_DT_FP32;
  d.rotate = a->rope_theta != 0.0f;
  d.rejected = rejected;
  if (d.rotate) {
    d.turn = dex::kTurnPerRadian;
    dex::rope_powers(a->rope_theta, kv->head_dim, d.power);
  }
  return dex::launch_paged_append(d, st) == cudaSuccess ? DEX_OK : DEX_ECUDA;
}

// Checks an attention call's sizes (host fields only) and fills the kernels' form of it.
static int attention_args(const dex_paged_kv* kv, const dex_attention_args* a, dex::PrefixAttnArgs* d) {
  const int rc = paged_kv(kv, &d->kv);
  if (rc) return rc;
  if (!a || a->n_tokens < 0 || a->n_tokens > kMaxTokens || a->n_heads < 1 || a->n_heads % kv->n_kv_heads ||
      a->n_heads / kv->n_kv_heads > 128 || a->max_q < 1 || a->prefix_len < 0 ||
      a->prefix_len > static_cast<int64_t>(kv->table_width) * kv->page_size)
    return DEX_EINVAL;
  d->n_tokens = a->n_tokens;
  d->H = a->n_heads;
  d->G = a->n_heads / kv->n_kv_heads;
  d->max_q = a->max_q < a->n_tokens ? a->max_q : a->n_tokens > 0 ? a->n_tokens : 1;
  // key tiles, and what segments cost beside them, are counted in 32 bits
  const int64_t tiles = static_cast<int64_t>(kv->table_width) * kv->page_size / 64 + 6;
  const int64_t segs = (static_cast<int64_t>(a->n_tokens) * d->G / 256 + kv->batch + 2) * kv->n_kv_heads;
  if (tiles * segs >= (int64_t(1) << 31)) return DEX_EINVAL;
  d->prefix_len = a->prefix_len;
  return DEX_OK;
}

extern "C" int dex_prefix_attention_workspace(const dex_paged_kv* kv, const dex_attention_args* a, size_t* bytes) {
  dex::PrefixAttnArgs d = {};
  const int rc = attention_args(kv, a, &d);
  if (rc || !bytes) return DEX_EINVAL;
  *bytes = dex::prefix_attention_workspace(d);
  return DEX_OK;
}

extern "C" int dex_prefix_attention(const dex_paged_kv* kv, const dex_attention_args* a, void* workspace,
                                    size_t workspace_bytes, int32_t* status, void* stream) {
  dex::PrefixAttnArgs d = {};
  const int rc = attention_args(kv, a, &d);
  if (rc) return rc;
  const float scale_log2 = a->scale * 1.4426950408889634f;
  if (!kv->pages || !kv->table || !aligned16(kv->pages) || !a->q_start || !a->seq_len || (a->tree_mask && a->max_q > 64) ||
      !(scale_log2 > -INFINITY && scale_log2 < INFINITY))
    return DEX_EINVAL;
  if (a->n_tokens == 0) return DEX_OK;
  const int64_t row = static_cast<int64_t>(a->n_heads) * kv->head_dim;
  if (!a->q || !a->out || !aligned16(a->q) || !aligned16(a->out) || a->q_stride % 8 || a->out_stride % 8 ||
      (a->n_tokens > 1 && a->out_stride < row))
    return DEX_EINVAL;
  const size_t need = dex::prefix_attention_workspace(d);
  if (need && (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255))) return DEX_EINVAL;
  if (workspace_bytes < need) return DEX_ECAPACITY;
  d.q = a->q;
  d.out = a->out;
  d.lse = a->lse;
  d.q_stride = a->q_stride;
  d.out_stride = a->out_stride;
  d.q_start = a->q_start;
  d.seq_len = a->seq_len;
  d.prefix_table = a->prefix_table ? a->prefix_table : kv->table;
  d.tree = a->tree_mask;
  d.scale_log2 = scale_log2;
  d.status = status;
  return dex::launch_prefix_attention(d, workspace, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DEX_OK : DEX_ECUDA;
}

extern "C" int dex_attention_mass(const dex_paged_kv* kv, const dex_mass_args* a, int32_t* status, void* stream) {
  dex::MassArgs d = {};
  const int rc = paged_kv(kv, &d.kv);
  if (rc) return rc;
  if (!a || a->n_tokens < 0 || a->n_tokens > kMaxTokens || a->n_heads < 1 || a->n_heads % kv->n_kv_heads ||
      a->n_heads / kv->n_kv_heads > 128 || a->window < 1 || a->first < 0 || (a->accumulate != 0 && a->accumulate != 1) ||
      a->mass_stride < static_cast<int64_t>(kv->table_width) * kv->page_size || a->mass_stride >= (int64_t(1) << 39))
    return DEX_EINVAL;
  // tiles of 256 positions of all sequences and K/V heads are counted in 32 bits
  if ((static_cast<int64_t>(kv->table_width) * kv->page_size / 256 + 1) * kv->batch * kv->n_kv_heads >= (int64_t(1) << 30))
    return DEX_EINVAL;
  const float scale_log2 = a->scale * 1.4426950408889634f;
  if (!kv->pages || !kv->table || !aligned16(kv->pages) || !a->q_start || !a->seq_len || !a->mass ||
      (reinterpret_cast<uintptr_t>(a->mass) & 3) || !(scale_log2 > -INFINITY && scale_log2 < INFINITY))
    return DEX_EINVAL;
  if (a->n_tokens == 0) return DEX_OK;
  if (!a->q || !a->lse || !aligned16(a->q) || a->q_stride % 8 ||
      (a->n_tokens > 1 && (a->q_stride < static_cast<int64_t>(a->n_heads) * kv->head_dim || a->q_stride >= (int64_t(1) << 38))))
    return DEX_EINVAL;
  d.q = a->q;
  d.lse = a->lse;
  d.mass = a->mass;
  d.q_stride = a->q_stride;
  d.mass_stride = a->mass_stride;
  d.q_start = a->q_start;
  d.seq_len = a->seq_len;
  d.n_tokens = a->n_tokens;
  d.H = a->n_heads;
  d.G = a->n_heads / kv->n_kv_heads;
  d.window = a->window;
  d.first = a->first;
  d.accumulate = a->accumulate;
  d.scale_log2 = scale_log2;
  d.status = status;
  return dex::launch_attention_mass(d, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DEX_OK : DEX_ECUDA;
}

extern "C" int dex_paged_evict(const dex_paged_kv* kv, const dex_evict_args* a, int32_t* status, void* stream) {
  dex::EvictArgs d = {};
  const int rc = paged_kv(kv, &d.kv);
  if (rc) return rc;
  const int64_t cap = static_cast<int64_t>(kv->table_width) * kv->page_size;
  if (!a || a->keep < 1 || a->recent < 0 || a->first < 0 || static_cast<int64_t>(a->first) + a->recent > a->keep ||
      a->mass_stride < cap || a->mass_stride >= (int64_t(1) << 39))
    return DEX_EINVAL;
  if (!kv->pages || !kv->table || !aligned16(kv->pages) || !a->mass || !a->seq_len || !a->new_len || !a->kept ||
      (reinterpret_cast<uintptr_t>(a->new_len) < reinterpret_cast<uintptr_t>(a->seq_len + kv->batch) &&
       reinterpret_cast<uintptr_t>(a->seq_len) < reinterpret_cast<uintptr_t>(a->new_len + kv->batch)) ||
      (reinterpret_cast<uintptr_t>(a->mass) & 3) || (reinterpret_cast<uintptr_t>(a->mass_out) & 3))
    return DEX_EINVAL;
  if (a->mass_out && (a->mass_out_stride < cap || a->mass_out_stride >= (int64_t(1) << 39) ||
                      (a->mass_out == a->mass && a->mass_out_stride != a->mass_stride)))
    return DEX_EINVAL;
  if (a->out_table && (a->out_table_width < 1 || a->out_table_stride < a->out_table_width || a->out_table == kv->table ||
                       static_cast<int64_t>(a->out_table_width) * kv->page_size > kMaxPositions))
    return DEX_EINVAL;
  d.mass = a->mass;
  d.mass_out = a->mass_out;
  d.mass_stride = a->mass_stride;
  d.mass_out_stride = a->mass_out_stride;
  d.seq_len = a->seq_len;
  d.new_len = a->new_len;
  d.kept = a->kept;
  d.out_table = a->out_table ? a->out_table : kv->table;
  d.out_table_stride = a->out_table ? a->out_table_stride : kv->table_stride;
  d.out_positions = static_cast<int32_t>(a->out_table ? static_cast<int64_t>(a->out_table_width) * kv->page_size : cap);
  d.keep = a->keep;
  d.recent = a->recent;
  d.first = a->first;
  d.status = status;
  return dex::launch_evict(d, static_cast<cudaStream_t>(stream)) == cudaSuccess ? DEX_OK : DEX_ECUDA;
}
