// Attention of a ragged batch of queries over a paged K/V cache whose sequences share a prefix.
#include "../../include/dex.h"
#include "common.cuh"
#include "kernels.h"

namespace dex {

namespace {

__device__ __forceinline__ float2 pair_f32(__nv_bfloat162 x) { return __bfloat1622float2(x); }
__device__ __forceinline__ float2 pair_f32(__half2 x) { return __half22float2(x); }
template <typename T> struct PairOf;
template <> struct PairOf<__nv_bfloat16> { using type = __nv_bfloat162; };
template <> struct PairOf<__half> { using type = __half2; };
__device__ __forceinline__ __nv_bfloat162 pair_of(float x, float y, __nv_bfloat162) { return __floats2bfloat162_rn(x, y); }
__device__ __forceinline__ __half2 pair_of(float x, float y, __half2) { return __floats2half2_rn(x, y); }

// The sequence whose queries hold token t, or -1: the last b with q_start[b] <= t.
__device__ __forceinline__ int seq_of_token(const PrefixAttnArgs& a, int t) {
  int lo = 0, hi = a.kv.batch - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (__ldg(a.q_start + mid) <= t) lo = mid;
    else hi = mid - 1;
  }
  return (__ldg(a.q_start + lo) <= t && t < __ldg(a.q_start + lo + 1)) ? lo : -1;
}

}  // namespace

// One warp per (token, query head): every key in turn, the running maximum and sum of the
// softmax in fp32, HD/32 dims per lane.
template <typename T, int HD>
__global__ void __launch_bounds__(128) prefix_attn_kernel(const __grid_constant__ PrefixAttnArgs a) {
  using T2 = typename PairOf<T>::type;
  constexpr int P = HD / 64;   // element pairs per lane
  const int t = blockIdx.x, lane = threadIdx.x & 31;
  const int h = blockIdx.y * 4 + (threadIdx.x >> 5);
  if (h >= a.H) return;
  const int b = seq_of_token(a, t);
  if (b < 0) return;
  const int q0 = __ldg(a.q_start + b), n = __ldg(a.q_start + b + 1) - q0, len = __ldg(a.seq_len + b);
  if (q0 < 0 || n > a.max_q || q0 + n > a.n_tokens) {
    if (a.status) atomicOr(a.status, DEX_ATTN_BAD_RANGE);
    return;
  }
  bool bad = len < 0 || len > (a.kv.table_width << a.kv.page_shift);
  if (bad && a.status) atomicOr(a.status, DEX_ATTN_BAD_RANGE);
  const int first = len - n, p = first + (t - q0);   // first query position, this one's
  const uint64_t tree = a.tree ? a.tree[t] : 0;
  const int end = bad ? 0 : a.tree ? len : p + 1;
  const int page_size = 1 << a.kv.page_shift;
  const int kvh = h / a.G;
  const T2* qp = reinterpret_cast<const T2*>(static_cast<const T*>(a.q) + t * a.q_stride + static_cast<int64_t>(h) * HD);
  float2 q[P], o[P];
#pragma unroll
  for (int i = 0; i < P; ++i) {
    q[i] = pair_f32(qp[i * 32 + lane]);
    o[i] = make_float2(0.f, 0.f);
  }
  float m = -INFINITY, l = 0.f;
  for (int j = 0; j < end; ++j) {
    if (a.tree && j >= first && !((tree >> (j - first)) & 1)) continue;
    const int32_t* tab = j < a.prefix_len ? a.prefix_table : a.kv.table + static_cast<int64_t>(b) * a.kv.table_stride;
    const int page = __ldg(tab + (j >> a.kv.page_shift));
    if (page < 0 || page >= a.kv.n_pages) {
      bad = true;
      if (a.status) atomicOr(a.status, DEX_ATTN_BAD_PAGE);
      break;
    }
    const T* kr = static_cast<const T*>(a.kv.pages) + page * a.kv.page_stride +
                  (static_cast<int64_t>(kvh) * page_size + (j & (page_size - 1))) * HD;
    const T* vr = kr + static_cast<int64_t>(a.kv.KVH) * page_size * HD;
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 k = pair_f32(reinterpret_cast<const T2*>(kr)[i * 32 + lane]);
      s = fmaf(q[i].x, k.x, fmaf(q[i].y, k.y, s));
    }
    s = warp_sum(s) * a.scale_log2;
    const float m1 = fmaxf(m, s), c = exp2f(m - m1), w = exp2f(s - m1);
    m = m1;
    l = l * c + w;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const float2 v = pair_f32(reinterpret_cast<const T2*>(vr)[i * 32 + lane]);
      o[i].x = o[i].x * c + w * v.x;
      o[i].y = o[i].y * c + w * v.y;
    }
  }
  const float inv = bad ? NAN : l > 0.f ? 1.0f / l : 0.f;
  T2* op = reinterpret_cast<T2*>(static_cast<T*>(a.out) + t * a.out_stride + static_cast<int64_t>(h) * HD);
#pragma unroll
  for (int i = 0; i < P; ++i) op[i * 32 + lane] = pair_of(o[i].x * inv, o[i].y * inv, T2());
  if (a.lse && lane == 0)
    a.lse[static_cast<int64_t>(t) * a.H + h] = bad ? NAN : l > 0.f ? (m + log2f(l)) * 0.6931471805599453f : -INFINITY;
}

size_t prefix_attention_workspace(const PrefixAttnArgs&) { return 0; }

cudaError_t launch_prefix_attention(const PrefixAttnArgs& a, void*, cudaStream_t st) {
  const dim3 grid(static_cast<unsigned>(a.n_tokens), static_cast<unsigned>((a.H + 3) / 4));
  if (a.kv.fp16) {
    if (a.kv.hd == 128) prefix_attn_kernel<__half, 128><<<grid, 128, 0, st>>>(a);
    else prefix_attn_kernel<__half, 64><<<grid, 128, 0, st>>>(a);
  } else {
    if (a.kv.hd == 128) prefix_attn_kernel<__nv_bfloat16, 128><<<grid, 128, 0, st>>>(a);
    else prefix_attn_kernel<__nv_bfloat16, 64><<<grid, 128, 0, st>>>(a);
  }
  return cudaGetLastError();
}

}  // namespace dex
