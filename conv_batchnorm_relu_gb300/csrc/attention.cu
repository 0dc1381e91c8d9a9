// Attention, forward and backward (declared in include/cbr.h): plain kernels, a warp for each query or key.
#include "common.cuh"
#include "token_ops.cuh"
#include "trunk_ops.h"

namespace cbr {
namespace {

using namespace tok;

constexpr int kWarps = 8;
constexpr int kPer = 4;   // elements of a head in each lane

struct At {
  int64_t b, t, h;
};

template <typename T>
__device__ __forceinline__ void load(float (&r)[kPer], const void* base, const int64_t* s, int64_t b, int64_t t, int64_t h,
                                     int dim, int lane) {
  const T* p = static_cast<const T*>(base) + b * s[0] + t * s[1] + h * s[2];
#pragma unroll
  for (int i = 0; i < kPer; ++i) r[i] = lane + 32 * i < dim ? to_f(p[lane + 32 * i]) : 0.f;
}

template <typename T>
__device__ __forceinline__ void store(const float (&r)[kPer], void* base, const int64_t* s, int64_t b, int64_t t, int64_t h,
                                      int dim, int lane) {
  T* p = static_cast<T*>(base) + b * s[0] + t * s[1] + h * s[2];
#pragma unroll
  for (int i = 0; i < kPer; ++i)
    if (lane + 32 * i < dim) p[lane + 32 * i] = from_f<T>(r[i]);
}

__device__ __forceinline__ float dot(const float (&a)[kPer], const float (&b)[kPer]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kPer; ++i) s = fmaf(a[i], b[i], s);
  return warp_reduce<Sum>(s);
}

// Keys that sequence b has, and those of them that query i sees.
__device__ __forceinline__ int64_t keys_of(const AttentionArgs& a, int64_t b) {
  return a.key_lengths ? min(max((int64_t)a.key_lengths[b], (int64_t)0), a.d.k_tokens) : a.d.k_tokens;
}
__device__ __forceinline__ int64_t start_of(const AttentionArgs& a, int64_t b) { return a.query_start ? a.query_start[b] : 0; }

// A warp for each query: the forward with a running maximum and sum, or the gradient at the query.
template <typename T, bool kBackward>
__global__ void __launch_bounds__(32 * kWarps) query_kernel(const AttentionArgs a) {
  const cbr_attention_desc_t& d = a.d;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= d.batch * d.heads_q * d.q_tokens) return;
  const int64_t i = row % d.q_tokens, h = row / d.q_tokens % d.heads_q, b = row / d.q_tokens / d.heads_q;
  const int64_t hk = h / (d.heads_q / d.heads_k);
  int64_t n = keys_of(a, b);
  if (d.causal) n = min(n, max(start_of(a, b) + i + 1, (int64_t)0));
  float q[kPer], k[kPer], v[kPer], acc[kPer] = {};
  load<T>(q, a.q, d.q_stride, b, i, h, d.head_dim, lane);
  if constexpr (!kBackward) {
    float m = -INFINITY, l = 0.f;
    for (int64_t j = 0; j < n; ++j) {
      load<T>(k, a.k, d.k_stride, b, j, hk, d.head_dim, lane);
      load<T>(v, a.v, d.v_stride, b, j, hk, d.head_dim, lane);
      const float s = d.scale * dot(q, k);
      const float mn = Max::of(m, s), keep = mn == -INFINITY ? 1.f : expf(m - mn), p = mn == -INFINITY ? 0.f : expf(s - mn);
      m = mn;
      l = l * keep + p;
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = acc[e] * keep + p * v[e];
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] = l == 0.f ? 0.f : acc[e] / l;
    store<T>(acc, a.o, d.o_stride, b, i, h, d.head_dim, lane);
    if (a.lse && lane == 0) a.lse[row] = l == 0.f ? -INFINITY : m + logf(l);
  } else {
    float up[kPer], o[kPer];
    load<T>(up, a.d_o, d.do_stride, b, i, h, d.head_dim, lane);
    load<T>(o, a.o, d.o_stride, b, i, h, d.head_dim, lane);
    const float delta = dot(up, o), lse = a.lse[row];
    if (lane == 0) static_cast<float*>(a.ws)[row] = delta;
    for (int64_t j = 0; j < n; ++j) {
      load<T>(k, a.k, d.k_stride, b, j, hk, d.head_dim, lane);
      load<T>(v, a.v, d.v_stride, b, j, hk, d.head_dim, lane);
      const float ds = expf(d.scale * dot(q, k) - lse) * (dot(up, v) - delta);
#pragma unroll
      for (int e = 0; e < kPer; ++e) acc[e] = fmaf(ds, k[e], acc[e]);
    }
#pragma unroll
    for (int e = 0; e < kPer; ++e) acc[e] *= d.scale;
    store<T>(acc, a.dq, d.dq_stride, b, i, h, d.head_dim, lane);
  }
}

// A warp for each key: its gradients, over the query heads that read it.
template <typename T>
__global__ void __launch_bounds__(32 * kWarps) key_kernel(const AttentionArgs a) {
  const cbr_attention_desc_t& d = a.d;
  const int lane = threadIdx.x & 31;
  const int64_t row = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5);
  if (row >= d.batch * d.heads_k * d.k_tokens) return;
  const int64_t j = row % d.k_tokens, hk = row / d.k_tokens % d.heads_k, b = row / d.k_tokens / d.heads_k;
  const int64_t start = start_of(a, b), first = d.causal ? max(j - start, (int64_t)0) : 0;
  float k[kPer], v[kPer], q[kPer], up[kPer], dk[kPer] = {}, dv[kPer] = {};
  if (j < keys_of(a, b)) {
    load<T>(k, a.k, d.k_stride, b, j, hk, d.head_dim, lane);
    load<T>(v, a.v, d.v_stride, b, j, hk, d.head_dim, lane);
    for (int g = 0; g < d.heads_q / d.heads_k; ++g) {
      const int64_t h = hk * (d.heads_q / d.heads_k) + g;
      for (int64_t i = first; i < d.q_tokens; ++i) {
        load<T>(q, a.q, d.q_stride, b, i, h, d.head_dim, lane);
        load<T>(up, a.d_o, d.do_stride, b, i, h, d.head_dim, lane);
        const int64_t at = (b * d.heads_q + h) * d.q_tokens + i;
        const float p = expf(d.scale * dot(q, k) - a.lse[at]);
        const float ds = p * (dot(up, v) - static_cast<const float*>(a.ws)[at]);
#pragma unroll
        for (int e = 0; e < kPer; ++e) dk[e] = fmaf(ds, q[e], dk[e]), dv[e] = fmaf(p, up[e], dv[e]);
      }
    }
  }
#pragma unroll
  for (int e = 0; e < kPer; ++e) dk[e] *= d.scale;
  store<T>(dk, a.dk, d.dk_stride, b, j, hk, d.head_dim, lane);
  store<T>(dv, a.dv, d.dv_stride, b, j, hk, d.head_dim, lane);
}

int launched() { return cudaGetLastError() == cudaSuccess ? CBR_OK : CBR_ERR_CUDA; }

template <typename T>
int backward(const AttentionArgs& a, cudaStream_t st) {
  const int64_t rows = a.d.batch * a.d.heads_q * a.d.q_tokens, keys = a.d.batch * a.d.heads_k * a.d.k_tokens;
  if (rows) query_kernel<T, true><<<(unsigned)((rows + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(a);
  if (keys) key_kernel<T><<<(unsigned)((keys + kWarps - 1) / kWarps), 32 * kWarps, 0, st>>>(a);
  return launched();
}

}  // namespace

size_t attention_backward_ws(const cbr_attention_desc_t& d) { return (size_t)d.batch * d.heads_q * d.q_tokens * 4; }

int launch_attention_backward(const AttentionArgs& a, cudaStream_t st) {
  return a.d.dtype == CBR_BF16 ? backward<__nv_bfloat16>(a, st) : backward<__half>(a, st);
}

}  // namespace cbr
