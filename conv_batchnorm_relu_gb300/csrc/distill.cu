// Distillation from a teacher's top logits, forward and backward (formulas: include/cbr.h).
//
// One block a row.  The row's largest logit, then the sum of exponentials (over all words and over
// those the teacher does not list, told apart by one bit a word in shared memory), then the
// gradient, each a sweep over the row; the teacher's entries are a short vector beside it.
#include <algorithm>

#include "cbr_internal.h"
#include "token_ops.cuh"

namespace cbr {
namespace {

using namespace tok;

constexpr int kThreads = 512;

struct Teacher {
  float mass;   // sum of p over the entries
  float rest;   // the tail's probability
  float norm;   // p_k = exp(t_k / T - norm) * inv
  float inv;
  bool any;     // whether the row has anything to learn from
};

__device__ __forceinline__ long long entry_id(const DistillArgs& a, long long row, int k) {
  const long long i = row * a.d.ids_stride + k;
  const long long id = a.d.id_bytes == 8 ? static_cast<const long long*>(a.top_ids)[i]
                                         : (long long)static_cast<const int*>(a.top_ids)[i];
  return id >= 0 && id < a.d.vocab ? id : -1;
}

__device__ __forceinline__ float entry_logit(const DistillArgs& a, long long row, int k) {
  return load_as_float(a.top_logits, a.d.top_dtype, row * a.d.top_stride + k);
}

__device__ __forceinline__ float entry_p(const Teacher& t, float x) { return __expf(x - t.norm) * t.inv; }

__device__ Teacher teacher_of(const DistillArgs& a, long long row, float inv_t, float* red) {
  Teacher t;
  float top = -INFINITY, any = 0.f;
  for (int k = threadIdx.x; k < (int)a.d.topk; k += kThreads) {
    if (entry_id(a, row, k) < 0) continue;
    const float x = entry_logit(a, row, k) * inv_t;
    top = fmaxf(top, x);
    if (a.teacher_lse || !(x == -INFINITY)) any = 1.f;
  }
  t.any = block_reduce<Max>(any, red) > 0.f;
  top = block_reduce<Max>(top, red);
  t.norm = a.teacher_lse ? a.teacher_lse[row] : (top == -INFINITY ? 0.f : top);
  t.inv = 1.f;
  float s = 0.f;
  for (int k = threadIdx.x; k < (int)a.d.topk; k += kThreads)
    if (entry_id(a, row, k) >= 0) s += entry_p(t, entry_logit(a, row, k) * inv_t);
  s = block_reduce<Sum>(s, red);
  if (a.teacher_lse) {
    t.mass = s;
    t.rest = fmaxf(0.f, 1.f - s);
  } else {
    t.mass = 1.f;
    t.inv = 1.f / s;
    t.rest = 0.f;
  }
  return t;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) distill_kernel(DistillArgs a) {
  extern __shared__ uint32_t listed[];
  __shared__ float red[32];
  const int words = (int)((a.d.vocab + 31) / 32);
  const float inv_t = 1.f / a.d.temperature;
  for (long long row = blockIdx.x; row < a.d.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.logits) + row * a.d.logits_stride;
    T* dx = a.dlogits ? static_cast<T*>(a.dlogits) + row * a.d.dlogits_stride : nullptr;
    const float w = a.row_weight ? a.row_weight[row] : 1.f;
    Teacher t{};
    float top = 0.f, total = 0.f, unlisted = 0.f;
    if (w != 0.f) {
      t = teacher_of(a, row, inv_t, red);
      for (int i = threadIdx.x; i < words; i += kThreads) listed[i] = 0;
      __syncthreads();
      for (int k = threadIdx.x; k < (int)a.d.topk; k += kThreads) {
        const long long id = entry_id(a, row, k);
        if (id >= 0) atomicOr(&listed[id >> 5], 1u << (id & 31));
      }
      __syncthreads();
    }
    bool live = w != 0.f && t.any;
    if (live) {
      top = -INFINITY;
      for (int v = threadIdx.x; v < (int)a.d.vocab; v += kThreads) top = Max::of(top, to_f(x[v]));
      top = block_reduce<Max>(top, red);
      live = top != -INFINITY;
      float s = 0.f, u = 0.f;
      for (int v = threadIdx.x; v < (int)a.d.vocab; v += kThreads) {
        const float e = __expf((to_f(x[v]) - top) * inv_t);
        s += e;
        if (!(listed[v >> 5] >> (v & 31) & 1u)) u += e;
      }
      total = block_reduce<Sum>(s, red);
      unlisted = block_reduce<Sum>(u, red);
    }
    const float q_rest = unlisted / total;
    if (!(q_rest > 0.f) && q_rest == q_rest) t.rest = 0.f;
    float l = 0.f;
    if (live) {
      for (int k = threadIdx.x; k < (int)a.d.topk; k += kThreads) {
        const long long id = entry_id(a, row, k);
        if (id < 0) continue;
        const float xt = entry_logit(a, row, k) * inv_t;
        const float p = entry_p(t, xt);
        const float log_q = (to_f(x[id]) - top) * inv_t - logf(total);
        if (!(p == 0.f)) l += p * (xt - t.norm + logf(t.inv) - log_q);
      }
      l = block_reduce<Sum>(l, red);
      if (t.rest != 0.f) l += t.rest * (logf(t.rest) - logf(q_rest));
    }
    if (threadIdx.x == 0) {
      a.loss[row] = live ? l * w * a.d.temperature * a.d.temperature : 0.f;
      if (a.stats) {
        a.stats[row * 3] = live ? top : 0.f;
        a.stats[row * 3 + 1] = live ? total : 0.f;
        a.stats[row * 3 + 2] = live ? unlisted : 0.f;
      }
    }
    if (!dx) continue;
    const float scale = w * a.d.temperature;
    const float all = t.mass + t.rest, some = t.rest != 0.f ? all - t.rest / q_rest : all;
    for (int v = threadIdx.x; v < (int)a.d.vocab; v += kThreads) {
      float g = 0.f;
      if (live) {
        const float q = __expf((to_f(x[v]) - top) * inv_t) / total;
        const bool in = listed[v >> 5] >> (v & 31) & 1u;
        g = q * (in ? all : some);
        if (in)
          for (int k = 0; k < (int)a.d.topk; ++k)
            if (entry_id(a, row, k) == v) g -= entry_p(t, entry_logit(a, row, k) * inv_t);
        g *= scale;
      }
      dx[v] = from_f<T>(g);
    }
    __syncthreads();
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) distill_backward_kernel(DistillArgs a) {
  extern __shared__ uint32_t listed[];
  __shared__ float red[32];
  const int words = (int)((a.d.vocab + 31) / 32);
  const float inv_t = 1.f / a.d.temperature;
  for (long long row = blockIdx.x; row < a.d.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.logits) + row * a.d.logits_stride;
    T* dx = static_cast<T*>(a.dlogits) + row * a.d.dlogits_stride;
    const float w = a.row_weight ? a.row_weight[row] : 1.f;
    const float top = a.stats[row * 3], total = a.stats[row * 3 + 1], unlisted = a.stats[row * 3 + 2];
    bool live = w != 0.f && !(total == 0.f);
    Teacher t{};
    if (live) {
      t = teacher_of(a, row, inv_t, red);
      live = t.any;
      for (int i = threadIdx.x; i < words; i += kThreads) listed[i] = 0;
      __syncthreads();
      for (int k = threadIdx.x; k < (int)a.d.topk; k += kThreads) {
        const long long id = entry_id(a, row, k);
        if (id >= 0) atomicOr(&listed[id >> 5], 1u << (id & 31));
      }
      __syncthreads();
    }
    const float q_rest = unlisted / total;
    if (!(q_rest > 0.f) && q_rest == q_rest) t.rest = 0.f;
    const float scale = w * a.d.temperature * (a.dloss ? a.dloss[row] : 1.f);
    const float all = t.mass + t.rest, some = t.rest != 0.f ? all - t.rest / q_rest : all;
    for (int v = threadIdx.x; v < (int)a.d.vocab; v += kThreads) {
      float g = 0.f;
      if (live) {
        const float q = __expf((to_f(x[v]) - top) * inv_t) / total;
        const bool in = listed[v >> 5] >> (v & 31) & 1u;
        g = q * (in ? all : some);
        if (in)
          for (int k = 0; k < (int)a.d.topk; ++k)
            if (entry_id(a, row, k) == v) g -= entry_p(t, entry_logit(a, row, k) * inv_t);
        g *= scale;
      }
      dx[v] = from_f<T>(g);
    }
    __syncthreads();
  }
}

template <typename K>
int launch(K kernel, const DistillArgs& a, int num_sms, cudaStream_t st) {
  const int smem = (int)((a.d.vocab + 31) / 32) * 4;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kernel), 64 * 1024)) return CBR_ERR_CUDA;
  const int grid = (int)std::min<long long>(a.d.rows, (long long)num_sms * 4);
  kernel<<<grid, kThreads, smem, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? CBR_OK : CBR_ERR_CUDA;
}

}  // namespace

int launch_distill(const DistillArgs& a, int num_sms, cudaStream_t st) {
  if (a.d.dtype == CBR_F32) return launch(distill_kernel<float>, a, num_sms, st);
  if (a.d.dtype == CBR_BF16) return launch(distill_kernel<__nv_bfloat16>, a, num_sms, st);
  return launch(distill_kernel<__half>, a, num_sms, st);
}

int launch_distill_backward(const DistillArgs& a, int num_sms, cudaStream_t st) {
  if (a.d.dtype == CBR_F32) return launch(distill_backward_kernel<float>, a, num_sms, st);
  if (a.d.dtype == CBR_BF16) return launch(distill_backward_kernel<__nv_bfloat16>, a, num_sms, st);
  return launch(distill_backward_kernel<__half>, a, num_sms, st);
}

}  // namespace cbr
