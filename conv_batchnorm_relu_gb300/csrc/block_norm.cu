// The norms around a gated residual block, forward and backward (formulas: include/cbr.h).
//
// One block a row; a thread owns the columns threadIdx.x, threadIdx.x + kThreads, ...  The
// backward's blocks walk runs of consecutive rows and add the parameter gradients of their run
// into block-private sums, which a second kernel adds up in a fixed order.
#include <algorithm>

#include "cbr_internal.h"
#include "token_ops.cuh"

namespace cbr {
namespace {

using namespace tok;

constexpr int kThreads = 256;
constexpr int kBlocksPerSm = 4;

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_forward_kernel(BlockNormArgs a) {
  __shared__ float red[32];
  const int dim = (int)a.d.dim;
  const float inv_d = 1.f / (float)dim;
  const bool center = a.d.kind == CBR_NORM_LAYER;
  for (long long row = blockIdx.x; row < a.d.rows; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.x) + row * a.d.x_stride;
    const T* f = a.branch ? static_cast<const T*>(a.branch) + row * a.d.branch_stride : nullptr;
    const float* gate = a.gate ? a.gate + row / a.d.gate_rows * dim : nullptr;
    float m1 = 0.f, r1 = 0.f, m2 = 0.f, r2 = 0.f;
    if (f) {
      if (center) {
        float s = 0.f;
        for (int c = threadIdx.x; c < dim; c += kThreads) s += to_f(f[c]);
        m1 = block_reduce<Sum>(s, red) * inv_d;
      }
      float s = 0.f;
      for (int c = threadIdx.x; c < dim; c += kThreads) s += (to_f(f[c]) - m1) * (to_f(f[c]) - m1);
      r1 = 1.f / sqrtf(block_reduce<Sum>(s, red) * inv_d + a.d.eps);
    }
    auto joined = [&](int c) {
      if (!f) return to_f(x[c]);
      const float n = (to_f(f[c]) - m1) * r1 * a.post_weight[c];
      return a.d.residual_scale * to_f(x[c]) + a.d.branch_scale * (gate ? gate[c] * n : n);
    };
    if (a.pre_weight) {
      if (center) {
        float s = 0.f;
        for (int c = threadIdx.x; c < dim; c += kThreads) s += joined(c);
        m2 = block_reduce<Sum>(s, red) * inv_d;
      }
      float s = 0.f;
      for (int c = threadIdx.x; c < dim; c += kThreads) s += (joined(c) - m2) * (joined(c) - m2);
      r2 = 1.f / sqrtf(block_reduce<Sum>(s, red) * inv_d + a.d.eps);
    }
    __syncthreads();
    for (int c = threadIdx.x; c < dim; c += kThreads) {
      const float v = joined(c);
      if (a.pre_weight)
        static_cast<T*>(a.h)[row * a.d.h_stride + c] = from_f<T>((v - m2) * r2 * a.pre_weight[c]);
      if (f) static_cast<T*>(a.x_out)[row * a.d.x_out_stride + c] = from_f<T>(v);
    }
    if (a.stats && threadIdx.x == 0) {
      float* s = a.stats + row * 4;
      s[0] = m1, s[1] = r1, s[2] = m2, s[3] = r2;
    }
  }
}

// The gate-gradient rows of a run of rows [first, last): a gate whose rows all lie in the run is
// written by the run's block; the others (at most the run's first and last) go to the block's two
// partial rows.
__host__ __device__ inline long long run_rows(long long rows, int blocks) { return (rows + blocks - 1) / blocks; }

template <typename T>
__global__ void __launch_bounds__(kThreads) norm_backward_kernel(BlockNormArgs a) {
  __shared__ float red[32];
  const int dim = (int)a.d.dim;
  const float inv_d = 1.f / (float)dim;
  const bool center = a.d.kind == CBR_NORM_LAYER;
  const long long run = run_rows(a.d.rows, gridDim.x), first = blockIdx.x * run, last = min(first + run, (long long)a.d.rows);
  float* sums = a.part + (long long)blockIdx.x * 4 * dim;   // pre_weight, post_weight, two gate rows
  for (int c = threadIdx.x; c < 4 * dim; c += kThreads) sums[c] = 0.f;
  __syncthreads();
  for (long long row = first; row < last; ++row) {
    const T* xo = static_cast<const T*>(a.x) + row * a.d.x_out_stride;
    const T* f = a.branch ? static_cast<const T*>(a.branch) + row * a.d.branch_stride : nullptr;
    const T* dxo = a.dx_out ? static_cast<const T*>(a.dx_out) + row * a.d.dx_out_stride : nullptr;
    const T* dh = a.pre_weight ? static_cast<const T*>(a.dh) + row * a.d.dh_stride : nullptr;
    const long long group = a.gate ? row / a.d.gate_rows : 0;
    const float* gate = a.gate ? a.gate + group * dim : nullptr;
    float* dgate = nullptr;
    if (gate) {
      const bool whole = group * a.d.gate_rows >= first && (group + 1) * a.d.gate_rows <= last;
      dgate = whole ? a.dgate + group * dim : sums + (2 + (group != first / a.d.gate_rows)) * dim;
      if (whole && row == group * a.d.gate_rows)
        for (int c = threadIdx.x; c < dim; c += kThreads) dgate[c] = 0.f;
    }
    const float* s4 = a.stats + row * 4;
    const float m1 = s4[0], r1 = s4[1], m2 = s4[2], r2 = s4[3];
    float mu = 0.f, mc = 0.f;
    if (dh) {
      float s = 0.f, t = 0.f;
      for (int c = threadIdx.x; c < dim; c += kThreads) {
        const float n = (to_f(xo[c]) - m2) * r2, u = to_f(dh[c]) * a.pre_weight[c];
        s += u;
        t += u * n;
      }
      if (center) mu = block_reduce<Sum>(s, red) * inv_d;
      mc = block_reduce<Sum>(t, red) * inv_d;
    }
    auto full = [&](int c) {
      float d = dxo ? to_f(dxo[c]) : 0.f;
      if (dh) d += r2 * (to_f(dh[c]) * a.pre_weight[c] - mu - (to_f(xo[c]) - m2) * r2 * mc);
      return d;
    };
    float mv = 0.f, me = 0.f;
    if (f) {
      float s = 0.f, t = 0.f;
      for (int c = threadIdx.x; c < dim; c += kThreads) {
        const float e = (to_f(f[c]) - m1) * r1, v = a.d.branch_scale * full(c) * (gate ? gate[c] : 1.f) * a.post_weight[c];
        s += v;
        t += v * e;
      }
      if (center) mv = block_reduce<Sum>(s, red) * inv_d;
      me = block_reduce<Sum>(t, red) * inv_d;
    }
    for (int c = threadIdx.x; c < dim; c += kThreads) {
      const float d = full(c);
      if (dh) sums[c] += to_f(dh[c]) * (to_f(xo[c]) - m2) * r2;
      if (f) {
        const float e = (to_f(f[c]) - m1) * r1, b = a.d.branch_scale * d, g = gate ? gate[c] : 1.f;
        sums[dim + c] += b * g * e;
        if (gate) dgate[c] += b * e * a.post_weight[c];
        static_cast<T*>(a.dbranch)[row * a.d.dbranch_stride + c] = from_f<T>(r1 * (b * g * a.post_weight[c] - mv - e * me));
      }
      static_cast<T*>(a.dx)[row * a.d.dx_stride + c] = from_f<T>(f ? a.d.residual_scale * d : d);
    }
  }
}

// Adds the blocks' sums in their order: block row y < 1 the weights, the others one gate each.
__global__ void __launch_bounds__(kThreads) norm_reduce_kernel(BlockNormArgs a, int blocks) {
  const int dim = (int)a.d.dim;
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= dim) return;
  const long long run = run_rows(a.d.rows, blocks);
  const long long stride = 4ll * dim;
  if (blockIdx.y == 0) {
    float s = 0.f, t = 0.f;
    for (int b = 0; b < blocks; ++b) {
      s += a.part[b * stride + c];
      t += a.part[b * stride + dim + c];
    }
    if (a.pre_weight) a.dpre_weight[c] = s;
    if (a.branch) a.dpost_weight[c] = t;
  }
  if (!a.gate) return;
  const long long groups = a.d.rows / a.d.gate_rows;
  for (long long g = blockIdx.y; g < groups; g += gridDim.y) {
    const long long b0 = g * a.d.gate_rows / run, b1 = ((g + 1) * a.d.gate_rows - 1) / run;
    if (b0 == b1) continue;
    float s = 0.f;
    for (long long b = b0; b <= b1; ++b) s += a.part[b * stride + (2 + (g != b * run / a.d.gate_rows)) * dim + c];
    a.dgate[g * dim + c] = s;
  }
}

template <typename T>
int backward(const BlockNormArgs& a, int num_sms, cudaStream_t st) {
  const int blocks = (int)std::min<long long>(a.d.rows, (long long)num_sms * kBlocksPerSm);
  norm_backward_kernel<T><<<blocks, kThreads, 0, st>>>(a);
  if (cudaGetLastError() != cudaSuccess) return CBR_ERR_CUDA;
  if (!a.branch && !a.pre_weight) return CBR_OK;
  const long long groups = a.gate ? a.d.rows / a.d.gate_rows : 1;
  const dim3 grid((unsigned)((a.d.dim + kThreads - 1) / kThreads), (unsigned)std::min<long long>(groups, 2 * blocks));
  norm_reduce_kernel<<<grid, kThreads, 0, st>>>(a, blocks);
  return cudaGetLastError() == cudaSuccess ? CBR_OK : CBR_ERR_CUDA;
}

}  // namespace

size_t block_norm_part_floats(const cbr_block_norm_desc_t& d) { return (size_t)kMaxCtas * kBlocksPerSm * 4 * d.dim; }

int launch_block_norm(const BlockNormArgs& a, int num_sms, cudaStream_t st) {
  const int grid = (int)std::min<long long>(a.d.rows, (long long)num_sms * 8);
  if (a.d.dtype == CBR_F32) norm_forward_kernel<float><<<grid, kThreads, 0, st>>>(a);
  else if (a.d.dtype == CBR_BF16) norm_forward_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a);
  else norm_forward_kernel<__half><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? CBR_OK : CBR_ERR_CUDA;
}

int launch_block_norm_backward(const BlockNormArgs& a, int num_sms, cudaStream_t st) {
  if (a.d.dtype == CBR_F32) return backward<float>(a, num_sms, st);
  if (a.d.dtype == CBR_BF16) return backward<__nv_bfloat16>(a, num_sms, st);
  return backward<__half>(a, num_sms, st);
}

}  // namespace cbr
