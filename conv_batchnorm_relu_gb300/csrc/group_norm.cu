// Group norm with an activation, channels last, forward and backward (declared in include/cbr.h): plain
// kernels, a block for each group of an image.
#include "common.cuh"
#include "token_ops.cuh"
#include "trunk_ops.h"

namespace cbr {
namespace {

using namespace tok;

constexpr int kThreads = 256;

__device__ float block_sum(float v) {
  __shared__ float part[kThreads / 32];
  v = warp_reduce<Sum>(v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  float s = 0.f;
  for (int i = 0; i < kThreads / 32; ++i) s += part[i];
  return s;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) forward_kernel(const GroupNormArgs a) {
  const cbr_group_norm_desc_t& d = a.d;
  const int per = d.channels / d.groups;
  const int64_t n = blockIdx.x / d.groups, c0 = blockIdx.x % d.groups * per, count = d.pixels * per;
  const T* x = static_cast<const T*>(a.x) + n * d.x_stride[0] + c0;
  T* y = static_cast<T*>(a.y) + n * d.y_stride[0] + c0;
  float s = 0.f;
  for (int64_t i = threadIdx.x; i < count; i += kThreads) s += to_f(x[i / per * d.x_stride[1] + i % per]);
  const float mean = block_sum(s) / (float)count;
  s = 0.f;
  for (int64_t i = threadIdx.x; i < count; i += kThreads) {
    const float v = to_f(x[i / per * d.x_stride[1] + i % per]) - mean;
    s = fmaf(v, v, s);
  }
  const float rstd = 1.f / sqrtf(block_sum(s) / (float)count + d.eps);
  for (int64_t i = threadIdx.x; i < count; i += kThreads) {
    const int64_t c = c0 + i % per;
    float z = (to_f(x[i / per * d.x_stride[1] + i % per]) - mean) * rstd;
    if (a.gamma) z = fmaf(z, a.gamma[c], a.beta[c]);
    if (d.act == CBR_ACT_RELU) z = z > 0.f ? z : 0.f * z;
    if (d.act == CBR_ACT_SILU) z = z / (1.f + expf(-z));
    y[i / per * d.y_stride[1] + i % per] = from_f<T>(z);
  }
  if (threadIdx.x == 0) a.mean[blockIdx.x] = mean, a.rstd[blockIdx.x] = rstd;
}

template <typename T>
__global__ void __launch_bounds__(kThreads) backward_kernel(const GroupNormArgs a) {
  const cbr_group_norm_desc_t& d = a.d;
  const int per = d.channels / d.groups;
  const int64_t n = blockIdx.x / d.groups, c0 = blockIdx.x % d.groups * per;
  const T* x = static_cast<const T*>(a.x) + n * d.x_stride[0] + c0;
  const T* dy = static_cast<const T*>(a.dy) + n * d.dy_stride[0] + c0;
  T* dx = static_cast<T*>(a.dx) + n * d.dx_stride[0] + c0;
  const float mean = a.mean[blockIdx.x], rstd = a.rstd[blockIdx.x];
  auto at = [&](int64_t p, int c, float& xh, float& g) {
    xh = (to_f(x[p * d.x_stride[1] + c]) - mean) * rstd;
    g = to_f(dy[p * d.dy_stride[1] + c]);
    const float z = a.gamma ? fmaf(xh, a.gamma[c0 + c], a.beta[c0 + c]) : xh;
    if (d.act == CBR_ACT_RELU) g = z > 0.f ? g : 0.f;
    if (d.act == CBR_ACT_SILU) {
      const float sig = 1.f / (1.f + expf(-z));
      g *= sig * (1.f + z * (1.f - sig));
    }
  };
  float u = 0.f, ux = 0.f;
  for (int c = 0; c < per; ++c) {
    float s = 0.f, sx = 0.f, xh, g;
    for (int64_t p = threadIdx.x; p < d.pixels; p += kThreads) {
      at(p, c, xh, g);
      s += g;
      sx = fmaf(g, xh, sx);
    }
    s = block_sum(s);
    sx = block_sum(sx);
    const float w = a.gamma ? a.gamma[c0 + c] : 1.f;
    u = fmaf(w, s, u);
    ux = fmaf(w, sx, ux);
    if (a.gamma && threadIdx.x == 0) {
      a.part[(2 * n) * d.channels + c0 + c] = sx;
      a.part[(2 * n + 1) * d.channels + c0 + c] = s;
    }
  }
  const float inv = 1.f / ((float)d.pixels * (float)per);
  for (int64_t i = threadIdx.x; i < d.pixels * per; i += kThreads) {
    const int c = (int)(i % per);
    float xh, g;
    at(i / per, c, xh, g);
    const float w = a.gamma ? a.gamma[c0 + c] : 1.f;
    dx[i / per * d.dx_stride[1] + c] = from_f<T>(rstd * (w * g - u * inv - xh * (ux * inv)));
  }
}

// dgamma and dbeta: the images' sums, in their order.
__global__ void __launch_bounds__(kThreads) reduce_kernel(const GroupNormArgs a) {
  const int c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= a.d.channels) return;
  float s[2] = {0.f, 0.f};
  for (int64_t n = 0; n < 2 * a.d.images; ++n) s[n & 1] += a.part[n * a.d.channels + c];
  a.dgamma[c] = s[0];
  a.dbeta[c] = s[1];
}

template <typename T>
void run(const GroupNormArgs& a, bool backward, cudaStream_t st) {
  const unsigned blocks = (unsigned)(a.d.images * a.d.groups);
  if (backward) backward_kernel<T><<<blocks, kThreads, 0, st>>>(a);
  else forward_kernel<T><<<blocks, kThreads, 0, st>>>(a);
}

int dispatch(const GroupNormArgs& a, bool backward, cudaStream_t st) {
  if (a.d.images > 0x7fffffff / a.d.groups) return CBR_ERR_UNSUPPORTED;
  if (a.d.dtype == CBR_F32) run<float>(a, backward, st);
  else if (a.d.dtype == CBR_BF16) run<__nv_bfloat16>(a, backward, st);
  else run<__half>(a, backward, st);
  if (backward && a.gamma) reduce_kernel<<<(a.d.channels + kThreads - 1) / kThreads, kThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? CBR_OK : CBR_ERR_CUDA;
}

}  // namespace

size_t group_norm_part_floats(const cbr_group_norm_desc_t& d) { return (size_t)d.images * 2 * d.channels; }
int launch_group_norm(const GroupNormArgs& a, cudaStream_t st) { return dispatch(a, false, st); }
int launch_group_norm_backward(const GroupNormArgs& a, cudaStream_t st) { return dispatch(a, true, st); }

}  // namespace cbr
