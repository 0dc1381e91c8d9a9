// The norm of a set of gradients and their clipping (declared in include/cbr.h).
//
// Two kernels: every block's part of the sum of squares, then (after it, on the stream) the scale from all
// parts and the scaled gradients.  The tensors' addresses travel in the launches' own parameters, kMost at
// a time, so a call keeps nothing on the device and can be captured.
#include <algorithm>

#include "common.cuh"
#include "token_ops.cuh"
#include "trunk_ops.h"

namespace cbr {
namespace {

using namespace tok;

constexpr int kThreads = 512;
constexpr int kBlocks = 304;       // parts of the sum for each launch
constexpr int kMost = 512;         // tensors in one launch's parameters
constexpr int kTile = 8192;        // elements that a block takes at a time
constexpr int kEpt = kTile / kThreads;

template <int N>
struct Table {
  const void* grad[N];
  void* out[N];
  int64_t size[N];
  int64_t tile[N + 1];   // the tensor's first tile
  uint8_t dtype[N];
  int count;
};

// A thread's sum of squares is taken over few elements in fp32 and added up in fp64, whose range no sum
// of squares of fp32 values leaves.  Where the fp32 sum is too large or too small to be exact it is taken
// again, of the elements times a power of two.
__device__ __forceinline__ double squares(const float (&v)[kEpt]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < kEpt; ++i) s = fmaf(v[i], v[i], s);
  if (s > 0x1p100f || s < 0x1p-80f) {
    const float f = s > 1.f ? 0x1p-100f : 0x1p100f;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < kEpt; ++i) s = fmaf(v[i] * f, v[i] * f, s);
    return (double)s * (f > 1.f ? 0x1p-200 : 0x1p200);
  }
  return s;
}

__device__ double block_sum(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
  for (int i = 0; i < kThreads / 32; ++i) v += part[i];
  return v;
}

template <int N>
__device__ __forceinline__ int tensor_of(const Table<N>& t, int64_t tile) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.tile[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <typename T>
__device__ __forceinline__ void load(float (&v)[kEpt], const void* p, int64_t at, int64_t size) {
#pragma unroll
  for (int i = 0; i < kEpt; ++i) {
    const int64_t e = at + i * kThreads + threadIdx.x;
    v[i] = e < size ? to_f(static_cast<const T*>(p)[e]) : 0.f;
  }
}

template <typename T>
__device__ __forceinline__ void store(const float (&v)[kEpt], float f, void* p, int64_t at, int64_t size) {
#pragma unroll
  for (int i = 0; i < kEpt; ++i) {
    const int64_t e = at + i * kThreads + threadIdx.x;
    if (e < size) static_cast<T*>(p)[e] = from_f<T>(v[i] * f);
  }
}

template <int N>
__device__ __forceinline__ void load_tile(float (&v)[kEpt], const Table<N>& t, int i, int64_t at) {
  if (t.dtype[i] == CBR_F32) load<float>(v, t.grad[i], at, t.size[i]);
  else if (t.dtype[i] == CBR_BF16) load<__nv_bfloat16>(v, t.grad[i], at, t.size[i]);
  else load<__half>(v, t.grad[i], at, t.size[i]);
}

template <int N>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ Table<N> t, double* part) {
  double sum = 0.0;
  for (int64_t tile = blockIdx.x; tile < t.tile[t.count]; tile += gridDim.x) {
    const int i = tensor_of(t, tile);
    float v[kEpt];
    load_tile(v, t, i, (tile - t.tile[i]) * kTile);
    sum += squares(v);
  }
  sum = block_sum(sum);
  if (threadIdx.x == 0) part[blockIdx.x] = sum;
}

// Every block adds the parts up in the same order; the first one of the call writes the norm and the scale.
__device__ float scale_of(const double* part, int parts, float max_norm, float unscale, float* norm_out, float* scale_out,
                          bool write) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += kThreads) s += part[i];
  s = block_sum(s);
  // the scale goes by the norm before it is rounded: one that is subnormal in fp32 has few digits, one past
  // its range none
  const double exact = sqrt(s) * (double)unscale;
  const float norm = (float)exact;
  const float scale = exact > max_norm    ? (float)((double)max_norm / exact * (double)unscale)
                      : exact <= max_norm ? unscale
                                          : norm;
  if (write && threadIdx.x == 0) *norm_out = norm, *scale_out = scale;
  return scale;
}

template <int N>
__global__ void __launch_bounds__(kThreads)
    scale_kernel(const __grid_constant__ Table<N> t, const double* part, int parts, float max_norm, float unscale,
                 float* norm_out, float* scale_out, int first) {
  const float f = scale_of(part, parts, max_norm, unscale, norm_out, scale_out, first && blockIdx.x == 0);
  for (int64_t tile = blockIdx.x; tile < t.tile[t.count]; tile += gridDim.x) {
    const int i = tensor_of(t, tile);
    if (f == 1.f && t.out[i] == t.grad[i]) continue;
    const int64_t at = (tile - t.tile[i]) * kTile;
    float v[kEpt];
    load_tile(v, t, i, at);
    if (t.dtype[i] == CBR_F32) store<float>(v, f, t.out[i], at, t.size[i]);
    else if (t.dtype[i] == CBR_BF16) store<__nv_bfloat16>(v, f, t.out[i], at, t.size[i]);
    else store<__half>(v, f, t.out[i], at, t.size[i]);
  }
}

template <int N>
Table<N> table(const ClipArgs& a, int64_t first) {
  Table<N> t;
  t.count = (int)std::min<int64_t>(N, a.count - first);
  int64_t tile = 0;
  for (int i = 0; i < t.count; ++i) {
    t.grad[i] = a.grads[first + i];
    t.out[i] = a.outs ? a.outs[first + i] : nullptr;
    t.size[i] = a.sizes[first + i];
    t.dtype[i] = (uint8_t)a.dtypes[first + i];
    t.tile[i] = tile;
    tile += (t.size[i] + kTile - 1) / kTile;
  }
  t.tile[t.count] = tile;
  return t;
}

int64_t launches(int64_t count) { return std::max<int64_t>(1, (count + kMost - 1) / kMost); }

}  // namespace

size_t clip_part_doubles(int64_t count) { return (size_t)launches(count) * kBlocks; }

int launch_clip(const ClipArgs& a, cudaStream_t st) {
  const int64_t n = launches(a.count);
  const int parts = (int)(n * kBlocks);
  for (int64_t l = 0; l < n; ++l)
    norm_kernel<kMost><<<kBlocks, kThreads, 0, st>>>(table<kMost>(a, l * kMost), a.part + l * kBlocks);
  for (int64_t l = 0; l < (a.outs ? n : 1); ++l) {
    Table<kMost> t = table<kMost>(a, l * kMost);
    if (!a.outs) t.tile[t.count] = 0;
    scale_kernel<kMost><<<kBlocks, kThreads, 0, st>>>(t, a.part, parts, a.max_norm, a.unscale, a.norm, a.scale, l == 0);
  }
  return cudaGetLastError() == cudaSuccess ? CBR_OK : CBR_ERR_CUDA;
}

}  // namespace cbr
