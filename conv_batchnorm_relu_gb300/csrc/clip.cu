// The norm of a set of gradients and their clipping (declared in include/cbr.h).
//
// Bound by memory: every gradient is read for the norm, and read and written for the result, as far as L2 does not
// hold it (400 fp32 tensors of 1.6 GB: 750 us, 6.4 TB/s, 94% of the copy rate).  Two kernels: every block's part of the
// sum of squares, then (after it, on the stream) the scale from all parts and the scaled gradients, from the last
// tensors to the first, whose ends are still in L2.  The tensors' addresses travel in the launches' own parameters, so a
// call keeps nothing on the device and can be captured.
//   A tile is 32 KB that start on a 16-byte boundary at or before the tensor's first element; a thread loads its next
// tile's vectors before it works on the last ones.
#include <algorithm>

#include "common.cuh"
#include "follow.cuh"
#include "token_ops.cuh"
#include "trunk_ops.h"

namespace cbr {
namespace {

using namespace tok;

constexpr int kThreads = 512;
constexpr int kBlocks = 304;              // two to an SM: parts of the sum for each launch
constexpr int kMost = 512, kFew = 64;     // tensors in one launch's parameters (14 and 2 KB)
constexpr int kVectors = 4;               // 16-byte vectors of a thread in a tile
constexpr int kTileBytes = kThreads * kVectors * 16;

template <int N>
struct Table {
  const void* grad[N];
  void* out[N];
  int64_t size[N];
  uint32_t tile[N + 1];   // the tensor's first tile
  uint8_t dtype[N];
  int32_t count;
};

// A thread's sum of squares is taken over one vector's values in each of four places in fp32 and added up in fp64, whose
// range no sum of squares of fp32 values leaves.  Where the fp32 sum is too large or too small to be exact it is taken
// again, of the values times a power of two.
template <int n>
__device__ __forceinline__ double squares(const float (&v)[n]) {
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < n; ++i) s = fmaf(v[i], v[i], s);
  if (s > 0x1p100f || s < 0x1p-80f) {
    const float f = s > 1.f ? 0x1p-100f : 0x1p100f;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < n; ++i) s = fmaf(v[i] * f, v[i] * f, s);
    return (double)s * (f > 1.f ? 0x1p-200 : 0x1p200);
  }
  return s;
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Where a tile lies: its tensor, and the index (from the 16-byte boundary on) of its first element.
struct Spot {
  int tensor;
  int64_t first;
};

template <int N>
__device__ __forceinline__ Spot spot_of(const Table<N>& t, uint32_t tile) {
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.tile[mid] <= tile) lo = mid;
    else hi = mid - 1;
  }
  const int elements = kTileBytes / (t.dtype[lo] == CBR_F32 ? 4 : 2);
  return Spot{lo, (int64_t)(tile - t.tile[lo]) * elements};
}

// A thread's vectors of a tile as they are stored; what is not of the tensor is 0.
struct Raw {
  uint4 v[kVectors];

  // The vector at index e, counted from the 16-byte boundary `skip` elements before the tensor.
  template <typename T>
  static __device__ __forceinline__ uint4 vector(const T* base, int skip, int64_t size, int64_t e) {
    constexpr int kPer = 16 / sizeof(T);
    uint4 v = make_uint4(0, 0, 0, 0);
    if (e >= skip && e + kPer <= skip + size) {
      asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "l"(base + e));
    } else if (e + kPer > skip && e < skip + size) {
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int k = 0; k < kPer; ++k) {
        if (e + k < skip || e + k >= skip + size) continue;
        if constexpr (sizeof(T) == 4) w[k] = *reinterpret_cast<const uint32_t*>(base + e + k);
        else w[k / 2] |= (uint32_t)*reinterpret_cast<const uint16_t*>(base + e + k) << (16 * (k & 1));
      }
      v = make_uint4(w[0], w[1], w[2], w[3]);
    }
    return v;
  }
  template <typename T>
  __device__ __forceinline__ void load(const void* grad, int64_t size, int64_t first) {
    const int skip = (int)(reinterpret_cast<uintptr_t>(grad) & 15) / (int)sizeof(T);
    const T* base = static_cast<const T*>(grad) - skip;
#pragma unroll
    for (int i = 0; i < kVectors; ++i) v[i] = vector<T>(base, skip, size, first + ((int64_t)i * kThreads + threadIdx.x) * (16 / sizeof(T)));
  }
  template <int N>
  __device__ __forceinline__ void load(const Table<N>& t, const Spot& s) {
    if (t.dtype[s.tensor] == CBR_F32) load<float>(t.grad[s.tensor], t.size[s.tensor], s.first);
    else load<__half>(t.grad[s.tensor], t.size[s.tensor], s.first);   // (16 bits of either type)
  }
  template <typename T>
  static __device__ __forceinline__ void values(const uint4& u, float (&f)[16 / sizeof(T)]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if constexpr (sizeof(T) == 4) {
        f[k] = __uint_as_float(w[k]);
      } else {
        const float2 p = unpack2<std::is_same_v<T, __nv_bfloat16>>(w[k]);
        f[2 * k] = p.x, f[2 * k + 1] = p.y;
      }
    }
  }
  template <typename T>
  __device__ __forceinline__ double sum() const {
    double s = 0.0;
    if constexpr (sizeof(T) == 4) {   // four vectors' 16 values at once
      float f[4 * kVectors];
#pragma unroll
      for (int i = 0; i < kVectors; ++i) values<T>(v[i], *reinterpret_cast<float(*)[4]>(f + 4 * i));
      s = squares(f);
    } else {
#pragma unroll
      for (int i = 0; i < kVectors; i += 2) {
        float f[16];
        values<T>(v[i], *reinterpret_cast<float(*)[8]>(f));
        values<T>(v[i + 1], *reinterpret_cast<float(*)[8]>(f + 8));
        s += squares(f);
      }
    }
    return s;
  }
  template <typename T>
  static __device__ __forceinline__ uint4 scaled(const uint4& u, float scale) {
    float f[16 / sizeof(T)];
    values<T>(u, f);
#pragma unroll
    for (int k = 0; k < 16 / (int)sizeof(T); ++k) f[k] *= scale;
    if constexpr (sizeof(T) == 4) {
      return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
    } else {
      constexpr bool kBf16 = std::is_same_v<T, __nv_bfloat16>;
      return make_uint4(pack2<kBf16>(f[0], f[1]), pack2<kBf16>(f[2], f[3]), pack2<kBf16>(f[4], f[5]), pack2<kBf16>(f[6], f[7]));
    }
  }
  // 16 bytes to the tensor's elements from e on, one by one those that it has.
  template <typename T>
  static __device__ __forceinline__ void put(T* base, int skip, int64_t size, int64_t e, const uint4& u, int count = 16 / sizeof(T)) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 16 / (int)sizeof(T); ++k) {
      if (k >= count || e + k < skip || e + k >= skip + size) continue;
      if constexpr (sizeof(T) == 4) reinterpret_cast<uint32_t*>(base)[e + k] = w[k];
      else reinterpret_cast<uint16_t*>(base)[e + k] = (uint16_t)(w[k / 2] >> (16 * (k & 1)));
    }
  }
  // The scaled values to `out`.  Where its 16-byte boundaries are others than the gradient's, a thread's store is the end
  // of its vector and the beginning of the next one's, which the next lane has (the last lane's is loaded again).
  template <typename T>
  __device__ __forceinline__ void store(float scale, const void* grad, void* out, int64_t size, int64_t first) const {
    constexpr int kPer = 16 / sizeof(T);
    const int skip = (int)(reinterpret_cast<uintptr_t>(grad) & 15) / (int)sizeof(T);
    const T* source = static_cast<const T*>(grad) - skip;
    T* base = static_cast<T*>(out) - skip;
    const int off = (int)(reinterpret_cast<uintptr_t>(base) & 15);   // bytes
    const int later = (16 - off) / (int)sizeof(T);                   // elements to the next boundary
#pragma unroll
    for (int i = 0; i < kVectors; ++i) {
      const int64_t e = first + ((int64_t)i * kThreads + threadIdx.x) * kPer;
      const uint4 u = scaled<T>(v[i], scale);
      if (off == 0) {
        if (e >= skip && e + kPer <= skip + size) st_global_v4(base + e, u);
        else put<T>(base, skip, size, e, u);
        continue;
      }
      uint4 n;
      n.x = __shfl_down_sync(0xffffffffu, u.x, 1);
      n.y = __shfl_down_sync(0xffffffffu, u.y, 1);
      n.z = __shfl_down_sync(0xffffffffu, u.z, 1);
      n.w = __shfl_down_sync(0xffffffffu, u.w, 1);
      if ((threadIdx.x & 31) == 31) n = scaled<T>(vector<T>(source, skip, size, e + kPer), scale);
      // bytes [16 - off, 32 - off) of (u, n): whole words, then the rest of a word
      uint32_t w[8] = {u.x, u.y, u.z, u.w, n.x, n.y, n.z, n.w};
      const int words = (16 - off) >> 2, rest = ((16 - off) & 3) * 8;
      if (words & 1)
#pragma unroll
        for (int k = 0; k < 7; ++k) w[k] = w[k + 1];
      if (words & 2)
#pragma unroll
        for (int k = 0; k < 6; ++k) w[k] = w[k + 2];
      const uint4 s = make_uint4(__funnelshift_r(w[0], w[1], rest), __funnelshift_r(w[1], w[2], rest), __funnelshift_r(w[2], w[3], rest),
                                 __funnelshift_r(w[3], w[4], rest));
      if (e == 0) put<T>(base, skip, size, 0, u, later);   // what lies before the first boundary
      if (e + later >= skip && e + later + kPer <= skip + size) st_global_v4(base + e + later, s);
      else put<T>(base, skip, size, e + later, s);
    }
  }
};

template <int N>
__global__ void __launch_bounds__(kThreads, 2) norm_kernel(const __grid_constant__ Table<N> t, double* part) {
  __shared__ double sums[kThreads / 32];
  const uint32_t tiles = t.tile[t.count];
  let_next_kernel_start();
  double sum = 0.0;
  Raw next;
  Spot at{}, after{};
  if (blockIdx.x < tiles) {
    after = spot_of(t, blockIdx.x);
    next.load(t, after);
  }
  for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const Raw raw = next;
    at = after;
    if (tile + gridDim.x < tiles) {
      after = spot_of(t, tile + gridDim.x);
      next.load(t, after);
    }
    const int type = t.dtype[at.tensor];
    sum += type == CBR_F32 ? raw.sum<float>() : type == CBR_BF16 ? raw.sum<__nv_bfloat16>() : raw.sum<__half>();
  }
  sum = warp_sum(sum);
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = sum;
  __syncthreads();
  if (threadIdx.x < 32) {
    sum = warp_sum(threadIdx.x < kThreads / 32 ? sums[threadIdx.x] : 0.0);
    if (threadIdx.x == 0) part[blockIdx.x] = sum;
  }
}

// Every block of the first launch adds the parts up in the same order, in one warp, and its first block writes norm and scale,
// which the launches behind it read (65536 tensors, 128 launches of each kernel: 1.6 ms; 8.0 where all added the parts up).
// The scale goes by the norm before it is rounded: one that is subnormal in fp32 has few digits, one past its range none.
__device__ __forceinline__ float scale_of(const double* part, int parts, float max_norm, float unscale, float* norm_out, float* scale_out,
                                          bool write) {
  double s = 0.0;
  for (int i = threadIdx.x; i < parts; i += 32) s += part[i];
  s = warp_sum(s);
  const double exact = sqrt(s) * (double)unscale;
  const float norm = (float)exact;
  const float scale = exact > max_norm    ? (float)((double)max_norm / exact * (double)unscale)
                      : exact <= max_norm ? unscale
                                          : norm;
  if (write && threadIdx.x == 0) *norm_out = norm, *scale_out = scale;
  return scale;
}

template <int N>
__global__ void __launch_bounds__(kThreads, 2)
    scale_kernel(const __grid_constant__ Table<N> t, const double* part, int parts, float max_norm, float unscale,
                 float* norm_out, float* scale_out, int first) {
  __shared__ float shared_scale;
  const uint32_t tiles = t.tile[t.count];
  Raw next;
  Spot at{}, after{};
  if (blockIdx.x < tiles) {
    after = spot_of(t, tiles - 1 - blockIdx.x);
    next.load(t, after);
  }
  wait_for_kernel_ahead();   // (gradients are only read up to here)
  if (threadIdx.x < 32) {
    const float f = first ? scale_of(part, parts, max_norm, unscale, norm_out, scale_out, blockIdx.x == 0) : *scale_out;
    if (threadIdx.x == 0) shared_scale = f;
  }
  __syncthreads();
  const float f = shared_scale;
  for (uint32_t tile = blockIdx.x; tile < tiles; tile += gridDim.x) {
    const Raw raw = next;
    at = after;
    if (tile + gridDim.x < tiles) {
      after = spot_of(t, tiles - 1 - tile - gridDim.x);
      if (!(f == 1.f && t.out[after.tensor] == t.grad[after.tensor])) next.load(t, after);
    }
    const int i = at.tensor, type = t.dtype[i];
    if (f == 1.f && t.out[i] == t.grad[i]) continue;
    if (type == CBR_F32) raw.store<float>(f, t.grad[i], t.out[i], t.size[i], at.first);
    else if (type == CBR_BF16) raw.store<__nv_bfloat16>(f, t.grad[i], t.out[i], t.size[i], at.first);
    else raw.store<__half>(f, t.grad[i], t.out[i], t.size[i], at.first);
  }
}

// The tensors from `first` on; false where they are more than 2^32 tiles.
template <int N>
bool table(const ClipArgs& a, int64_t first, Table<N>& t) {
  t.count = (int)std::min<int64_t>(N, a.count - first);
  int64_t tile = 0;
  for (int i = 0; i < t.count; ++i) {
    const int64_t n = a.sizes[first + i], elt = a.dtypes[first + i] == CBR_F32 ? 4 : 2;
    t.grad[i] = a.grads[first + i];
    t.out[i] = a.outs ? a.outs[first + i] : nullptr;
    t.size[i] = n;
    t.dtype[i] = (uint8_t)a.dtypes[first + i];
    t.tile[i] = (uint32_t)tile;
    const int64_t skip = static_cast<int64_t>(reinterpret_cast<uintptr_t>(t.grad[i]) & 15);
    tile += n ? (n * elt + skip + kTileBytes - 1) / kTileBytes : 0;
    if (tile >= (int64_t(1) << 32) - kBlocks) return false;
  }
  t.tile[t.count] = (uint32_t)tile;
  return true;
}

int64_t launches(int64_t count) { return std::max<int64_t>(1, (count + kMost - 1) / kMost); }

template <int N>
int launch(const ClipArgs& a, cudaStream_t st) {
  const int64_t n = launches(a.count);
  const int parts = (int)(n * kBlocks);
  Table<N> t;
  for (int64_t l = 0; l < n; ++l)
    if (!table<N>(a, l * N, t)) return CBR_ERR_UNSUPPORTED;
  for (int64_t l = 0; l < n; ++l) {
    if (n > 1) table<N>(a, l * N, t);
    norm_kernel<N><<<kBlocks, kThreads, 0, st>>>(t, a.part + l * kBlocks);
  }
  for (int64_t l = a.outs ? n - 1 : 0; l >= 0; --l) {
    if (n > 1) table<N>(a, l * N, t);
    if (!a.outs) t.tile[t.count] = 0;
    if (l == n - 1 || !a.outs) {
      if (!launch_behind(&scale_kernel<N>, dim3(a.outs ? kBlocks : 1), kThreads, 0, st, t, a.part, parts, a.max_norm, a.unscale, a.norm, a.scale, 1))
        return CBR_ERR_CUDA;
    } else {
      scale_kernel<N><<<kBlocks, kThreads, 0, st>>>(t, a.part, parts, a.max_norm, a.unscale, a.norm, a.scale, 0);
    }
  }
  return cudaGetLastError() == cudaSuccess ? CBR_OK : CBR_ERR_CUDA;
}

}  // namespace

size_t clip_part_doubles(int64_t count) { return (size_t)launches(count) * kBlocks; }

int launch_clip(const ClipArgs& a, cudaStream_t st) { return a.count <= kFew ? launch<kFew>(a, st) : launch<kMost>(a, st); }

}  // namespace cbr
