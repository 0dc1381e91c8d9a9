// Group norm with an activation, channels last, forward and backward (declared in include/cbr.h).
//
// Bound by memory: x is read once and y written once where that can be.  A cluster of up to 16 blocks takes an
// image, each block a run of its pixels: the block reads its run (16-byte vectors, a thread keeps its channels),
// keeps it in shared memory and takes each channel's moments; the blocks exchange their groups' moments
// through distributed shared memory; then each normalises what it holds and writes it.  Of an image that is
// more than a cluster holds the rest is read again, mostly from L2.  The backward does the same with x and dy, and
// the sums of g and g xh.  Where a few images are larger than that, clusters would leave most SMs idle: the
// moments (sums) and the result are launches of their own, over runs of pixels on every SM.
//   Moments: a thread sums its values' differences from its first one, and their squares, which costs no digits
// where the mean is far from 0; means and squared deviations are merged by their counts.  All merges have a fixed
// order.
#include <cooperative_groups.h>

#include <algorithm>
#include <mutex>
#include <set>
#include <utility>

#include "cbr_internal.h"
#include "common.cuh"
#include "token_ops.cuh"
#include "trunk_ops.h"

namespace cbr {
namespace gn {
namespace {

using namespace tok;

constexpr int kThreads = 256, kWarps = kThreads / 32, kMaxCluster = 16;
constexpr int64_t kSms = 152;   // of the device that the rules on blocks are made for

struct Params {
  const void* x;
  const void* dy;
  void* y;               // forward y, backward dx
  const float* gamma;    // null: ones (and beta zeros)
  const float* beta;
  float* mean;           // [images][groups]
  float* rstd;
  float* part;           // moments or sums of runs (see the launchers)
  float* group_part;
  int64_t x_stride[2], dy_stride[2], y_stride[2];
  int64_t pixels;
  int64_t base;          // pixels of a run; the first `extra` runs have one more
  int extra;
  int channels, groups, per, act;   // per: channels of a group
  int keep;              // pixels of a run that stay in shared memory
  int runs;              // of an image, one to a block
  float eps;
};

// kVec neighbouring channels of a pixel, as they are stored.
template <typename T, int kVec>
struct Vec {
  static constexpr int kBytes = kVec * (int)sizeof(T);
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes == 16)
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
    else if constexpr (kBytes == 8)
      asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    else if constexpr (kBytes == 4)
      asm volatile("ld.global.b32 %0, [%1];" : "=r"(w[0]) : "l"(p));
    else
      asm volatile("ld.global.u16 %0, [%1];" : "=r"(w[0]) : "l"(p));
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes == 16) st_global_v4(p, make_uint4(w[0], w[1], w[2], w[3]));
    else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
  }
  // to and from shared memory, `i` vectors from its start
  __device__ __forceinline__ void put(uint8_t* s, int i) const {
    uint8_t* p = s + (size_t)i * kBytes;
    if constexpr (kBytes == 16) *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
    else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
  }
  __device__ __forceinline__ void take(const uint8_t* s, int i) {
    const uint8_t* p = s + (size_t)i * kBytes;
    if constexpr (kBytes == 16) {
      const uint4 v = *reinterpret_cast<const uint4*>(p);
      w[0] = v.x, w[1] = v.y, w[2] = v.z, w[3] = v.w;
    } else if constexpr (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x, w[1] = v.y;
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    }
  }
  __device__ __forceinline__ void get(float (&v)[kVec]) const {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) v[i] = __uint_as_float(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; i += 2) {
        const float2 f = unpack2<std::is_same_v<T, __nv_bfloat16>>(w[i / 2]);
        v[i] = f.x;
        if constexpr (kVec > 1) v[i + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ void set(const float (&v)[kVec]) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < kVec; ++i) w[i] = __float_as_uint(v[i]);
    } else if constexpr (kVec == 1) {
      w[0] = pack2<std::is_same_v<T, __nv_bfloat16>>(v[0], 0.f);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; i += 2) w[i / 2] = pack2<std::is_same_v<T, __nv_bfloat16>>(v[i], v[i + 1]);
    }
  }
};

// How a block's threads lie over its run: a thread has a column (kVec channels) and every `rows`th pixel.
struct Lay {
  int columns;   // vectors of a pixel
  int across;    // of them at a time: the threads of a row
  int rows;      // rows of threads; threads behind the last have nothing to do
  template <int kVec>
  static __device__ __forceinline__ Lay of(int channels) {
    Lay l;
    l.columns = channels / kVec;
    l.across = min(l.columns, kThreads);
    l.rows = kThreads / l.across;
    return l;
  }
};

// The pixels of run `r` of an image.
__device__ __forceinline__ int64_t run_begin(const Params& a, int r) { return a.base * r + min(r, a.extra); }
__device__ __forceinline__ int run_length(const Params& a, int r) { return (int)a.base + (r < a.extra); }
// Of `n` pixels, those of row `row` of `rows`.
__device__ __forceinline__ int turns(int n, int row, int rows) { return row < n ? (n - row + rows - 1) / rows : 0; }

__device__ __forceinline__ float act_of(float z, int act) {
  if (act == CBR_ACT_RELU) return Max::of(z, 0.f);
  if (act == CBR_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
  return z;
}
__device__ __forceinline__ float act_slope(float z, float up, int act) {
  if (act == CBR_ACT_RELU) return z > 0.f ? up : 0.f;
  if (act == CBR_ACT_SILU) {
    const float s = __fdividef(1.f, 1.f + __expf(-z));
    return up * (s * fmaf(z, 1.f - s, 1.f));
  }
  return up;
}

// What a channel is normalised with: z = (x - mean) scale + shift.
template <int kVec>
struct Channel {
  float mean[kVec], scale[kVec], shift[kVec], rstd[kVec];
  __device__ __forceinline__ void of(const Params& a, int c, const float* mean_of, const float* rstd_of) {
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int g = (c + i) / a.per;
      mean[i] = mean_of[g];
      rstd[i] = rstd_of[g];
      scale[i] = a.gamma ? rstd[i] * a.gamma[c + i] : rstd[i];
      shift[i] = a.gamma ? a.beta[c + i] : 0.f;
    }
  }
};

constexpr int kBatch = 4;   // a thread's loads in flight for each operand

// Shared memory: two values of each channel for each row of threads, two of each group twice, the kept pixels.
template <int kVec>
__host__ __device__ constexpr int table_floats(int channels) {
  return channels > kThreads * kVec ? channels : kThreads * kVec;
}

// ---------------------------------------------------------------- forward

// A run's moments: `table` gets (mean, squared deviations) of every channel in every row of threads; `kept` the
// first pixels.
template <typename T, int kVec>
__device__ __forceinline__ void moments(const Params& a, const T* x, int n, float* table, uint8_t* kept) {
  const Lay l = Lay::of<kVec>(a.channels);
  const int row = threadIdx.x / l.across, size = table_floats<kVec>(a.channels);
  if (row >= l.rows) return;
  for (int col = threadIdx.x % l.across; col < l.columns; col += l.across) {
    const T* p = x + (int64_t)col * kVec;
    float first[kVec], s[kVec], q[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) first[i] = s[i] = q[i] = 0.f;
    for (int at = row; at < n; at += l.rows * kBatch) {
      Vec<T, kVec> v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (at + b * l.rows < n) v[b].load(p + (at + b * l.rows) * a.x_stride[1]);
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int pixel = at + b * l.rows;
        if (pixel >= n) continue;
        if (pixel < a.keep) v[b].put(kept, pixel * l.columns + col);
        float f[kVec];
        v[b].get(f);
        if (pixel == row)
#pragma unroll
          for (int i = 0; i < kVec; ++i) first[i] = f[i];
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float d = f[i] - first[i];
          s[i] += d;
          q[i] = fmaf(d, d, q[i]);
        }
      }
    }
    const int count = turns(n, row, l.rows);
    if (count == 0) continue;
    const float inv = 1.f / (float)count;
    float* m = table + row * a.channels + col * kVec;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const float shift = s[i] * inv;
      m[i] = first[i] + shift;
      m[size + i] = q[i] - s[i] * shift;
    }
  }
}

// The groups' moments of a run from its channels': a warp for each group.
template <int kVec>
__device__ __forceinline__ void group_moments(const Params& a, int n, const float* table, float2* groups) {
  const Lay l = Lay::of<kVec>(a.channels);
  const int size = table_floats<kVec>(a.channels), lane = threadIdx.x & 31;
  for (int g = threadIdx.x >> 5; g < a.groups; g += kWarps) {
    const float* m = table + g * a.per;
    const float ref = n ? m[0] : 0.f;
    float s = 0.f, q = 0.f;
    for (int e = lane; e < l.rows * a.per; e += 32) {
      const int row = e / a.per, at = row * a.channels + e % a.per, count = turns(n, row, l.rows);
      if (count) s = fmaf((float)count, m[at] - ref, s);
    }
    const float mean = n ? ref + warp_reduce<Sum>(s) / ((float)n * (float)a.per) : 0.f;
    for (int e = lane; e < l.rows * a.per; e += 32) {
      const int row = e / a.per, at = row * a.channels + e % a.per, count = turns(n, row, l.rows);
      if (count) q += fmaf((float)count * (m[at] - mean), m[at] - mean, m[size + at]);
    }
    q = warp_reduce<Sum>(q);
    if (lane == 0) groups[g] = make_float2(mean, q);
  }
}

__device__ __forceinline__ float rstd_of(float squares, float n, float eps) { return 1.f / sqrtf(fmaxf(squares, 0.f) / n + eps); }

// A run normalised: the kept pixels from shared memory, the others read again.
template <typename T, int kVec>
__device__ __forceinline__ void normalise(const Params& a, const T* x, T* y, int n, const float* mean, const float* rstd, const uint8_t* kept) {
  const Lay l = Lay::of<kVec>(a.channels);
  const int row = threadIdx.x / l.across;
  if (row >= l.rows) return;
  for (int col = threadIdx.x % l.across; col < l.columns; col += l.across) {
    Channel<kVec> c;
    c.of(a, col * kVec, mean, rstd);
    for (int at = row; at < n; at += l.rows * kBatch) {
      Vec<T, kVec> v[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int pixel = at + b * l.rows;
        if (pixel < a.keep && pixel < n) v[b].take(kept, pixel * l.columns + col);
        else if (pixel < n) v[b].load(x + pixel * a.x_stride[1] + (int64_t)col * kVec);
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int pixel = at + b * l.rows;
        if (pixel >= n) continue;
        float f[kVec];
        v[b].get(f);
#pragma unroll
        for (int i = 0; i < kVec; ++i) f[i] = act_of(fmaf(f[i] - c.mean[i], c.scale[i], c.shift[i]), a.act);
        v[b].set(f);
        v[b].store(y + pixel * a.y_stride[1] + (int64_t)col * kVec);
      }
    }
  }
}

template <typename T, int kVec>
struct Shared {
  float* table;
  float2* groups;
  float* stat;     // mean, then rstd; backward: the two means of a group
  uint8_t* kept;
  __device__ __forceinline__ Shared(const Params& a, uint8_t* smem) {
    table = reinterpret_cast<float*>(smem);
    groups = reinterpret_cast<float2*>(table + 2 * table_floats<kVec>(a.channels));
    stat = reinterpret_cast<float*>(groups + a.groups);
    kept = smem + ((8 * table_floats<kVec>(a.channels) + 16 * a.groups + 15) & ~15);
  }
};

template <typename T, int kVec>
__global__ void __launch_bounds__(kThreads, 2) cluster_forward_kernel(const __grid_constant__ Params a) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint8_t smem[];
  const Shared<T, kVec> s(a, smem);
  const cg::cluster_group cluster = cg::this_cluster();
  const int run = (int)cluster.block_rank();
  const int64_t image = blockIdx.x / a.runs;
  const int n = run_length(a, run);
  const T* x = static_cast<const T*>(a.x) + image * a.x_stride[0] + run_begin(a, run) * a.x_stride[1];
  moments<T, kVec>(a, x, n, s.table, s.kept);
  __syncthreads();
  group_moments<kVec>(a, n, s.table, s.groups);
  cluster.sync();
  const float total = (float)a.pixels * (float)a.per;
  for (int g = threadIdx.x; g < a.groups; g += kThreads) {
    float2 m[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < a.runs) m[r] = cluster.map_shared_rank(s.groups, r)[g];
    // relative to the first run's, which is never empty
    const float ref = m[0].x;
    float sum = 0.f, q = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < a.runs && run_length(a, r)) sum = fmaf((float)run_length(a, r) * (float)a.per, m[r].x - ref, sum);
    const float mean = ref + sum / total;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < a.runs && run_length(a, r)) q += fmaf((float)run_length(a, r) * (float)a.per * (m[r].x - mean), m[r].x - mean, m[r].y);
    const float rstd = rstd_of(q, total, a.eps);
    s.stat[g] = mean;
    s.stat[a.groups + g] = rstd;
    if (run == 0) a.mean[image * a.groups + g] = mean, a.rstd[image * a.groups + g] = rstd;
  }
  __syncthreads();
  cluster.barrier_arrive();   // the other blocks' moments are not read any more
  normalise<T, kVec>(a, x, static_cast<T*>(a.y) + image * a.y_stride[0] + run_begin(a, run) * a.y_stride[1], n, s.stat, s.stat + a.groups, s.kept);
  cluster.barrier_wait();
}

// Few large images: every run's moments, [image][run][group], then the images', then the result.
template <typename T, int kVec>
__global__ void __launch_bounds__(kThreads, 2) moments_kernel(const __grid_constant__ Params a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const Shared<T, kVec> s(a, smem);
  const int run = blockIdx.x % a.runs;
  const int64_t image = blockIdx.x / a.runs;
  const int n = run_length(a, run);
  moments<T, kVec>(a, static_cast<const T*>(a.x) + image * a.x_stride[0] + run_begin(a, run) * a.x_stride[1], n, s.table, s.kept);
  __syncthreads();
  group_moments<kVec>(a, n, s.table, reinterpret_cast<float2*>(a.group_part) + (int64_t)blockIdx.x * a.groups);
}

// A warp for each group of an image.
__global__ void __launch_bounds__(128) merge_moments_kernel(const __grid_constant__ Params a, int64_t images) {
  const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (at >= images * a.groups) return;
  const float2* m = reinterpret_cast<const float2*>(a.group_part) + at / a.groups * a.runs * a.groups + at % a.groups;
  const float ref = m[0].x, total = (float)a.pixels * (float)a.per;
  float sum = 0.f, q = 0.f;
  for (int r = lane; r < a.runs; r += 32) sum = fmaf((float)run_length(a, r) * (float)a.per, m[(int64_t)r * a.groups].x - ref, sum);
  const float mean = ref + warp_reduce<Sum>(sum) / total;
  for (int r = lane; r < a.runs; r += 32) {
    const float2 v = m[(int64_t)r * a.groups];
    q += fmaf((float)run_length(a, r) * (float)a.per * (v.x - mean), v.x - mean, v.y);
  }
  q = warp_reduce<Sum>(q);
  if (lane == 0) a.mean[at] = mean, a.rstd[at] = rstd_of(q, total, a.eps);
}

// Runs in the opposite order to the moments', whose last ones are still in L2.
template <typename T, int kVec>
__global__ void __launch_bounds__(kThreads, 2) normalise_kernel(const __grid_constant__ Params a) {
  const int block = gridDim.x - 1 - blockIdx.x, run = block % a.runs;
  const int64_t image = block / a.runs;
  normalise<T, kVec>(a, static_cast<const T*>(a.x) + image * a.x_stride[0] + run_begin(a, run) * a.x_stride[1],
                     static_cast<T*>(a.y) + image * a.y_stride[0] + run_begin(a, run) * a.y_stride[1], run_length(a, run), a.mean + image * a.groups,
                     a.rstd + image * a.groups, nullptr);
}

// ---------------------------------------------------------------- backward

// A run's sums of g and g xh: `table` gets them of every channel in every row of threads.
template <typename T, int kVec>
__device__ __forceinline__ void sums(const Params& a, int64_t image, const T* x, const T* dy, int n, float* table, uint8_t* kept) {
  const Lay l = Lay::of<kVec>(a.channels);
  const int row = threadIdx.x / l.across, size = table_floats<kVec>(a.channels);
  if (row >= l.rows) return;
  uint8_t* kept_dy = kept + (size_t)a.keep * a.channels * sizeof(T);
  for (int col = threadIdx.x % l.across; col < l.columns; col += l.across) {
    Channel<kVec> c;
    c.of(a, col * kVec, a.mean + image * a.groups, a.rstd + image * a.groups);
    float s[kVec], sx[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) s[i] = sx[i] = 0.f;
    for (int at = row; at < n; at += l.rows * kBatch) {
      Vec<T, kVec> v[kBatch], u[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (at + b * l.rows < n) {
          v[b].load(x + (at + b * l.rows) * a.x_stride[1] + (int64_t)col * kVec);
          u[b].load(dy + (at + b * l.rows) * a.dy_stride[1] + (int64_t)col * kVec);
        }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int pixel = at + b * l.rows;
        if (pixel >= n) continue;
        if (pixel < a.keep) {
          v[b].put(kept, pixel * l.columns + col);
          u[b].put(kept_dy, pixel * l.columns + col);
        }
        float f[kVec], up[kVec];
        v[b].get(f);
        u[b].get(up);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float d = f[i] - c.mean[i], g = act_slope(fmaf(d, c.scale[i], c.shift[i]), up[i], a.act);
          s[i] += g;
          sx[i] = fmaf(g, d * c.rstd[i], sx[i]);
        }
      }
    }
    float* t = table + row * a.channels + col * kVec;
#pragma unroll
    for (int i = 0; i < kVec; ++i) t[i] = s[i], t[size + i] = sx[i];
  }
}

// The rows of threads added up, into the first row's place.
template <int kVec>
__device__ __forceinline__ void channel_sums(const Params& a, float* table) {
  const Lay l = Lay::of<kVec>(a.channels);
  const int size = table_floats<kVec>(a.channels);
  for (int c = threadIdx.x; c < a.channels; c += kThreads) {
    float s = 0.f, sx = 0.f;
    for (int r = 0; r < l.rows; ++r) s += table[r * a.channels + c], sx += table[size + r * a.channels + c];
    table[c] = s;
    table[size + c] = sx;
  }
}

// The groups' sums of gamma g and gamma g xh of a run: a warp for each group.
template <int kVec>
__device__ __forceinline__ void group_sums(const Params& a, const float* table, float2* groups) {
  const int size = table_floats<kVec>(a.channels), lane = threadIdx.x & 31;
  for (int g = threadIdx.x >> 5; g < a.groups; g += kWarps) {
    float s = 0.f, sx = 0.f;
    for (int e = lane; e < a.per; e += 32) {
      const int c = g * a.per + e;
      const float w = a.gamma ? a.gamma[c] : 1.f;
      s = fmaf(w, table[c], s);
      sx = fmaf(w, table[size + c], sx);
    }
    s = warp_reduce<Sum>(s);
    sx = warp_reduce<Sum>(sx);
    if (lane == 0) groups[g] = make_float2(s, sx);
  }
}

// A run's dx, from the means of gamma g and gamma g xh over its image's groups.
template <typename T, int kVec>
__device__ __forceinline__ void gradient(const Params& a, int64_t image, const T* x, const T* dy, T* dx, int n, const float* mean_g,
                                         const float* mean_gx, const uint8_t* kept) {
  const Lay l = Lay::of<kVec>(a.channels);
  const int row = threadIdx.x / l.across;
  if (row >= l.rows) return;
  const uint8_t* kept_dy = kept + (size_t)a.keep * a.channels * sizeof(T);
  for (int col = threadIdx.x % l.across; col < l.columns; col += l.across) {
    Channel<kVec> c;
    c.of(a, col * kVec, a.mean + image * a.groups, a.rstd + image * a.groups);
    float m[kVec], mx[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int g = (col * kVec + i) / a.per;
      m[i] = c.rstd[i] * mean_g[g];
      mx[i] = c.rstd[i] * mean_gx[g];
    }
    for (int at = row; at < n; at += l.rows * kBatch) {
      Vec<T, kVec> v[kBatch], u[kBatch];
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int pixel = at + b * l.rows;
        if (pixel < a.keep && pixel < n) {
          v[b].take(kept, pixel * l.columns + col);
          u[b].take(kept_dy, pixel * l.columns + col);
        } else if (pixel < n) {
          v[b].load(x + pixel * a.x_stride[1] + (int64_t)col * kVec);
          u[b].load(dy + pixel * a.dy_stride[1] + (int64_t)col * kVec);
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) {
        const int pixel = at + b * l.rows;
        if (pixel >= n) continue;
        float f[kVec], up[kVec];
        v[b].get(f);
        u[b].get(up);
#pragma unroll
        for (int i = 0; i < kVec; ++i) {
          const float d = f[i] - c.mean[i], g = act_slope(fmaf(d, c.scale[i], c.shift[i]), up[i], a.act);
          f[i] = fmaf(g, c.scale[i], -fmaf(d * c.rstd[i], mx[i], m[i]));
        }
        v[b].set(f);
        v[b].store(dx + pixel * a.y_stride[1] + (int64_t)col * kVec);
      }
    }
  }
}

template <typename T, int kVec>
__global__ void __launch_bounds__(kThreads, 2) cluster_backward_kernel(const __grid_constant__ Params a) {
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint8_t smem[];
  const Shared<T, kVec> s(a, smem);
  const cg::cluster_group cluster = cg::this_cluster();
  const int run = (int)cluster.block_rank(), size = table_floats<kVec>(a.channels);
  const int64_t image = blockIdx.x / a.runs, begin = run_begin(a, run);
  const int n = run_length(a, run);
  const T* x = static_cast<const T*>(a.x) + image * a.x_stride[0] + begin * a.x_stride[1];
  const T* dy = static_cast<const T*>(a.dy) + image * a.dy_stride[0] + begin * a.dy_stride[1];
  sums<T, kVec>(a, image, x, dy, n, s.table, s.kept);
  __syncthreads();
  channel_sums<kVec>(a, s.table);
  __syncthreads();
  group_sums<kVec>(a, s.table, s.groups);
  cluster.sync();
  const float inv = 1.f / ((float)a.pixels * (float)a.per);
  for (int g = threadIdx.x; g < a.groups; g += kThreads) {
    float2 m[kMaxCluster];
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < a.runs) m[r] = cluster.map_shared_rank(s.groups, r)[g];
    float sum = 0.f, sum_x = 0.f;
#pragma unroll
    for (int r = 0; r < kMaxCluster; ++r)
      if (r < a.runs) sum += m[r].x, sum_x += m[r].y;
    s.stat[g] = sum * inv;
    s.stat[a.groups + g] = sum_x * inv;
  }
  // the image's sums of the parameters' gradients, a share of the channels by each block
  if (a.gamma) {
    const int first = (int)((int64_t)a.channels * run / a.runs), last = (int)((int64_t)a.channels * (run + 1) / a.runs);
    for (int c = first + threadIdx.x; c < last; c += kThreads) {
      float v = 0.f, vx = 0.f;
#pragma unroll 4
      for (int r = 0; r < a.runs; ++r) {
        const float* t = cluster.map_shared_rank(s.table, r);
        v += t[c];
        vx += t[size + c];
      }
      a.part[2 * image * a.channels + c] = vx;
      a.part[(2 * image + 1) * a.channels + c] = v;
    }
  }
  __syncthreads();
  cluster.barrier_arrive();   // the other blocks' sums are not read any more
  gradient<T, kVec>(a, image, x, dy, static_cast<T*>(a.y) + image * a.y_stride[0] + begin * a.y_stride[1], n, s.stat, s.stat + a.groups, s.kept);
  cluster.barrier_wait();
}

template <typename T, int kVec>
__global__ void __launch_bounds__(kThreads, 2) sums_kernel(const __grid_constant__ Params a) {
  extern __shared__ __align__(16) uint8_t smem[];
  const Shared<T, kVec> s(a, smem);
  const int run = blockIdx.x % a.runs, size = table_floats<kVec>(a.channels);
  const int64_t image = blockIdx.x / a.runs, begin = run_begin(a, run);
  sums<T, kVec>(a, image, static_cast<const T*>(a.x) + image * a.x_stride[0] + begin * a.x_stride[1],
                static_cast<const T*>(a.dy) + image * a.dy_stride[0] + begin * a.dy_stride[1], run_length(a, run), s.table, s.kept);
  __syncthreads();
  channel_sums<kVec>(a, s.table);
  __syncthreads();
  group_sums<kVec>(a, s.table, reinterpret_cast<float2*>(a.group_part) + (int64_t)blockIdx.x * a.groups);
  if (a.gamma)
    for (int c = threadIdx.x; c < a.channels; c += kThreads) {
      a.part[2 * (int64_t)blockIdx.x * a.channels + c] = s.table[size + c];
      a.part[(2 * (int64_t)blockIdx.x + 1) * a.channels + c] = s.table[c];
    }
}

// The images' means of gamma g and gamma g xh, behind the runs' sums: a warp for each group of an image.
__global__ void __launch_bounds__(128) merge_sums_kernel(const __grid_constant__ Params a, int64_t images) {
  const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (at >= images * a.groups) return;
  const float2* m = reinterpret_cast<const float2*>(a.group_part) + at / a.groups * a.runs * a.groups + at % a.groups;
  float s = 0.f, sx = 0.f;
  for (int r = lane; r < a.runs; r += 32) {
    const float2 v = m[(int64_t)r * a.groups];
    s += v.x;
    sx += v.y;
  }
  s = warp_reduce<Sum>(s);
  sx = warp_reduce<Sum>(sx);
  const float inv = 1.f / ((float)a.pixels * (float)a.per);
  float* means = a.group_part + 2 * images * a.runs * a.groups + 2 * (at / a.groups) * a.groups + at % a.groups;
  if (lane == 0) means[0] = s * inv, means[a.groups] = sx * inv;
}

template <typename T, int kVec>
__global__ void __launch_bounds__(kThreads, 2) gradient_kernel(const __grid_constant__ Params a) {
  const int block = gridDim.x - 1 - blockIdx.x, run = block % a.runs;
  const int64_t image = block / a.runs, begin = run_begin(a, run);
  const float* means = a.group_part + 2 * (int64_t)gridDim.x * a.groups + 2 * image * a.groups;
  gradient<T, kVec>(a, image, static_cast<const T*>(a.x) + image * a.x_stride[0] + begin * a.x_stride[1],
                    static_cast<const T*>(a.dy) + image * a.dy_stride[0] + begin * a.dy_stride[1],
                    static_cast<T*>(a.y) + image * a.y_stride[0] + begin * a.y_stride[1], run_length(a, run), means, means + a.groups, nullptr);
}

// dgamma and dbeta: `rows` rows of [dgamma's channels][dbeta's], added up by eight rows of threads that take turns, then
// in their order.
__global__ void __launch_bounds__(256) parameters_kernel(const float* part, int64_t rows, int channels, float* dgamma, float* dbeta) {
  __shared__ float sum[8][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < 2 * channels) {
#pragma unroll 8
    for (int64_t r = row; r < rows; r += 8) s += part[r * 2 * channels + c];
  }
  sum[row][lane] = s;
  __syncthreads();
  if (row || c >= 2 * channels) return;
#pragma unroll
  for (int r = 1; r < 8; ++r) s += sum[r][lane];
  if (c < channels) dgamma[c] = s;
  else dbeta[c - channels] = s;
}

// ---------------------------------------------------------------- host side

// How a call is laid out.  cluster: runs is a cluster's blocks, one to a run; else the runs of an image, all on their
// own.
struct Plan {
  bool cluster;
  int runs;
  int64_t budget;   // bytes of shared memory for a block
};

// Shared memory beside the kept pixels, with the widest vectors that a type has.
int64_t table_bytes(const cbr_group_norm_desc_t& d) {
  return 8 * (int64_t)std::max(d.channels, kThreads * (d.dtype == CBR_F32 ? 4 : 8)) + 16 * (int64_t)d.groups + 16;
}

Plan plan_of(const cbr_group_norm_desc_t& d, bool backward) {
  Plan p{};
  const int64_t table = table_bytes(d), images = std::max<int64_t>(d.images, 1);
  // two blocks to an SM, so that one loads while the other stores; wide tables leave room for one
  p.budget = table <= 48 * 1024 ? 112 * 1024 : 226 * 1024;
  const int64_t image = d.pixels * d.channels * (d.dtype == CBR_F32 ? 4 : 2) * (backward ? 2 : 1), room = p.budget - table;
  int64_t need = 1;
  while (need < kMaxCluster && need * room < image) need *= 2;
  // an image in 16 blocks that hold a part of it, where images alone keep the SMs busy
  p.cluster = need * room >= image || images * kMaxCluster >= 2 * kSms;
  if (p.cluster) {
    // more blocks while SMs are without one, and a run keeps a few KB
    while (need < kMaxCluster && images * need <= kSms && image / (2 * need) >= 4096) need *= 2;
    p.runs = (int)need;
  } else {
    p.runs = (int)std::max<int64_t>(1, std::min<int64_t>(d.pixels, (4 * kSms + images - 1) / images));
  }
  return p;
}

// Clusters of more than 8 blocks have to be asked for, once for each kernel and device.
bool allow_wide_cluster(const void* kern) {
  static std::mutex mu;
  static std::set<std::pair<int, const void*>> done;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  std::lock_guard<std::mutex> lk(mu);
  if (done.count({dev, kern})) return true;
  if (cudaFuncSetAttribute(kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1) != cudaSuccess) {
    cudaGetLastError();
    return false;
  }
  done.insert({dev, kern});
  return true;
}

template <typename T, int kVec>
int launch(const GroupNormArgs& g, bool backward, cudaStream_t st) {
  const cbr_group_norm_desc_t& d = g.d;
  const Plan plan = plan_of(d, backward);
  Params a{};
  a.x = g.x;
  a.dy = g.dy;
  a.y = backward ? g.dx : g.y;
  a.gamma = g.gamma;
  a.beta = g.beta;
  a.mean = g.mean;
  a.rstd = g.rstd;
  for (int i = 0; i < 2; ++i) {
    a.x_stride[i] = d.x_stride[i];
    a.dy_stride[i] = d.dy_stride[i];
    a.y_stride[i] = backward ? d.dx_stride[i] : d.y_stride[i];
  }
  a.pixels = d.pixels;
  a.channels = d.channels;
  a.groups = d.groups;
  a.per = d.channels / d.groups;
  a.act = d.act;
  a.runs = plan.runs;
  a.base = d.pixels / plan.runs;
  a.extra = (int)(d.pixels % plan.runs);
  a.eps = d.eps;
  if (d.images > 0x7fffffff / plan.runs || d.images > 0x7fffffff / d.groups) return CBR_ERR_UNSUPPORTED;
  const int64_t rows = plan.cluster ? d.images : d.images * plan.runs;
  a.part = g.part;
  a.group_part = g.part + (backward ? 2 * rows * d.channels : 0);
  const int64_t fixed = ((8 * (int64_t)table_floats<kVec>(d.channels) + 16 * (int64_t)d.groups + 15) & ~int64_t(15));
  const int64_t pixel = (int64_t)d.channels * sizeof(T) * (backward ? 2 : 1);
  const unsigned blocks = (unsigned)(d.images * plan.runs);
  if (plan.cluster) {
    const int64_t longest = (d.pixels + plan.runs - 1) / plan.runs;
    a.keep = (int)std::min<int64_t>(longest, std::max<int64_t>(0, (plan.budget - fixed) / pixel));
    const auto kern = backward ? &cluster_backward_kernel<T, kVec> : &cluster_forward_kernel<T, kVec>;
    if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), 227 * 1024)) return CBR_ERR_CUDA;
    if (plan.runs > 8 && !allow_wide_cluster(reinterpret_cast<const void*>(kern))) return CBR_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(blocks);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)(fixed + a.keep * pixel);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = (unsigned)plan.runs;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, a) != cudaSuccess) {
      cudaGetLastError();
      return CBR_ERR_CUDA;
    }
  } else {
    const unsigned warps = (unsigned)((d.images * d.groups + 3) / 4);
    const auto first = backward ? &sums_kernel<T, kVec> : &moments_kernel<T, kVec>;
    if (!ensure_smem_attr(reinterpret_cast<const void*>(first), 227 * 1024)) return CBR_ERR_CUDA;
    first<<<blocks, kThreads, (size_t)fixed, st>>>(a);
    if (backward) {
      merge_sums_kernel<<<warps, 128, 0, st>>>(a, d.images);
      gradient_kernel<T, kVec><<<blocks, kThreads, 0, st>>>(a);
    } else {
      merge_moments_kernel<<<warps, 128, 0, st>>>(a, d.images);
      normalise_kernel<T, kVec><<<blocks, kThreads, 0, st>>>(a);
    }
  }
  if (backward && g.gamma)
    parameters_kernel<<<(2 * d.channels + 31) / 32, 256, 0, st>>>(g.part, rows, d.channels, g.dgamma, g.dbeta);
  return cudaGetLastError() == cudaSuccess ? CBR_OK : CBR_ERR_CUDA;
}

// The widest vectors that a map's channels, strides and addresses allow.
template <typename T>
int dispatch(const GroupNormArgs& g, bool backward, cudaStream_t st) {
  const cbr_group_norm_desc_t& d = g.d;
  const int64_t* strides[3] = {d.x_stride, backward ? d.dy_stride : d.y_stride, backward ? d.dx_stride : d.x_stride};
  const void* maps[3] = {g.x, backward ? g.dy : g.y, backward ? g.dx : g.x};
  auto fits = [&](int vec) {
    if (d.channels % vec) return false;
    for (int i = 0; i < 3; ++i) {
      if (reinterpret_cast<uintptr_t>(maps[i]) % (vec * sizeof(T))) return false;
      if ((d.images > 1 && strides[i][0] % vec) || (d.pixels > 1 && strides[i][1] % vec)) return false;
    }
    return true;
  };
  if constexpr (sizeof(T) == 2)
    if (fits(8)) return launch<T, 8>(g, backward, st);
  if (fits(4)) return launch<T, 4>(g, backward, st);
  return launch<T, 1>(g, backward, st);
}

int dispatch(const GroupNormArgs& g, bool backward, cudaStream_t st) {
  if (g.d.dtype == CBR_F32) return dispatch<float>(g, backward, st);
  return g.d.dtype == CBR_BF16 ? dispatch<__nv_bfloat16>(g, backward, st) : dispatch<__half>(g, backward, st);
}

}  // namespace
}  // namespace gn

size_t group_norm_forward_floats(const cbr_group_norm_desc_t& d) {
  const gn::Plan p = gn::plan_of(d, false);
  return p.cluster ? 0 : (size_t)d.images * p.runs * 2 * d.groups;
}
size_t group_norm_backward_floats(const cbr_group_norm_desc_t& d, bool parameters) {
  const gn::Plan p = gn::plan_of(d, true);
  if (p.cluster) return parameters ? (size_t)d.images * 2 * d.channels : 0;
  return (size_t)d.images * p.runs * 2 * (d.channels + d.groups) + (size_t)d.images * 2 * d.groups;
}
int launch_group_norm(const GroupNormArgs& a, cudaStream_t st) { return gn::dispatch(a, false, st); }
int launch_group_norm_backward(const GroupNormArgs& a, cudaStream_t st) { return gn::dispatch(a, true, st); }

}  // namespace cbr
