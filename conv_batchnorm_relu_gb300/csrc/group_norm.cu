// Group norm with an activation, channels last, forward and backward (declared in include/cbr.h).
//
// Bound by memory: x is read once and y written once where that can be.  Maps that fit the shared memory of all SMs
// at once go to clusters of up to 16 blocks: a cluster takes an image, each block a run of its pixels, which it reads
// (16-byte vectors, a thread keeps its channels) and keeps; the blocks exchange their groups' moments through
// distributed shared memory; then each normalises what it holds and writes it.  Small images are cut into slices
// of whole groups instead, which need no exchange.
//   Larger maps are a stream of tasks on a resident grid: the moments of an image's runs, and, some images later, their
// results, which read x again from L2.  So HBM is read and written all the time, which clusters that load, wait and
// store do not do (128x112x112x128 bf16 in clusters of 16: 298 us, as a stream 179: 4.6 TB/s of what has to move, and as
// much again from L2).
//   The backward does the same with x and dy, and the sums of g and g xh.
//   Moments: a thread sums its values' differences from its first one, and their squares, which costs no digits
// where the mean is far from 0; means and squared deviations are merged by their counts.  All merges have a fixed
// order.
#include <cooperative_groups.h>

#include <algorithm>
#include <climits>
#include <mutex>
#include <set>
#include <utility>

#include "cbr_internal.h"
#include "common.cuh"
#include "follow.cuh"
#include "group_norm_tasks.h"
#include "token_ops.cuh"
#include "trunk_ops.h"

namespace cbr {
namespace gn {
namespace {

using namespace tok;

constexpr int kThreads = 256, kMaxCluster = 16;
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
  int channels, groups, per, act;   // of a slice: blocks along y take slices of whole groups; per: channels of a group
  int all_channels, all_groups;
  int keep;              // pixels of a run that stay in shared memory: all of them (clusters), or none
  int runs;              // of an image, one to a block
  float eps;
};

// The parameters of this block's slice of the channels.
template <typename T>
__device__ __forceinline__ Params slice_of(Params a) {
  const int c = blockIdx.y * a.channels, g = blockIdx.y * a.groups;
  a.x = static_cast<const T*>(a.x) + c;
  a.dy = static_cast<const T*>(a.dy) + c;
  a.y = static_cast<T*>(a.y) + c;
  if (a.gamma) a.gamma += c, a.beta += c;
  a.mean += g;
  a.rstd += g;
  a.part += c;
  a.group_part += 2 * g;
  return a;
}

// kVec neighbouring channels of a pixel, as they are stored.
template <typename T, int kVec>
struct Vec {
  static constexpr int kBytes = kVec * (int)sizeof(T);
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4, kPairs = (kVec + 1) / 2;
  uint32_t w[kWords];

  __device__ __forceinline__ void load(const uint8_t* p) {
    if constexpr (kBytes == 16)
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "l"(p));
    else if constexpr (kBytes == 8)
      asm volatile("ld.global.L1::no_allocate.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "l"(p));
    else if constexpr (kBytes == 4)
      asm volatile("ld.global.b32 %0, [%1];" : "=r"(w[0]) : "l"(p));
    else
      asm volatile("ld.global.u16 %0, [%1];" : "=r"(w[0]) : "l"(p));
  }
  // global to shared memory without registers; asynchronous where the width allows
  static __device__ __forceinline__ void copy(uint32_t to, const uint8_t* p) {
    if constexpr (kBytes == 16) asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(p) : "memory");
    else if constexpr (kBytes >= 4) asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(to), "l"(p), "n"(kBytes) : "memory");
    else asm volatile("{\n\t.reg .u16 h;\n\tld.global.u16 h, [%1];\n\tst.shared.u16 [%0], h;\n\t}" ::"r"(to), "l"(p) : "memory");
  }
  // once: nobody reads it while this call runs, so L2 may give up its place first
  template <bool once = false>
  __device__ __forceinline__ void store(uint8_t* p) const {
    if constexpr (once && kBytes == 16) __stcs(reinterpret_cast<uint4*>(p), make_uint4(w[0], w[1], w[2], w[3]));
    else if constexpr (once && kBytes == 8) __stcs(reinterpret_cast<uint2*>(p), make_uint2(w[0], w[1]));
    else if constexpr (kBytes == 16) st_global_v4(p, make_uint4(w[0], w[1], w[2], w[3]));
    else if constexpr (kBytes == 8) *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[1]);
    else if constexpr (kBytes == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
    else *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
  }
  __device__ __forceinline__ void take(uint32_t from) {
    if constexpr (kBytes == 16)
      asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(from));
    else if constexpr (kBytes == 8)
      asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(from));
    else if constexpr (kBytes == 4)
      asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(from));
    else
      asm volatile("ld.shared.u16 %0, [%1];" : "=r"(w[0]) : "r"(from));
  }
  // as pairs of 32-bit values (a single one: with 0)
  __device__ __forceinline__ void get(float2 (&v)[kPairs]) const {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) v[i] = unpack2<std::is_same_v<T, __nv_bfloat16>>(w[i]);
    } else {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) v[i] = make_float2(__uint_as_float(w[2 * i]), kVec > 1 ? __uint_as_float(w[2 * i + (kVec > 1)]) : 0.f);
    }
  }
  __device__ __forceinline__ void set(const float2 (&v)[kPairs]) {
    if constexpr (sizeof(T) == 2) {
#pragma unroll
      for (int i = 0; i < kPairs; ++i) w[i] = pack2<std::is_same_v<T, __nv_bfloat16>>(v[i].x, v[i].y);
    } else {
#pragma unroll
      for (int i = 0; i < kVec; ++i) w[i] = __float_as_uint(i & 1 ? v[i / 2].y : v[i / 2].x);
    }
  }
};

// Two 32-bit values in one instruction.
__device__ __forceinline__ uint64_t bits(float2 v) { return (uint64_t)__float_as_uint(v.y) << 32 | __float_as_uint(v.x); }
__device__ __forceinline__ float2 pair(uint64_t v) { return make_float2(__uint_as_float((uint32_t)v), __uint_as_float((uint32_t)(v >> 32))); }
__device__ __forceinline__ float2 add(float2 a, float2 b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return pair(d);
}
__device__ __forceinline__ float2 sub(float2 a, float2 b) {
  uint64_t d;
  asm("sub.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)));
  return pair(d);
}
__device__ __forceinline__ float2 fma(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits(a)), "l"(bits(b)), "l"(bits(c)));
  return pair(d);
}

// How a block's threads lie over its run: a thread has a column (kVec channels) and every `rows`th pixel.  Threads behind
// the last row have nothing to do.
struct Lay {
  int columns;   // vectors of a pixel, at most kThreads
  int rows;      // of threads
  int row, col;  // this thread's
  template <int kVec>
  static __device__ __forceinline__ Lay of(int channels) {
    Lay l;
    l.columns = channels / kVec;
    l.rows = kThreads / l.columns;
    l.row = threadIdx.x / l.columns;
    l.col = threadIdx.x - l.row * l.columns;
    return l;
  }
};

// The pixels of run `r` of an image.
__device__ __forceinline__ int64_t run_begin(const Params& a, int r) { return a.base * r + min(r, a.extra); }
__device__ __forceinline__ int run_length(const Params& a, int r) { return (int)a.base + (r < a.extra); }
// Of `n` pixels, those of this thread's row.
__device__ __forceinline__ int turns(int n, const Lay& l) { return l.row < l.rows && l.row < n ? (n - l.row + l.rows - 1) / l.rows : 0; }

// SiLU's exponential and quotient are the hardware's, for f32 maps too: by their bounds good to (5 + 1.2 |z|) 2^-23 of the
// result (a z that is off by half a step alone makes |z| 2^-24 of it), and 0 below -87.  (With expf and a rounded quotient 64x112x112x64 f32 took 121 us for 95, backward 206 for 157.)
template <int kAct>
__device__ __forceinline__ float act_of(float z) {
  if constexpr (kAct == CBR_ACT_RELU) return Max::of(z, 0.f);
  if constexpr (kAct == CBR_ACT_SILU) return __fdividef(z, 1.f + __expf(-z));
  return z;
}
template <int kAct>
__device__ __forceinline__ float act_slope(float z, float up) {
  if constexpr (kAct == CBR_ACT_RELU) return z > 0.f ? up : 0.f;
  if constexpr (kAct == CBR_ACT_SILU) {
    const float s = __fdividef(1.f, 1.f + __expf(-z));
    return up * (s * fmaf(z, 1.f - s, 1.f));
  }
  return up;
}
__device__ __forceinline__ float act_of(float z, int act) {
  return act == CBR_ACT_RELU ? act_of<CBR_ACT_RELU>(z) : act == CBR_ACT_SILU ? act_of<CBR_ACT_SILU>(z) : z;
}
__device__ __forceinline__ float act_slope(float z, float up, int act) {
  return act == CBR_ACT_RELU ? act_slope<CBR_ACT_RELU>(z, up) : act == CBR_ACT_SILU ? act_slope<CBR_ACT_SILU>(z, up) : up;
}
// Runs the body made for the activation.
template <typename Body>
__device__ __forceinline__ void by_act(int act, Body body) {
  if (act == CBR_ACT_RELU) body(std::integral_constant<int, CBR_ACT_RELU>{});
  else if (act == CBR_ACT_SILU) body(std::integral_constant<int, CBR_ACT_SILU>{});
  else body(std::integral_constant<int, CBR_ACT_NONE>{});
}

// Values so far apart that rstd^2 leaves fp32's range, or their differences do: x is taken times a power of two near rstd,
// and rstd divided by it, one value at a time, by blocks that have such a channel.  (That the code is there costs 256x56x56x64
// f16 backward 1.5%, 105 and 106.7 us, clusters' backward 1 to 2% and 1x224x224x64 f32's 3.5%.)
__device__ __forceinline__ bool is_far(float rstd) { return rstd < 0x1p-50f; }
__device__ __forceinline__ float far_unit(float rstd) { return __uint_as_float(max(__float_as_uint(rstd) & 0x7f800000u, 0x00800000u)); }
// 1 / unit
__device__ __forceinline__ float far_rest(float unit) { return __uint_as_float(0x7f000000u - __float_as_uint(unit)); }
struct Far {
  float unit, mean, scale, shift, rest;   // rest: rstd less its unit

  __device__ __forceinline__ Far(const Params& a, int c, float center, float rstd) {
    unit = far_unit(rstd);
    mean = -center * unit;
    rest = rstd * far_rest(unit);
    scale = a.gamma ? rest * a.gamma[c] : rest;
    shift = a.gamma ? a.beta[c] : 0.f;
  }
  __device__ __forceinline__ float distance(float x) const { return fmaf(x, unit, mean); }
  __device__ __forceinline__ float result(float x, int act) const { return act_of(fmaf(distance(x), scale, shift), act); }
  __device__ __forceinline__ float slope(float x, float up, int act) const { return act_slope(fmaf(distance(x), scale, shift), up, act); }
  // (the two means are of gamma g and gamma g xh)
  __device__ __forceinline__ float gradient(float x, float up, int act, float rstd, float mean_g, float mean_gx) const {
    const float times = scale * unit, mx = -rstd * rest * mean_gx;
    return fmaf(slope(x, up, act), times, fmaf(distance(x), mx, -rstd * mean_g));
  }
};

// A thread's channels of an array in shared memory.
template <int kVec>
__device__ __forceinline__ void take_channels(float2 (&v)[(kVec + 1) / 2], const float* p, int col) {
  p += col * kVec;
  if constexpr (kVec == 1) {
    v[0] = make_float2(p[0], 0.f);
  } else {
#pragma unroll
    for (int i = 0; i < kVec / 4; ++i) {
      const float4 u = reinterpret_cast<const float4*>(p)[i];
      v[2 * i] = make_float2(u.x, u.y);
      v[2 * i + 1] = make_float2(u.z, u.w);
    }
  }
}

// A thread's pixels of a column in kOps maps: global and shared-memory addresses of the first, and the steps to the next
// ones.  Shared memory has `slots` places for them (a multiple of the batches), used in turn.
template <int kOps>
struct Way {
  const uint8_t* at[kOps];
  int64_t step[kOps];
  uint32_t held[kOps], held_step;
  int all, slots;
};
// By the maps read: pixels that a thread takes at a time, batches of them that it has asked for, blocks to an SM.  The
// forward moves more and computes less: deeper rings (two blocks with 5 batches and three with 3: 180 and 234 us at
// 128x112x112x128 bf16, 67 and 70 at 64x64x64x128 f32); the backward is near enough with two blocks and three (107.7 and
// 106.9 us at 256x56x56x64 f16, 99 and 108 at 64x64x64x128 f32).
template <int kOps>
constexpr int kBatch = 4 / kOps;
template <int kOps, int kBytes>
constexpr int kAhead = kOps == 1 ? 5 : kBytes == 16 ? 3 : 6;
template <int kOps>
constexpr int kResident = kOps == 1 ? 2 : 3;

// Reads a column through shared memory, some batches ahead from the start on.  A thread reads only what it has
// copied itself, so it waits for its own copies alone.
template <typename V, int kOps>
struct Reader {
  static constexpr int kBatch = gn::kBatch<kOps>;
  Way<kOps> way;       // of the next pixel to ask for
  uint32_t from[kOps];
  int asked = 0, slot = 0;

  __device__ __forceinline__ explicit Reader(const Way<kOps>& w) : way(w) {
#pragma unroll
    for (int o = 0; o < kOps; ++o) from[o] = w.held[o];
#pragma unroll 1
    for (int i = 0; i < kAhead<kOps, V::kBytes>; ++i) ask();
  }
  __device__ __forceinline__ void copy() {
#pragma unroll
    for (int o = 0; o < kOps; ++o) {
      V::copy(way.held[o], way.at[o]);
      way.held[o] += way.held_step;
      way.at[o] += way.step[o];
    }
  }
  __device__ __forceinline__ void ask() {
    if (asked + kBatch <= way.all) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b) copy();
      asked += kBatch;
      slot += kBatch;
      if (slot == way.slots) {
        slot = 0;
#pragma unroll
        for (int o = 0; o < kOps; ++o) way.held[o] -= way.slots * way.held_step;
      }
    } else {
      for (; asked < way.all; ++asked) copy();   // the last ones: less than a batch, which a ring has room for
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
  // take() gets each pixel's vectors.
  template <typename Take>
  __device__ __forceinline__ void run(Take take) {
    V v[kBatch][kOps];
    int done = 0, at = 0;
    auto fetch = [&](int b) {
#pragma unroll
      for (int o = 0; o < kOps; ++o) {
        v[b][o].take(from[o]);
        from[o] += way.held_step;
      }
    };
#pragma unroll 1
    for (; done + kBatch <= way.all; done += kBatch) {
      asm volatile("cp.async.wait_group %0;" ::"n"(kAhead<kOps, V::kBytes> - 1) : "memory");
#pragma unroll
      for (int b = 0; b < kBatch; ++b) fetch(b);
      at += kBatch;
      if (at == way.slots) {
        at = 0;
#pragma unroll
        for (int o = 0; o < kOps; ++o) from[o] -= way.slots * way.held_step;
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b) take(v[b]);
      ask();   // into the places just read
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
#pragma unroll 1
    for (; done < way.all; ++done) {
      fetch(0);
      take(v[0]);
    }
  }
};

// Goes over a column that shared memory holds.
template <typename V, int kOps, typename Take>
__device__ __forceinline__ void reread(const Way<kOps>& way, Take take) {
  constexpr int kBatch = gn::kBatch<kOps>;
  V v[kBatch][kOps];
  uint32_t from[kOps];
  int done = 0;
#pragma unroll
  for (int o = 0; o < kOps; ++o) from[o] = way.held[o];
  auto fetch = [&](int b) {
#pragma unroll
    for (int o = 0; o < kOps; ++o) {
      v[b][o].take(from[o]);
      from[o] += way.held_step;
    }
  };
#pragma unroll 1
  for (; done + kBatch <= way.all; done += kBatch) {
#pragma unroll
    for (int b = 0; b < kBatch; ++b) fetch(b);
#pragma unroll
    for (int b = 0; b < kBatch; ++b) take(v[b]);
  }
#pragma unroll 1
  for (; done < way.all; ++done) {
    fetch(0);
    take(v[0]);
  }
}

template <int kVec>
constexpr int kTable = kThreads * kVec;   // values of all channels in all rows of threads, at the most

// Shared memory holds a run's pixels one after the other (a.keep of them, dy's behind x's), or, where a.keep is 0, a ring
// for each thread: kAhead batches of vectors, a step of all threads apart.
template <typename T, int kVec, int kOps>
__device__ __forceinline__ Way<kOps> way_of(const Params& a, const Lay& l, const T* x, const T* dy, const uint8_t* kept, int n) {
  using V = Vec<T, kVec>;
  const int col = l.col;
  Way<kOps> w;
  const bool ring = a.keep == 0;
  w.at[0] = reinterpret_cast<const uint8_t*>(x + l.row * a.x_stride[1] + (int64_t)col * kVec);
  w.step[0] = l.rows * a.x_stride[1] * (int64_t)sizeof(T);
  w.held[0] = smem_u32(kept) + (ring ? threadIdx.x : l.row * l.columns + col) * V::kBytes;
  w.held_step = (ring ? kThreads : l.rows * l.columns) * V::kBytes;
  w.slots = ring ? kAhead<kOps, V::kBytes> * kBatch<kOps> : INT_MAX;
  w.all = turns(n, l);
  if constexpr (kOps == 2) {
    w.at[1] = reinterpret_cast<const uint8_t*>(dy + l.row * a.dy_stride[1] + (int64_t)col * kVec);
    w.step[1] = l.rows * a.dy_stride[1] * (int64_t)sizeof(T);
    w.held[1] = w.held[0] + (ring ? w.slots * w.held_step : a.keep * a.channels * (uint32_t)sizeof(T));
  }
  return w;
}

// ---------------------------------------------------------------- forward

// A run's moments: `table` gets (mean, squared deviations) of every channel in every row of threads.
template <typename T, int kVec>
__device__ __forceinline__ void moments(const Params& a, const Lay& l, const T* x, int n, float* table, const uint8_t* kept) {
  using V = Vec<T, kVec>;
  const Way<1> way = way_of<T, kVec, 1>(a, l, x, nullptr, kept, n);
  if (way.all == 0) return;
  Reader<V, 1> reader(way);
  float2 first[V::kPairs], s[V::kPairs], q[V::kPairs];
  V v;
  v.load(way.at[0]);
  v.get(first);
#pragma unroll
  for (int i = 0; i < V::kPairs; ++i) s[i] = q[i] = make_float2(0.f, 0.f);
  reader.run([&](V (&v)[1]) {
    float2 f[V::kPairs];
    v[0].get(f);
#pragma unroll
    for (int i = 0; i < V::kPairs; ++i) {
      const float2 d = sub(f[i], first[i]);
      s[i] = add(s[i], d);
      q[i] = fma(d, d, q[i]);
    }
  });
  const float inv = 1.f / (float)way.all;
  float* m = table + l.row * a.channels + l.col * kVec;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    const float si = i & 1 ? s[i / 2].y : s[i / 2].x, qi = i & 1 ? q[i / 2].y : q[i / 2].x;
    m[i] = (i & 1 ? first[i / 2].y : first[i / 2].x) + si * inv;
    m[kTable<kVec> + i] = qi - si * (si * inv);
  }
}

// How `many` sums of `terms` terms are shared out: 2^log lanes (at most a warp) to each.
struct Team {
  int log;
  static __device__ __forceinline__ Team of(int many, int terms) {
    // the largest power of two that is no more than the terms nor the threads there are for each sum
    const int most = min(min(32, terms), max(1, kThreads / many));
    return Team{31 - __clz(most)};
  }
  __device__ __forceinline__ int lanes() const { return 1 << log; }
  __device__ __forceinline__ int sub() const { return threadIdx.x & (lanes() - 1); }
  __device__ __forceinline__ int first() const { return threadIdx.x >> log; }   // of the sums
  __device__ __forceinline__ int teams() const { return kThreads >> log; }
  __device__ __forceinline__ float sum(float v) const {
    for (int o = lanes() >> 1; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
  }
};
// Of the sums over a run: rows of threads into channels, channels into groups, runs into images.
struct Teams {
  Team channels, groups, runs;
  static __device__ __forceinline__ Teams of(const Params& a, const Lay& l) {
    return Teams{Team::of(a.channels, l.rows), Team::of(a.groups, a.per), Team::of(a.groups, a.runs)};
  }
};

// The channels' moments of a run, from the rows of threads', into the first row's place.
template <int kVec>
__device__ __forceinline__ void channel_moments(const Params& a, const Lay& l, Team team, int n, float* table) {
  const int lanes = team.lanes(), sub = team.sub();
  const int base = n / l.rows, extra = n - base * l.rows, rows = min(n, l.rows);
  const float inv = 1.f / (float)max(n, 1);
  for (int first = 0; first < a.channels; first += team.teams()) {
    const int c = first + team.first();
    const bool in = c < a.channels;
    const float* m = table + min(c, a.channels - 1);
    const float ref = m[0];
    float s = 0.f, q = 0.f;
    for (int r = sub; r < rows; r += lanes) s = fmaf((float)(base + (r < extra)), m[r * a.channels] - ref, s);
    const float mean = ref + team.sum(s) * inv;
    for (int r = sub; r < rows; r += lanes) {
      const float d = m[r * a.channels] - mean;
      q += fmaf((float)(base + (r < extra)) * d, d, m[kTable<kVec> + r * a.channels]);
    }
    q = team.sum(q);
    __syncwarp();
    if (in && sub == 0) table[c] = n ? mean : 0.f, table[kTable<kVec> + c] = n ? q : 0.f;
  }
}

// The groups' moments of a run from its channels', which have n values each.
template <int kVec>
__device__ __forceinline__ void group_moments(const Params& a, Team team, int n, const float* table, float2* groups) {
  const int lanes = team.lanes(), sub = team.sub();
  const float inv = 1.f / (float)a.per;
  for (int first = 0; first < a.groups; first += team.teams()) {
    const int g = first + team.first();
    const float* m = table + min(g, a.groups - 1) * a.per;
    const float ref = m[0];
    float s = 0.f, q = 0.f;
    for (int e = sub; e < a.per; e += lanes) s += m[e] - ref;
    const float mean = ref + team.sum(s) * inv;
    for (int e = sub; e < a.per; e += lanes) {
      const float d = m[e] - mean;
      q += fmaf((float)n * d, d, m[kTable<kVec> + e]);
    }
    q = team.sum(q);
    if (g < a.groups && sub == 0) groups[g] = make_float2(mean, q);
  }
}

// (count, mean, squared deviations) of two sets as one.  An empty set has no mean to differ from: the square of the other's
// may be past the range.
__device__ __forceinline__ void merge_moments(float& n, float& mean, float& q, float n2, float mean2, float q2) {
  if (n2 == 0.f) return;
  if (n == 0.f) {
    n = n2, mean = mean2, q = q2;
    return;
  }
  const float d = mean2 - mean, share = n2 / (n + n2);
  mean = fmaf(d, share, mean);
  q += fmaf(d * d, n * share, q2);
  n += n2;
}

// (squares may be below 0 by their roundings; 0 where they are not finite)
__device__ __forceinline__ float rstd_of(float squares, float n, float eps) {
  return 1.f / sqrtf((fabsf(squares) < INFINITY ? fmaxf(squares, 0.f) : INFINITY) / n + eps);
}

// Squares past fp32's range (of values some 2^64 apart), infinities and NaN leave a group's sums infinite or NaN, and its
// rstd 0.  Its moments are then taken again by the block that merges them, from x, in 64 bits, whose sums are what the
// definition says wherever an infinity stands.  (That the code is there costs 1% of the stream, 128x112x112x128 bf16 176.5 and
// 179 us, and 0.2 us of the smallest maps; as a function that is called it cost the stream 16%.)
__device__ __forceinline__ bool lost(float rstd) { return !(rstd > 0.f); }

template <int kWarps>
__device__ __forceinline__ double block_sum(double v, double* sums) {
#pragma unroll 1
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0.0;
#pragma unroll 1
  for (int i = 0; i < kWarps; ++i) v += sums[i];
  return v;
}

// x: a group's first value; the block has kWarps warps, which `sums` has places for.  By the whole block.  Whether there is
// an infinity or a NaN is seen first, by a plain sum; one NaN is enough (128x112x112x128 bf16, all NaN: 4.9 ms).
template <int kWarps, typename T>
__device__ __forceinline__ void far_moments(const T* x, int64_t stride, int64_t pixels, int per, float eps, double* sums, float* mean, float* rstd) {
  constexpr uint32_t kTurns = 64;
  const int width = min(per, kWarps * 32), rows = kWarps * 32 / width, row = threadIdx.x / width;
  float plain = 0.f;
#pragma unroll 1
  for (uint32_t first = 0; first < (uint32_t)pixels; first += kTurns * rows) {
    if (row < rows)
#pragma unroll 1
      for (int c = threadIdx.x - row * width; c < per; c += width)
#pragma unroll 4
        for (uint32_t p = first + row; p < min((uint32_t)pixels, first + kTurns * rows); p += rows) plain = fmaf(to_f(x[p * stride + c]), 0x1p-40f, plain);
    if (__syncthreads_or(plain != plain)) break;
  }
  // 1 / (values of the group), from 32 bits by a Newton step
  const double all = (double)pixels * per, near = (double)(1.f / (float)all), share = near * (2.0 - all * near);
  double center = block_sum<kWarps>((double)plain, sums);
  if (!(fabs(center) < 0x1p127)) {
    if (threadIdx.x == 0) *mean = (float)center, *rstd = __int_as_float(0x7fffffff);
    return;
  }
  center = 0.0;
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    double s = 0.0;
    if (row < rows)
#pragma unroll 1
      for (int c = threadIdx.x - row * width; c < per; c += width)
#pragma unroll 4
        for (uint32_t p = row; p < (uint32_t)pixels; p += rows) {
          const double d = (double)to_f(x[p * stride + c]) - center;
          s += pass ? d * d : d;
        }
    s = block_sum<kWarps>(s, sums) * share;
    // (eps beside squares that fp32 does not hold, or sums of them: the root in 32 bits, of what is above 2^-80)
    if (pass && threadIdx.x == 0) *mean = (float)center, *rstd = 0x1p-80f / sqrtf((float)((s + (double)eps) * 0x1p-160));
    center = s;
  }
}

// Shared memory: two values of each channel for each row of threads; two of each group (a run's); two more (an image's);
// five of each channel (what the results are computed with); the channels' groups; the kept pixels or rings.
__host__ __device__ constexpr int64_t shared_bytes(int64_t table, int channels, int groups) {
  return 8 * table + 16 * (((int64_t)groups + 1) & ~1) + 20 * (((int64_t)channels + 3) & ~3) + ((2 * (int64_t)channels + 15) & ~15);
}
template <typename T, int kVec>
struct Shared {
  float* table;
  float2* groups;
  float* stat;        // mean, then rstd (backward: the two means) of each group
  float* coef;        // mean, scale, shift (backward: and two more) of each channel, `step` apart
  uint16_t* group;
  uint8_t* kept;
  int step;
  __device__ __forceinline__ Shared(const Params& a, uint8_t* smem) {
    const int even = (a.groups + 1) & ~1;
    step = (a.channels + 3) & ~3;
    table = reinterpret_cast<float*>(smem);
    groups = reinterpret_cast<float2*>(table + 2 * kTable<kVec>);
    stat = reinterpret_cast<float*>(groups + even);
    coef = stat + 2 * even;
    group = reinterpret_cast<uint16_t*>(coef + 5 * step);
    kept = smem + shared_bytes(kTable<kVec>, a.channels, a.groups);
  }
  // the channels' groups, visible to the block after its next barrier
  __device__ __forceinline__ void set_groups(const Params& a) const {
    for (int c = threadIdx.x; c < a.channels; c += kThreads) group[c] = (uint16_t)(c / a.per);
  }
  // z = (x - mean) scale + shift.  Whether a channel's values are far apart.
  __device__ __forceinline__ bool set_channels(const Params& a, const float* mean, const float* rstd) const {
    bool far = false;
    for (int c = threadIdx.x; c < a.channels; c += kThreads) {
      const int g = group[c];
      coef[c] = mean[g];
      coef[step + c] = a.gamma ? rstd[g] * a.gamma[c] : rstd[g];
      coef[2 * step + c] = a.gamma ? a.beta[c] : 0.f;
      far |= is_far(rstd[g]);
    }
    return far;
  }
  // dx = scale g - rstd (mean_g + (x - mean) rstd mean_gx)
  __device__ __forceinline__ void set_gradient(const Params& a, const float* rstd) const {
    for (int c = threadIdx.x; c < a.channels; c += kThreads) {
      const int g = group[c];
      const float r = -rstd[g];
      coef[3 * step + c] = r * stat[g];
      coef[4 * step + c] = r * rstd[g] * stat[a.groups + g];
    }
  }
};

// Where values are far apart: each(channel, its coefficients) for a thread's channels, whose values are taken from memory.
template <typename T, int kVec, typename Each>
__device__ __forceinline__ void each_far(const Params& a, const Lay& l, const Shared<T, kVec>& s, const float* rstd, Each each) {
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if (l.row >= l.rows) return;
#pragma unroll 1
  for (int c = l.col * kVec; c < (l.col + 1) * kVec; ++c) each(c, Far(a, c, s.coef[c], rstd[s.group[c]]));
}

// A run normalised: what shared memory holds (kHeld), or read again.  ready() brings the coefficients, the whole block
// in step, after the first loads, and says whether a channel's values are far apart.
template <typename T, int kVec, bool kHeld, typename Ready>
__device__ __forceinline__ void normalise(const Params& a, const Lay& l, const Shared<T, kVec>& s, const T* x, T* y, int n, Ready ready) {
  using V = Vec<T, kVec>;
  std::conditional_t<kHeld, Way<1>, Reader<V, 1>> source(way_of<T, kVec, 1>(a, l, x, nullptr, s.kept, n));
  if (__builtin_expect(ready(), 0)) {
    each_far(a, l, s, s.stat + a.groups, [&](int c, const Far& w) {
#pragma unroll 1
      for (int p = l.row; p < n; p += l.rows) y[p * a.y_stride[1] + c] = from_f<T>(w.result(to_f(x[p * a.x_stride[1] + c]), a.act));
    });
    return;
  }
  float2 mean[V::kPairs], scale[V::kPairs], shift[V::kPairs];
  take_channels<kVec>(mean, s.coef, l.col);
  take_channels<kVec>(scale, s.coef + s.step, l.col);
  take_channels<kVec>(shift, s.coef + 2 * s.step, l.col);
  uint8_t* out = reinterpret_cast<uint8_t*>(y + l.row * a.y_stride[1] + l.col * kVec);
  const int64_t out_step = l.rows * a.y_stride[1] * (int64_t)sizeof(T);
  by_act(a.act, [&](auto act) {
    auto make = [&](V (&v)[1]) {
      float2 f[V::kPairs];
      v[0].get(f);
#pragma unroll
      for (int i = 0; i < V::kPairs; ++i) {
        f[i] = fma(sub(f[i], mean[i]), scale[i], shift[i]);
        f[i] = make_float2(act_of<decltype(act)::value>(f[i].x), act_of<decltype(act)::value>(f[i].y));
      }
      v[0].set(f);
      v[0].template store<!kHeld>(out);
      out += out_step;
    };
    if constexpr (kHeld) reread<V, 1>(source, make);
    else source.run(make);
  });
}

template <typename T, int kVec>
__global__ void __launch_bounds__(kThreads, 2) cluster_forward_kernel(const __grid_constant__ Params whole) {
  const Params a = slice_of<T>(whole);
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint8_t smem[];
  const Shared<T, kVec> s(a, smem);
  const cg::cluster_group cluster = cg::this_cluster();
  const int run = (int)cluster.block_rank();
  const int64_t image = blockIdx.x / a.runs;
  const int n = run_length(a, run);
  const T* x = static_cast<const T*>(a.x) + image * a.x_stride[0] + run_begin(a, run) * a.x_stride[1];
  const Lay l = Lay::of<kVec>(a.channels);
  const Teams teams = Teams::of(a, l);
  s.set_groups(a);
  moments<T, kVec>(a, l, x, n, s.table, s.kept);
  __syncthreads();
  channel_moments<kVec>(a, l, teams.channels, n, s.table);
  __syncthreads();
  group_moments<kVec>(a, teams.groups, n, s.table, s.groups);
  cluster.sync();
  const float total = (float)a.pixels * (float)a.per;
  bool again = false;
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
    again |= lost(rstd);
    s.stat[g] = mean;
    s.stat[a.groups + g] = rstd;
    if (run == 0) a.mean[image * a.all_groups + g] = mean, a.rstd[image * a.all_groups + g] = rstd;
  }
  if (__builtin_expect(__syncthreads_or(again), 0)) {   // the same in all blocks, as their sums are
#pragma unroll 1
    for (int g = 0; g < a.groups; ++g) {
      if (!lost(s.stat[a.groups + g])) continue;
      far_moments<kThreads / 32>(x - run_begin(a, run) * a.x_stride[1] + g * a.per, a.x_stride[1], a.pixels, a.per, a.eps,
                                 reinterpret_cast<double*>(s.table), s.stat + g, s.stat + a.groups + g);
      if (run == 0 && threadIdx.x == 0) a.mean[image * a.all_groups + g] = s.stat[g], a.rstd[image * a.all_groups + g] = s.stat[a.groups + g];
    }
    cluster.sync();   // nobody writes before all have read: y may be x
  }
  cluster.barrier_arrive();   // the other blocks' moments are not read any more
  const bool far = __syncthreads_or(s.set_channels(a, s.stat, s.stat + a.groups));
  normalise<T, kVec, true>(a, l, s, x, static_cast<T*>(a.y) + image * a.y_stride[0] + run_begin(a, run) * a.y_stride[1], n, [&] { return far; });
  cluster.barrier_wait();
}

// ---------------------------------------------------------------- backward

// A run's sums of g and g xh: `table` gets them (the second still to be multiplied by rstd, or by the rest of it) of every
// channel in every row of threads.  ready() as above, whose answer it gives.
template <typename T, int kVec, typename Ready>
__device__ __forceinline__ bool sums(const Params& a, const Lay& l, const Shared<T, kVec>& s, const T* x, const T* dy, int n, const float* rstd,
                                     Ready ready) {
  using V = Vec<T, kVec>;
  Reader<V, 2> reader(way_of<T, kVec, 2>(a, l, x, dy, s.kept, n));
  if (__builtin_expect(ready(), 0)) {
    each_far(a, l, s, rstd, [&](int c, const Far& w) {
      float sum = 0.f, sum_x = 0.f;
#pragma unroll 1
      for (int p = l.row; p < n; p += l.rows) {
        const float v = to_f(x[p * a.x_stride[1] + c]), g = w.slope(v, to_f(dy[p * a.dy_stride[1] + c]), a.act);
        sum += g;
        sum_x = fmaf(g, w.distance(v), sum_x);
      }
      s.table[l.row * a.channels + c] = sum;
      s.table[kTable<kVec> + l.row * a.channels + c] = sum_x;
    });
    return true;
  }
  float2 mean[V::kPairs], scale[V::kPairs], shift[V::kPairs], sum[V::kPairs], sum_x[V::kPairs];
  take_channels<kVec>(mean, s.coef, l.col);
  take_channels<kVec>(scale, s.coef + s.step, l.col);
  take_channels<kVec>(shift, s.coef + 2 * s.step, l.col);
#pragma unroll
  for (int i = 0; i < V::kPairs; ++i) sum[i] = sum_x[i] = make_float2(0.f, 0.f);
  by_act(a.act, [&](auto act) {
    reader.run([&](V (&v)[2]) {
      float2 f[V::kPairs], up[V::kPairs];
      v[0].get(f);
      v[1].get(up);
#pragma unroll
      for (int i = 0; i < V::kPairs; ++i) {
        const float2 d = sub(f[i], mean[i]), z = fma(d, scale[i], shift[i]);
        const float2 g = make_float2(act_slope<decltype(act)::value>(z.x, up[i].x), act_slope<decltype(act)::value>(z.y, up[i].y));
        sum[i] = add(sum[i], g);
        sum_x[i] = fma(g, d, sum_x[i]);
      }
    });
  });
  if (l.row >= l.rows) return false;
  float* t = s.table + l.row * a.channels + l.col * kVec;
#pragma unroll
  for (int i = 0; i < kVec; ++i) {
    t[i] = i & 1 ? sum[i / 2].y : sum[i / 2].x;
    t[kTable<kVec> + i] = i & 1 ? sum_x[i / 2].y : sum_x[i / 2].x;
  }
  return false;
}

// The channels' sums of a run, from the rows of threads', into the first row's place.
template <int kVec>
__device__ __forceinline__ void channel_sums(const Params& a, const Lay& l, Team team, float* table, const uint16_t* group, const float* rstd,
                                             bool far) {
  const int lanes = team.lanes(), sub = team.sub();
  for (int first = 0; first < a.channels; first += team.teams()) {
    const int c = first + team.first();
    const float* t = table + min(c, a.channels - 1);
    float s = 0.f, sx = 0.f;
    for (int r = sub; r < l.rows; r += lanes) s += t[r * a.channels], sx += t[kTable<kVec> + r * a.channels];
    s = team.sum(s);
    sx = team.sum(sx);
    __syncwarp();
    if (c < a.channels && sub == 0) {
      float r = rstd[group[c]];
      if (far) r *= far_rest(far_unit(r));
      table[c] = s, table[kTable<kVec> + c] = sx * r;
    }
  }
}

// The groups' sums of gamma g and gamma g xh of a run.
template <int kVec>
__device__ __forceinline__ void group_sums(const Params& a, Team team, const float* table, float2* groups) {
  const int lanes = team.lanes(), sub = team.sub();
  for (int first = 0; first < a.groups; first += team.teams()) {
    const int g = first + team.first(), at = min(g, a.groups - 1) * a.per;
    float s = 0.f, sx = 0.f;
    for (int e = sub; e < a.per; e += lanes) {
      const float w = a.gamma ? a.gamma[at + e] : 1.f;
      s = fmaf(w, table[at + e], s);
      sx = fmaf(w, table[kTable<kVec> + at + e], sx);
    }
    s = team.sum(s);
    sx = team.sum(sx);
    if (g < a.groups && sub == 0) groups[g] = make_float2(s, sx);
  }
}

// A run's dx, from the means of gamma g and gamma g xh over its image's groups; kHeld and ready() as above.
template <typename T, int kVec, bool kHeld, typename Ready>
__device__ __forceinline__ void gradient(const Params& a, const Lay& l, const Shared<T, kVec>& s, const T* x, const T* dy, T* dx, int n,
                                         const float* rstd, Ready ready) {
  using V = Vec<T, kVec>;
  std::conditional_t<kHeld, Way<2>, Reader<V, 2>> source(way_of<T, kVec, 2>(a, l, x, dy, s.kept, n));
  if (__builtin_expect(ready(), 0)) {
    each_far(a, l, s, rstd, [&](int c, const Far& w) {
      const int g = s.group[c];
#pragma unroll 1
      for (int p = l.row; p < n; p += l.rows)
        dx[p * a.y_stride[1] + c] = from_f<T>(w.gradient(to_f(x[p * a.x_stride[1] + c]), to_f(dy[p * a.dy_stride[1] + c]), a.act, rstd[g], s.stat[g],
                                                         s.stat[a.groups + g]));
    });
    return;
  }
  float2 mean[V::kPairs], scale[V::kPairs], shift[V::kPairs], m[V::kPairs], mx[V::kPairs];
  take_channels<kVec>(mean, s.coef, l.col);
  take_channels<kVec>(scale, s.coef + s.step, l.col);
  take_channels<kVec>(shift, s.coef + 2 * s.step, l.col);
  take_channels<kVec>(m, s.coef + 3 * s.step, l.col);
  take_channels<kVec>(mx, s.coef + 4 * s.step, l.col);
  uint8_t* out = reinterpret_cast<uint8_t*>(dx + l.row * a.y_stride[1] + l.col * kVec);
  const int64_t out_step = l.rows * a.y_stride[1] * (int64_t)sizeof(T);
  by_act(a.act, [&](auto act) {
    auto make = [&](V (&v)[2]) {
      float2 f[V::kPairs], up[V::kPairs];
      v[0].get(f);
      v[1].get(up);
#pragma unroll
      for (int i = 0; i < V::kPairs; ++i) {
        const float2 d = sub(f[i], mean[i]), z = fma(d, scale[i], shift[i]);
        const float2 g = make_float2(act_slope<decltype(act)::value>(z.x, up[i].x), act_slope<decltype(act)::value>(z.y, up[i].y));
        f[i] = fma(g, scale[i], fma(d, mx[i], m[i]));
      }
      v[0].set(f);
      v[0].template store<!kHeld>(out);
      out += out_step;
    };
    if constexpr (kHeld) reread<V, 2>(source, make);
    else source.run(make);
  });
}

template <typename T, int kVec>
__global__ void __launch_bounds__(kThreads, 2) cluster_backward_kernel(const __grid_constant__ Params whole) {
  let_next_kernel_start();
  const Params a = slice_of<T>(whole);
  namespace cg = cooperative_groups;
  extern __shared__ __align__(16) uint8_t smem[];
  const Shared<T, kVec> s(a, smem);
  const cg::cluster_group cluster = cg::this_cluster();
  const int run = (int)cluster.block_rank();
  const int64_t image = blockIdx.x / a.runs, begin = run_begin(a, run);
  const int n = run_length(a, run);
  const T* x = static_cast<const T*>(a.x) + image * a.x_stride[0] + begin * a.x_stride[1];
  const T* dy = static_cast<const T*>(a.dy) + image * a.dy_stride[0] + begin * a.dy_stride[1];
  const Lay l = Lay::of<kVec>(a.channels);
  const Teams teams = Teams::of(a, l);
  const float *mean = a.mean + image * a.all_groups, *rstd = a.rstd + image * a.all_groups;
  s.set_groups(a);
  const bool far = sums<T, kVec>(a, l, s, x, dy, n, rstd, [&] {
    __syncthreads();
    return __syncthreads_or(s.set_channels(a, mean, rstd)) != 0;
  });
  __syncthreads();
  channel_sums<kVec>(a, l, teams.channels, s.table, s.group, rstd, far);
  __syncthreads();
  group_sums<kVec>(a, teams.groups, s.table, s.groups);
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
        vx += t[kTable<kVec> + c];
      }
      a.part[2 * image * a.all_channels + c] = vx;
      a.part[(2 * image + 1) * a.all_channels + c] = v;
    }
  }
  __syncthreads();
  cluster.barrier_arrive();   // the other blocks' sums are not read any more
  s.set_gradient(a, rstd);
  __syncthreads();
  gradient<T, kVec, true>(a, l, s, x, dy, static_cast<T*>(a.y) + image * a.y_stride[0] + begin * a.y_stride[1], n, rstd, [&] { return far; });
  cluster.barrier_wait();
}

// ---------------------------------------------------------------- maps larger than the clusters' shared memory

template <typename T, int kVec, int kOps>
__host__ __device__ constexpr int ring_bytes() {
  return kOps * kAhead<kOps, Vec<T, kVec>::kBytes> * kBatch<kOps> * kThreads * Vec<T, kVec>::kBytes;
}

// Tasks in one order (group_norm_tasks.h), dealt out to the blocks in turn.  A block takes its tasks in that order, so
// whatever one waits for is done or being done by a block that waits for less; `lag` is such that it is nearly always
// done, and that what is read again is in L2.
struct Stream {
  Params a;
  Order order;
  uint32_t* counts;   // of each image's runs whose moments are there, then one for each image: 1 when they are merged
  float* means;       // backward: the images' two means of each group
  uint32_t* err;
};

// Waits until a count has been reached; a wait that runs out is reported.  (A block that takes an image's moments again
// needs 4 ns for each of its values.)
__device__ __forceinline__ void wait_for(const Stream& f, const uint32_t* count, uint32_t n) {
  if (ld_acquire_gpu(count) >= n) return;
  const uint64_t t0 = globaltimer_ns(), limit = kWaitLimitNs + 32 * (uint64_t)f.a.pixels * f.a.channels;
  while (ld_acquire_gpu(count) < n) {
    if (globaltimer_ns() - t0 > limit) {
      report_error(f.err, kErrWaitOperand);
      return;
    }
    __nanosleep(100);
  }
}
// After a barrier of the block: what it has written is there for those who see the count.
__device__ __forceinline__ void tell(uint32_t* count) {
  if (threadIdx.x == 0) {
    __threadfence();
    atomicAdd(count, 1u);
  }
}

// The image's moments (backward: means) from its runs'.  What other blocks have written comes through L2, kFew of a lane's
// values at a time.  Whether a group of this thread has lost its squares.
template <bool kBack>
__device__ __forceinline__ bool merge_runs(const Params& a, Team team, const float2* part, float* mean, float* second) {
  constexpr int kFew = kBack ? 8 : 16;
  const int lanes = team.lanes(), sub = team.sub();
  const float total = (float)a.pixels * (float)a.per;
  bool any = false;
  for (int first = 0; first < a.groups; first += team.teams()) {
    const int g = first + team.first();
    const float2* m = part + min(g, a.groups - 1);
    float n = 0.f, s = 0.f, q = 0.f;   // forward: count, mean, squared deviations
    for (int r = sub; r < a.runs; r += kFew * lanes) {
      float2 v[kFew];
#pragma unroll
      for (int i = 0; i < kFew; ++i)
        if (r + i * lanes < a.runs) v[i] = __ldcg(m + (int64_t)(r + i * lanes) * a.groups);
#pragma unroll
      for (int i = 0; i < kFew; ++i) {
        if (r + i * lanes >= a.runs) continue;
        if constexpr (kBack) s += v[i].x, q += v[i].y;
        else merge_moments(n, s, q, (float)run_length(a, r + i * lanes) * (float)a.per, v[i].x, v[i].y);
      }
    }
    if constexpr (kBack) {
      s = team.sum(s) / total;
      q = team.sum(q) / total;
    } else {
      for (int o = 1; o < lanes; o *= 2) {
        const float n2 = __shfl_xor_sync(0xffffffffu, n, o), s2 = __shfl_xor_sync(0xffffffffu, s, o), q2 = __shfl_xor_sync(0xffffffffu, q, o);
        // the lower lane's first, so that both get the same
        if (sub & o) {
          float n1 = n2, s1 = s2, q1 = q2;
          merge_moments(n1, s1, q1, n, s, q);
          n = n1, s = s1, q = q1;
        } else {
          merge_moments(n, s, q, n2, s2, q2);
        }
      }
      q = rstd_of(q, total, a.eps);
      any |= lost(q);
    }
    if (g < a.groups && sub == 0) mean[g] = s, second[g] = q;
  }
  return any;
}

template <typename T, int kVec, bool kBack>
__global__ void __launch_bounds__(kThreads, kResident<1 + kBack>) stream_kernel(const __grid_constant__ Stream f) {
  extern __shared__ __align__(16) uint8_t smem[];
  const Params& a = f.a;
  const Shared<T, kVec> s(a, smem);
  const Lay l = Lay::of<kVec>(a.channels);
  const Teams teams = Teams::of(a, l);
  s.set_groups(a);
  // the block's own sums of the parameters' gradients, behind the rings
  float* own = reinterpret_cast<float*>(s.kept + ring_bytes<T, kVec, 1 + kBack>());
  if constexpr (kBack)
    for (int c = threadIdx.x; c < 2 * a.channels; c += kThreads) own[c] = 0.f;
  __syncthreads();
  const uint32_t runs = a.runs, all = Task::total(f.order.images, runs);
  for (uint32_t i = blockIdx.x; i < all; i += gridDim.x) {
    const Task task = Task::of(f.order, i);
    const uint32_t image = task.image;
    const int run = (int)task.run, n = run_length(a, run);
    const int64_t begin = run_begin(a, run), at = (int64_t)image * a.groups;
    const T* x = static_cast<const T*>(a.x) + image * a.x_stride[0] + begin * a.x_stride[1];
    const T* dy = kBack ? static_cast<const T*>(a.dy) + image * a.dy_stride[0] + begin * a.dy_stride[1] : nullptr;
    float2* part = reinterpret_cast<float2*>(a.group_part) + at * runs;
    const float *mean = a.mean + at, *rstd = a.rstd + at;
    if (task.kind == kMoments) {
      [[maybe_unused]] bool far = false;
      if constexpr (kBack) {
        far = sums<T, kVec>(a, l, s, x, dy, n, rstd, [&] {
          __syncthreads();   // the task before may have its coefficients yet to read
          return __syncthreads_or(s.set_channels(a, mean, rstd)) != 0;
        });
      } else {
        moments<T, kVec>(a, l, x, n, s.table, s.kept);
      }
      __syncthreads();
      if constexpr (kBack) channel_sums<kVec>(a, l, teams.channels, s.table, s.group, rstd, far);
      else channel_moments<kVec>(a, l, teams.channels, n, s.table);
      __syncthreads();
      if constexpr (kBack) {
        for (int c = threadIdx.x; c < a.channels; c += kThreads) {
          own[c] += s.table[kTable<kVec> + c];
          own[a.channels + c] += s.table[c];
        }
        group_sums<kVec>(a, teams.groups, s.table, part + run * a.groups);
      } else {
        group_moments<kVec>(a, teams.groups, n, s.table, part + run * a.groups);
      }
      __syncthreads();
      tell(f.counts + image);
    } else if (__builtin_expect(task.kind == kMerge, 0)) {
      wait_for(f, f.counts + image, runs);
      if constexpr (kBack) {
        merge_runs<true>(a, teams.runs, part, f.means + 2 * at, f.means + 2 * at + a.groups);
        __syncthreads();
      } else if (__builtin_expect(__syncthreads_or(merge_runs<false>(a, teams.runs, part, a.mean + at, a.rstd + at)), 0)) {
#pragma unroll 1
        for (int g = 0; g < a.groups; ++g)
          if (lost(rstd[g]))
            far_moments<kThreads / 32>(x + g * a.per, a.x_stride[1], a.pixels, a.per, a.eps, reinterpret_cast<double*>(s.table), a.mean + at + g,
                                       a.rstd + at + g);
        __syncthreads();
      }
      tell(f.counts + f.order.images + image);
    } else {
      auto ready = [&] {
        wait_for(f, f.counts + f.order.images + image, 1);
        __syncthreads();   // the task before may have its coefficients yet to read
        // what another block has written comes through L2
        const float *first = kBack ? f.means + 2 * at : mean, *second = kBack ? f.means + 2 * at + a.groups : rstd;
        for (int g = threadIdx.x; g < a.groups; g += kThreads) s.stat[g] = __ldcg(first + g), s.stat[a.groups + g] = __ldcg(second + g);
        __syncthreads();
        bool far;
        if constexpr (kBack) {
          far = s.set_channels(a, mean, rstd);
          s.set_gradient(a, rstd);
        } else {
          far = s.set_channels(a, s.stat, s.stat + a.groups);
        }
        return __syncthreads_or(far) != 0;
      };
      T* y = static_cast<T*>(a.y) + image * a.y_stride[0] + begin * a.y_stride[1];
      if constexpr (kBack) gradient<T, kVec, false>(a, l, s, x, dy, y, n, rstd, ready);
      else normalise<T, kVec, false>(a, l, s, x, y, n, ready);
    }
  }
  __syncthreads();
  if constexpr (kBack) {
    if (a.gamma)
      for (int c = threadIdx.x; c < 2 * a.channels; c += kThreads) a.part[2 * (int64_t)blockIdx.x * a.channels + c] = own[c];
  }
}

// ---------------------------------------------------------------- more channels than a block has columns for

// Pixels of more than 256 vectors (2048 channels of 16 bits; 256 where they do not divide into vectors): moments (sums) of
// every channel of every run, [image][run][2][channels]; the images' groups from them; the results, which read x again.
template <typename T, int kVec, bool kBack>
__global__ void __launch_bounds__(kThreads) wide_sums_kernel(const __grid_constant__ Params a) {
  let_next_kernel_start();
  using V = Vec<T, kVec>;
  const int run = blockIdx.x % a.runs, n = run_length(a, run);
  const int64_t image = blockIdx.x / a.runs, begin = run_begin(a, run);
  float* part = a.part + 2 * (int64_t)blockIdx.x * a.channels;
  for (int col = threadIdx.x; col < a.channels / kVec; col += kThreads) {
    const T* x = static_cast<const T*>(a.x) + image * a.x_stride[0] + begin * a.x_stride[1] + (int64_t)col * kVec;
    const T* dy = kBack ? static_cast<const T*>(a.dy) + image * a.dy_stride[0] + begin * a.dy_stride[1] + (int64_t)col * kVec : nullptr;
    float2 mean[V::kPairs], scale[V::kPairs], shift[V::kPairs], s[V::kPairs], q[V::kPairs];
    [[maybe_unused]] float rstd[kVec];
    bool far = false;
    V v;
    [[maybe_unused]] V u;
    v.load(reinterpret_cast<const uint8_t*>(x));
    v.get(mean);   // forward: the first value
#pragma unroll
    for (int i = 0; i < V::kPairs; ++i) s[i] = q[i] = make_float2(0.f, 0.f);
    if constexpr (kBack) {
      float m[2 * V::kPairs] = {}, c[2 * V::kPairs] = {}, h[2 * V::kPairs] = {};
#pragma unroll
      for (int i = 0; i < kVec; ++i) {
        const int64_t ch = col * kVec + i, g = image * a.groups + ch / a.per;
        m[i] = a.mean[g];
        rstd[i] = a.rstd[g];
        far |= is_far(rstd[i]);
        c[i] = a.gamma ? rstd[i] * a.gamma[ch] : rstd[i];
        h[i] = a.gamma ? a.beta[ch] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < V::kPairs; ++i)
        mean[i] = make_float2(m[2 * i], m[2 * i + 1]), scale[i] = make_float2(c[2 * i], c[2 * i + 1]), shift[i] = make_float2(h[2 * i], h[2 * i + 1]);
    }
    if (kBack && __builtin_expect(far, 0)) {
#pragma unroll 1
      for (int i = 0; i < kVec; ++i) {
        const int ch = col * kVec + i;
        const Far w(a, ch, a.mean[image * a.groups + ch / a.per], a.rstd[image * a.groups + ch / a.per]);
        float sum = 0.f, sum_x = 0.f;
#pragma unroll 1
        for (int p = 0; p < n; ++p) {
          const float value = to_f(x[p * a.x_stride[1] + i]), g = w.slope(value, to_f(dy[p * a.dy_stride[1] + i]), a.act);
          sum += g;
          sum_x = fmaf(g, w.distance(value), sum_x);
        }
        part[ch] = sum_x * w.rest;
        part[a.channels + ch] = sum;
      }
      continue;
    }
    by_act(a.act, [&](auto act) {
#pragma unroll 4
      for (int p = 0; p < n; ++p) {
        float2 f[V::kPairs];
        [[maybe_unused]] float2 up[V::kPairs];
        v.load(reinterpret_cast<const uint8_t*>(x + p * a.x_stride[1]));
        v.get(f);
        if constexpr (kBack) {
          u.load(reinterpret_cast<const uint8_t*>(dy + p * a.dy_stride[1]));
          u.get(up);
        }
#pragma unroll
        for (int i = 0; i < V::kPairs; ++i) {
          const float2 d = sub(f[i], mean[i]);
          float2 g = d;
          if constexpr (kBack) {
            const float2 z = fma(d, scale[i], shift[i]);
            g = make_float2(act_slope<decltype(act)::value>(z.x, up[i].x), act_slope<decltype(act)::value>(z.y, up[i].y));
          }
          s[i] = add(s[i], g);
          q[i] = fma(g, d, q[i]);
        }
      }
    });
    const float inv = 1.f / (float)n;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const float si = i & 1 ? s[i / 2].y : s[i / 2].x, qi = i & 1 ? q[i / 2].y : q[i / 2].x;
      const int c = col * kVec + i;
      part[c] = kBack ? qi * rstd[i] : (i & 1 ? mean[i / 2].y : mean[i / 2].x) + si * inv;
      part[a.channels + c] = kBack ? si : qi - si * (si * inv);
    }
  }
}

// A block for each group of an image; kFew moments of a thread are on their way at a time (3 of 90x100x333 f32, one group:
// forward with one at a time and 256 threads 179 us).
constexpr int kMergeThreads = 1024;
template <typename T, bool kBack>
__global__ void __launch_bounds__(kMergeThreads) wide_merge_kernel(const __grid_constant__ Params a, float* means) {
  constexpr int kFew = 8;
  __shared__ float3 sets[kMergeThreads / 32];
  wait_for_kernel_ahead();
  let_next_kernel_start();
  const int64_t image = blockIdx.x / a.groups;
  const int c0 = blockIdx.x % a.groups * a.per;
  const float total = (float)a.pixels * (float)a.per;
  float n = 0.f, s = 0.f, q = 0.f;
  const float* part = a.part + 2 * image * a.runs * a.channels + c0;
  const int all = a.runs * a.per;
  for (int e = threadIdx.x; e < all; e += kFew * kMergeThreads) {
    float first[kFew], second[kFew];
#pragma unroll
    for (int i = 0; i < kFew; ++i) {
      const int at = min(e + i * kMergeThreads, all - 1), r = at / a.per, c = at - r * a.per;
      first[i] = part[2 * (int64_t)r * a.channels + c];
      second[i] = part[(2 * (int64_t)r + 1) * a.channels + c];
    }
#pragma unroll
    for (int i = 0; i < kFew; ++i) {
      const int at = e + i * kMergeThreads, r = at / a.per;
      if (at >= all) continue;
      if constexpr (kBack) {
        const float w = a.gamma ? a.gamma[c0 + at - r * a.per] : 1.f;
        s = fmaf(w, second[i], s);
        q = fmaf(w, first[i], q);
      } else {
        merge_moments(n, s, q, (float)run_length(a, r), first[i], second[i]);
      }
    }
  }
  auto merge = [&](float n2, float s2, float q2) {
    if constexpr (kBack) s += s2, q += q2;
    else merge_moments(n, s, q, n2, s2, q2);
  };
  for (int o = 1; o < 32; o *= 2) {   // the lower lane's first; the first lane's is the warp's
    const float n2 = __shfl_down_sync(0xffffffffu, n, o), s2 = __shfl_down_sync(0xffffffffu, s, o), q2 = __shfl_down_sync(0xffffffffu, q, o);
    merge(n2, s2, q2);
  }
  if ((threadIdx.x & 31) == 0) sets[threadIdx.x >> 5] = make_float3(n, s, q);
  __syncthreads();
  if constexpr (kBack) {
    if (threadIdx.x) return;
    for (int w = 1; w < kMergeThreads / 32; ++w) merge(sets[w].x, sets[w].y, sets[w].z);
    means[2 * image * a.groups + blockIdx.x % a.groups] = s / total;
    means[(2 * image + 1) * a.groups + blockIdx.x % a.groups] = q / total;
  } else {
    __shared__ bool again;
    __shared__ double sums[kMergeThreads / 32];
    if (threadIdx.x == 0) {
      for (int w = 1; w < kMergeThreads / 32; ++w) merge(sets[w].x, sets[w].y, sets[w].z);
      const float rstd = rstd_of(q, total, a.eps);
      a.mean[blockIdx.x] = s;
      a.rstd[blockIdx.x] = rstd;
      again = lost(rstd);
    }
    __syncthreads();
    if (again)
      far_moments<kMergeThreads / 32>(static_cast<const T*>(a.x) + image * a.x_stride[0] + c0, a.x_stride[1], a.pixels, a.per, a.eps, sums,
                                      a.mean + blockIdx.x, a.rstd + blockIdx.x);
  }
}

template <typename T, int kVec, bool kBack>
__global__ void __launch_bounds__(kThreads) wide_result_kernel(const __grid_constant__ Params a, const float* means) {
  using V = Vec<T, kVec>;
  const int run = blockIdx.x % a.runs, n = run_length(a, run);
  const int64_t image = blockIdx.x / a.runs, begin = run_begin(a, run);
  wait_for_kernel_ahead();
  let_next_kernel_start();
  for (int col = threadIdx.x; col < a.channels / kVec; col += kThreads) {
    const T* x = static_cast<const T*>(a.x) + image * a.x_stride[0] + begin * a.x_stride[1] + (int64_t)col * kVec;
    const T* dy = kBack ? static_cast<const T*>(a.dy) + image * a.dy_stride[0] + begin * a.dy_stride[1] + (int64_t)col * kVec : nullptr;
    T* y = static_cast<T*>(a.y) + image * a.y_stride[0] + begin * a.y_stride[1] + (int64_t)col * kVec;
    float mean[2 * V::kPairs] = {}, scale[2 * V::kPairs] = {}, shift[2 * V::kPairs] = {}, m[2 * V::kPairs] = {}, mx[2 * V::kPairs] = {};
    bool far = false;
#pragma unroll
    for (int i = 0; i < kVec; ++i) {
      const int ch = col * kVec + i, group = ch / a.per;
      const float rstd = a.rstd[image * a.groups + group];
      far |= is_far(rstd);
      mean[i] = a.mean[image * a.groups + group];
      scale[i] = a.gamma ? rstd * a.gamma[ch] : rstd;
      shift[i] = a.gamma ? a.beta[ch] : 0.f;
      if constexpr (kBack) {
        m[i] = -rstd * means[2 * image * a.groups + group];
        mx[i] = -rstd * rstd * means[(2 * image + 1) * a.groups + group];
      }
    }
    if (__builtin_expect(far, 0)) {
#pragma unroll 1
      for (int i = 0; i < kVec; ++i) {
        const int ch = col * kVec + i, group = ch / a.per;
        const float rstd = a.rstd[image * a.groups + group];
        const Far w(a, ch, a.mean[image * a.groups + group], rstd);
#pragma unroll 1
        for (int p = 0; p < n; ++p) {
          const float value = to_f(x[p * a.x_stride[1] + i]);
          float v;
          if constexpr (kBack)
            v = w.gradient(value, to_f(dy[p * a.dy_stride[1] + i]), a.act, rstd, means[2 * image * a.groups + group],
                           means[(2 * image + 1) * a.groups + group]);
          else
            v = w.result(value, a.act);
          y[p * a.y_stride[1] + i] = from_f<T>(v);
        }
      }
      continue;
    }
    by_act(a.act, [&](auto act) {
#pragma unroll 4
      for (int p = 0; p < n; ++p) {
        V v;
        [[maybe_unused]] V u;
        float2 f[V::kPairs];
        [[maybe_unused]] float2 up[V::kPairs];
        v.load(reinterpret_cast<const uint8_t*>(x + p * a.x_stride[1]));
        v.get(f);
        if constexpr (kBack) {
          u.load(reinterpret_cast<const uint8_t*>(dy + p * a.dy_stride[1]));
          u.get(up);
        }
        auto of = [&](float value, float upper, int i) {
          const float d = value - mean[i], z = fmaf(d, scale[i], shift[i]);
          if constexpr (kBack) return fmaf(act_slope<decltype(act)::value>(z, upper), scale[i], fmaf(d, mx[i], m[i]));
          else return act_of<decltype(act)::value>(z);
        };
#pragma unroll
        for (int i = 0; i < V::kPairs; ++i) f[i] = make_float2(of(f[i].x, kBack ? up[i].x : 0.f, 2 * i), of(f[i].y, kBack ? up[i].y : 0.f, 2 * i + 1));
        v.set(f);
        v.store(reinterpret_cast<uint8_t*>(y + p * a.y_stride[1]));
      }
    });
  }
}

// dgamma and dbeta: `rows` rows of [dgamma's channels][dbeta's], added up by 32 rows of threads that take turns, then
// in their order.
__global__ void __launch_bounds__(1024) parameters_kernel(const float* part, int64_t rows, int channels, float* dgamma, float* dbeta) {
  __shared__ float sum[32][33];
  const int lane = threadIdx.x & 31, row = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  wait_for_kernel_ahead();
  if (c < 2 * channels) {
#pragma unroll 8
    for (int64_t r = row; r < rows; r += 32) s += part[r * 2 * channels + c];
  }
  sum[row][lane] = s;
  __syncthreads();
  // a warp for each channel now
  s = warp_reduce<Sum>(sum[lane][row]);
  const int mine = blockIdx.x * 32 + row;
  if (lane || mine >= 2 * channels) return;
  if (mine < channels) dgamma[mine] = s;
  else dbeta[mine - channels] = s;
}

// ---------------------------------------------------------------- host side

// How a call is laid out.  cluster: runs is a cluster's blocks, one to a run; else the runs of an image, tasks of
// a grid of at most kStreamBlocks.
struct Plan {
  bool cluster;
  int runs;
  int slices;       // of the channels, blocks of their own (with one run)
  int64_t lag;
  int64_t budget;   // bytes of shared memory for a block
};
constexpr int64_t kStreamBlocks = 3 * 192;   // of a stream's grid, at the most
constexpr int64_t kRunBytes = 192 * 1024, kShortRun = 32 * 1024, kMostRuns = 1024;

// Shared memory beside the kept pixels, with the widest vectors that a type has.
int64_t table_bytes(const cbr_group_norm_desc_t& d) {
  return shared_bytes(kThreads * (d.dtype == CBR_F32 ? 4 : 8), d.channels, d.groups);
}

// Runs of an image whose channels are more than a block's columns, and the floats of their moments and means.
int64_t wide_runs(const cbr_group_norm_desc_t& d) {
  return std::max<int64_t>(1, std::min<int64_t>(d.pixels, (4 * kSms + d.images - 1) / std::max<int64_t>(d.images, 1)));
}
size_t wide_floats(const cbr_group_norm_desc_t& d) {
  return d.channels > kThreads ? (size_t)d.images * 2 * ((size_t)wide_runs(d) * d.channels + d.groups) : 0;
}

Plan plan_of(const cbr_group_norm_desc_t& d, bool backward) {
  Plan p{};
  if (d.channels > kThreads * (d.dtype == CBR_F32 ? 4 : 8)) {
    p.cluster = true;   // not used: see wide_runs()
    p.runs = p.slices = 1;
    return p;
  }
  const int64_t table = table_bytes(d), images = std::max<int64_t>(d.images, 1);
  // two blocks to an SM, so that one loads while the other stores; wide tables leave room for one
  p.budget = table + 8 * d.channels <= 64 * 1024 ? 112 * 1024 : 226 * 1024;
  const int64_t elt = d.dtype == CBR_F32 ? 4 : 2, pixel = d.channels * elt * (backward ? 2 : 1), image = d.pixels * pixel;
  const int64_t room = p.budget - table;
  p.slices = 1;
  // A small map of few images: slices of whole groups need no exchange.  Their pixels are at least 64 bytes wide and
  // whole vectors, and a block has at most 32 KB, which it reads in one go.
  for (int s = d.groups; s > 1 && images < kSms; --s) {
    const int64_t width = d.channels / s * elt;
    if (d.groups % s || width < 64 || width % 16 || images * s > 2 * kSms) continue;
    if (image / s <= 32 * 1024) {
      p.cluster = true;
      p.runs = 1;
      p.slices = s;
      return p;
    }
    break;   // fewer slices are larger yet
  }
  // Images that a cluster holds go to clusters (256 of 56x56x64 f16 forward: 58 us, as a stream 76); the backward of many that
  // take wide ones goes as well as a stream (256 of 56x56x64 f16, nine blocks each: 108.7 and 107.7 us; 256 of 28x28x256: 117
  // and 108).
  int64_t need = std::max<int64_t>(1, (image + room - 1) / room);
  p.cluster = need <= kMaxCluster && (!backward || need <= 8 || images * need <= 8 * kSms) && (d.pixels + need - 1) / need * pixel <= room;
  if (p.cluster) {
    // more blocks while SMs are without one, and a run keeps a few KB
    while (2 * need <= kMaxCluster && images * need <= kSms && image / (2 * need) >= 4096) need *= 2;
    p.runs = (int)need;
    return p;
  }
  // Runs of 192 KB, whose reading a run's fixed cost (the merges, a few us) is small beside; shorter ones where that
  // leaves blocks without one (32 of 112x112x64 f16: forward in four runs a block 57 us, in one 36; backward in four
  // and two 66 and 61).
  const int64_t blocks = kSms * (backward ? kResident<2> : kResident<1>);
  const int64_t run = std::min(kRunBytes, std::max(kShortRun, image * images / ((backward ? 4 : 2) * kSms)));
  p.runs = (int)std::max<int64_t>(1, std::min<int64_t>(std::min<int64_t>(d.pixels, kMostRuns), (image + run - 1) / run));
  // a result is this many images behind: the tasks between are at least those in flight
  p.lag = std::min<int64_t>(images, (blocks + 2 * p.runs - 1) / (2 * p.runs) + 1);
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
  a.all_channels = d.channels;
  a.all_groups = d.groups;
  a.channels = d.channels / plan.slices;
  a.groups = d.groups / plan.slices;
  a.per = d.channels / d.groups;
  a.act = d.act;
  a.runs = plan.runs;
  a.base = d.pixels / plan.runs;
  a.extra = (int)(d.pixels % plan.runs);
  a.eps = d.eps;
  if (d.images > 0x7fffffff / (2 * plan.runs + 1) || d.images > 0x7fffffff / d.groups) return CBR_ERR_UNSUPPORTED;
  a.part = g.part;
  const int64_t fixed = shared_bytes(kTable<kVec>, a.channels, a.groups);
  const int64_t pixel = (int64_t)a.channels * sizeof(T) * (backward ? 2 : 1);
  const int64_t longest = (d.pixels + plan.runs - 1) / plan.runs;
  int64_t rows = d.images;
  if (d.channels / kVec > kThreads) {
    a.channels = d.channels;
    a.groups = d.groups;
    a.runs = (int)wide_runs(d);
    a.base = d.pixels / a.runs;
    a.extra = (int)(d.pixels % a.runs);
    rows = d.images * a.runs;
    float* means = a.part + 2 * rows * d.channels;
    const unsigned blocks = (unsigned)rows, groups = (unsigned)(d.images * d.groups);
    if (backward) {
      wide_sums_kernel<T, kVec, true><<<blocks, kThreads, 0, st>>>(a);
      if (!launch_behind(&wide_merge_kernel<T, true>, dim3(groups), kMergeThreads, 0, st, a, means) ||
          !launch_behind(&wide_result_kernel<T, kVec, true>, dim3(blocks), kThreads, 0, st, a, means))
        return CBR_ERR_CUDA;
    } else {
      wide_sums_kernel<T, kVec, false><<<blocks, kThreads, 0, st>>>(a);
      if (!launch_behind(&wide_merge_kernel<T, false>, dim3(groups), kMergeThreads, 0, st, a, means) ||
          !launch_behind(&wide_result_kernel<T, kVec, false>, dim3(blocks), kThreads, 0, st, a, means))
        return CBR_ERR_CUDA;
    }
  } else if (plan.cluster) {
    a.keep = (int)longest;
    const auto kern = backward ? &cluster_backward_kernel<T, kVec> : &cluster_forward_kernel<T, kVec>;
    if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), 227 * 1024)) return CBR_ERR_CUDA;
    if (plan.runs > 8 && !allow_wide_cluster(reinterpret_cast<const void*>(kern))) return CBR_ERR_CUDA;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(d.images * plan.runs), (unsigned)plan.slices);
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
    Stream f{};
    const int64_t own = backward ? 8 * (int64_t)a.channels : 0;
    // [groups' moments of every run][the images' means][parameters' sums of every block][counts]
    a.group_part = g.part;
    f.means = a.group_part + 2 * d.images * plan.runs * a.groups;
    a.part = f.means + (backward ? 2 * d.images * a.groups : 0);
    f.counts = reinterpret_cast<uint32_t*>(a.part + (backward ? 2 * kStreamBlocks * a.channels : 0));
    f.a = a;
    f.order = Order{(uint32_t)d.images, (uint32_t)plan.runs, (uint32_t)(plan.lag + 1) / 2, (uint32_t)plan.lag};
    f.err = g.err;
    if (cudaMemsetAsync(f.counts, 0, (size_t)d.images * 8, st) != cudaSuccess) return CBR_ERR_CUDA;
    const auto kern = backward ? &stream_kernel<T, kVec, true> : &stream_kernel<T, kVec, false>;
    const int smem = (int)(fixed + (backward ? ring_bytes<T, kVec, 2>() : ring_bytes<T, kVec, 1>()) + own);
    if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), 227 * 1024)) return CBR_ERR_CUDA;
    const int fit = blocks_that_fit(reinterpret_cast<const void*>(kern), kThreads, smem);
    if (fit < 1) return CBR_ERR_CUDA;
    rows = std::min<int64_t>(std::min<int64_t>(kStreamBlocks, (int64_t)fit * g.num_sms), (int64_t)Task::total((uint32_t)d.images, (uint32_t)plan.runs));
    // blocks wait for one another's runs: all of them have to be there at once
    void* args[] = {&f};
    if (cudaLaunchCooperativeKernel(reinterpret_cast<const void*>(kern), dim3((unsigned)rows), dim3(kThreads), args, (size_t)smem, st) !=
        cudaSuccess) {
      cudaGetLastError();
      return CBR_ERR_CUDA;
    }
  }
  if (backward && g.gamma &&
      !launch_behind(&parameters_kernel, dim3((unsigned)(2 * d.channels + 31) / 32), 1024, 0, st, a.part, rows, (int)d.channels, g.dgamma, g.dbeta))
    return CBR_ERR_CUDA;
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
  // The backward of 8 channels a thread does not fit the registers of three blocks to an SM (138 us, and 107 with 8-byte
  // vectors, at 256x56x56x64 f16); it is left to pixels with more vectors than a block has threads.
  if constexpr (sizeof(T) == 2)
    if ((!backward || d.channels > 4 * kThreads) && fits(8)) return launch<T, 8>(g, backward, st);
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
  return std::max(gn::wide_floats(d), p.cluster ? 0 : (size_t)d.images * (2 * (size_t)p.runs * d.groups + 2));
}
size_t group_norm_backward_floats(const cbr_group_norm_desc_t& d, bool parameters) {
  const gn::Plan p = gn::plan_of(d, true);
  const size_t cluster = parameters ? (size_t)d.images * 2 * d.channels : 0;
  const size_t stream = (size_t)d.images * (2 * ((size_t)p.runs + 1) * d.groups + 2) + 2 * (size_t)gn::kStreamBlocks * d.channels;
  return std::max(gn::wide_floats(d), p.cluster ? cluster : stream);
}
int launch_group_norm(const GroupNormArgs& a, cudaStream_t st) { return gn::dispatch(a, false, st); }
int launch_group_norm_backward(const GroupNormArgs& a, cudaStream_t st) { return gn::dispatch(a, true, st); }

}  // namespace cbr
