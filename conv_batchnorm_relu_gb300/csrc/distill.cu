// Distillation from a teacher's top logits, forward and backward (formulas: include/cbr.h).
//
// A row is cut into slices, one for each block of a cluster (one block where the row is short), and
// stays in shared memory between its sweeps, so the logits cross HBM once.  A block works through
// rows with three kinds of warps:
//   producer   one thread: bulk copies of coming rows into a ring of buffers, bulk copies of
//              finished gradients out of them;
//   teacher    one warp, a row ahead: the entries' ids, p and log p into shared memory;
//   consumers  take the listed logits out of the slice (each one's place holds -infinity from then
//              on, so the sweep sums unlisted words alone, with no test in it), sweep for the
//              largest logit and the sum of exponentials, exchange (largest, unlisted, listed) with
//              the cluster's other blocks, sweep again turning logits into gradients in place, and
//              put the listed words' gradients in.
// The exponent is formed from the difference to the largest logit, not from scaled logits: exact
// near the largest, and finite for rows masked with the type's lowest value.
#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>
#include <type_traits>

#include "cbr_internal.h"
#include "common.cuh"
#include "token_ops.cuh"

namespace cbr {
namespace {

using namespace tok;

enum Mode { kLoss, kBoth, kGradient };

constexpr int kMaxWarps = 8;        // consumers
constexpr int kMaxBuffers = 4;
constexpr int kMaxCluster = 8;
constexpr int kRepeated = 1 << 30;  // in an entry's id: the same id was listed before

struct Plan {
  int slices;       // of a row: the cluster's blocks (kGradient: independent work items)
  int width;        // elements of a slice, a multiple of 128
  int buffers;
  int buffer_bytes;
  int warps;
  int kp;           // room for entries
  int smem;
};

struct Header {
  uint64_t full[kMaxBuffers], empty[kMaxBuffers], t_full[2], t_free[2], x_full[2];
  float red[kMaxWarps][4];
  float xch[2][kMaxCluster][4];   // (largest, unlisted, listed) of each block of the cluster
  float teacher[2][8];            // mass, rest, weight, state
  int repeated;
};
enum { kMass, kRest, kWeight, kState };
enum { kDead, kEmpty, kLive };    // weight 0 (not even loaded), nothing to learn from, the rest

__device__ __forceinline__ uint32_t map_to_rank(uint32_t addr, uint32_t rank) {
  uint32_t r;
  asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(addr), "r"(rank));
  return r;
}
__device__ __forceinline__ void st_cluster(uint32_t addr, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool wait_cluster(uint32_t bar, uint32_t parity) {
  uint64_t t0 = 0;
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
    if (ok) return true;
    const uint64_t t = globaltimer_ns();
    if (!t0) t0 = t;
    if (t - t0 > kWaitLimitNs) return false;
  }
}
__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void bulk_store_1d(void* dst, uint32_t src, uint32_t bytes) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group [%0], [%1], %2;" ::"l"(dst), "r"(src), "r"(bytes) : "memory");
}

// 2^x.  With 16-bit logits results below 2^-126 are taken as 0 (below what f16 and the sums can
// show; a bf16 gradient under 2^-126 becomes 0).  32-bit gradients keep their subnormal range.
template <typename T>
__device__ __forceinline__ float ex2(float x) {
  float r;
  if constexpr (sizeof(T) == 2) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  else asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// The logits of 16 bytes.
template <typename T>
struct Chunk {
  static constexpr int n = 16 / sizeof(T);
  float v[n];
  __device__ __forceinline__ Chunk(uint4 w) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) {
        v[i] = __uint_as_float(u[i]);
      } else {
        const float2 f = unpack2<std::is_same_v<T, __nv_bfloat16>>(u[i]);
        v[2 * i] = f.x;
        v[2 * i + 1] = f.y;
      }
    }
  }
  __device__ __forceinline__ uint4 packed() const {
    uint32_t u[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (sizeof(T) == 4) u[i] = __float_as_uint(v[i]);
      else u[i] = pack2<std::is_same_v<T, __nv_bfloat16>>(v[2 * i], v[2 * i + 1]);
    }
    return make_uint4(u[0], u[1], u[2], u[3]);
  }
  __device__ __forceinline__ float largest() const {
    float m = v[0];
#pragma unroll
    for (int i = 1; i < n; ++i) m = Max::of(m, v[i]);
    return m;
  }
};

// A running (largest, sum of 2^((s - largest) c)) pair, the sum in two parts.
struct Running {
  float top = -INFINITY, unlisted = 0.f, listed = 0.f;
};
template <typename T>
__device__ __forceinline__ void raise(Running& r, float m, float c) {
  if (!(m <= r.top)) {   // NaN gets in, too, and stays
    m = Max::of(m, r.top);
    const float f = r.top == -INFINITY ? 0.f : ex2<T>((r.top - m) * c);
    r.unlisted *= f;
    r.listed *= f;
    r.top = m;
    if (m != m) r.unlisted = m;
  }
}
template <typename T>
__device__ __forceinline__ Running merge_warp(Running r, float c) {
  const float m = warp_reduce<Max>(r.top);
  const float f = r.top == -INFINITY ? 0.f : ex2<T>((r.top - m) * c);
  return Running{m, warp_reduce<Sum>(r.unlisted * f), warp_reduce<Sum>(r.listed * f)};
}

// Where a slice's elements lie in a buffer: element j at lead + j, so that global and shared
// addresses agree modulo 16; chunks [c0, c1) are whole, the others hold `edge` elements.
template <typename T>
struct Slice {
  static constexpr int kN = 16 / sizeof(T);
  int n, lead, c0, c1, chunks;
  __device__ __forceinline__ Slice(const T* p, int n_) : n(n_) {
    lead = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    c0 = lead ? 1 : 0;
    c1 = max(c0, (lead + n) / kN);
    chunks = n ? (lead + n + kN - 1) / kN : 0;
  }
  __device__ __forceinline__ uint32_t whole_bytes() const { return (uint32_t)(c1 - c0) * 16u; }
  __device__ __forceinline__ bool ragged() const { return n && (c0 != 0 || c1 != chunks); }
  // Thread i of the first 2 * kN holds a place of the first or of the last chunk; -1: none.
  __device__ __forceinline__ int edge_place(int i) const {
    if (i >= 2 * kN || !n) return -1;
    if (i < kN) return c0 ? i : -1;
    if (c1 >= chunks || (chunks == 1 && c0)) return -1;
    return (chunks - 1) * kN + i - kN;
  }
};

__device__ __forceinline__ int entry_id(const DistillArgs& a, long long row, int k) {
  const long long i = row * a.d.ids_stride + k;
  const long long id = a.d.id_bytes == 8 ? static_cast<const long long*>(a.top_ids)[i]
                                         : (long long)static_cast<const int*>(a.top_ids)[i];
  return id >= 0 && id < a.d.vocab ? (int)id : -1;
}

// The teacher's distribution of a row, by one warp.
__device__ void teach(const DistillArgs& a, long long row, float inv_t, int* ids, float* p, float* lp, float* out) {
  const int lane = threadIdx.x & 31, k_n = (int)a.d.topk;
  const float w = a.row_weight ? a.row_weight[row] : 1.f;
  if (w == 0.f) {
    if (lane == 0) out[kWeight] = 0.f, out[kState] = (float)kDead;
    return;
  }
  float top = -INFINITY;
  bool any = false;
  for (int k = lane; k < k_n; k += 32) {
    const int id = entry_id(a, row, k);
    const float x = id < 0 ? -INFINITY : load_as_float(a.top_logits, a.d.top_dtype, row * a.d.top_stride + k) * inv_t;
    ids[k] = id;
    lp[k] = x;
    top = Max::of(top, x);
    any |= id >= 0;
  }
  any = __any_sync(0xffffffffu, any);
  top = warp_reduce<Max>(top);
  float norm, mass = 0.f;
  if (a.teacher_lse) {
    norm = a.teacher_lse[row];
  } else {
    any = any && top != -INFINITY;
    float s = 0.f;
    for (int k = lane; k < k_n; k += 32)
      if (ids[k] >= 0) s += expf(lp[k] - top);
    norm = top + logf(warp_reduce<Sum>(s));
  }
  for (int k = lane; k < k_n; k += 32) {
    const float l = lp[k] - norm, q = ids[k] >= 0 ? expf(l) : 0.f;
    lp[k] = l;
    p[k] = q;
    mass += q;
  }
  mass = warp_reduce<Sum>(mass);
  if (lane == 0) {
    out[kMass] = a.teacher_lse ? mass : 1.f;
    out[kRest] = a.teacher_lse ? fmaxf(0.f, 1.f - mass) : 0.f;
    out[kWeight] = w;
    out[kState] = (float)(any ? kLive : kEmpty);
  }
}

template <typename T, int kMode>
__global__ void __launch_bounds__((kMaxWarps + 2) * 32, 2)
    distill_kernel(const __grid_constant__ DistillArgs a, const __grid_constant__ Plan plan) {
  extern __shared__ __align__(128) uint8_t smem[];
  Header& h = *reinterpret_cast<Header*>(smem);
  int* const ids0 = reinterpret_cast<int*>(smem + (sizeof(Header) + 15) / 16 * 16);
  float* const p0 = reinterpret_cast<float*>(ids0 + 2 * plan.kp);
  float* const lp0 = p0 + 2 * plan.kp;
  float* const sk0 = lp0 + 2 * plan.kp;
  uint8_t* const ring = smem + plan.smem - plan.buffers * plan.buffer_bytes;
  const uint32_t bars = smem_u32(&h);
  auto bar = [&](const uint64_t* b) { return bars + (uint32_t)(reinterpret_cast<const uint8_t*>(b) - smem); };

  constexpr bool kAcross = kMode != kGradient;   // whether a row's blocks exchange their sums
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int across = kAcross ? plan.slices : 1;
  const int rank = across > 1 ? (int)(blockIdx.x % across) : 0;
  if (threadIdx.x == 0) {
    for (int i = 0; i < kMaxBuffers; ++i) {
      mbar_init(bar(&h.full[i]), 1);
      mbar_init(bar(&h.empty[i]), plan.warps);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(&h.t_full[i]), 1);
      mbar_init(bar(&h.t_free[i]), plan.warps);
      mbar_init(bar(&h.x_full[i]), across);
    }
    h.repeated = -1;
    fence_mbarrier_init();
  }
  if (across > 1) cluster_sync();
  else __syncthreads();

  // Work item i of this block: a row and a slice of it.
  const long long first = kAcross ? blockIdx.x / across : blockIdx.x;
  const long long step = kAcross ? gridDim.x / across : gridDim.x;
  const long long items = kAcross ? a.d.rows : a.d.rows * plan.slices;
  auto row_of = [&](long long i) { return kAcross ? i : i / plan.slices; };
  auto begin_of = [&](long long i) { return (kAcross ? rank : (int)(i % plan.slices)) * plan.width; };
  auto slice_n = [&](int begin) { return max(0, min(plan.width, (int)a.d.vocab - begin)); };
  auto logits_at = [&](long long row, int begin) {
    return static_cast<const T*>(a.logits) + row * a.d.logits_stride + begin;
  };
  auto grad_at = [&](long long row, int begin) { return static_cast<T*>(a.dlogits) + row * a.d.dlogits_stride + begin; };
  // A wait that runs out is reported, and its warps leave their loop; the others' waits then run out,
  // too, so that every block comes to its end.

  if (warp == plan.warps) {   // ------------------------------------------------ producer
    if (lane == 0) {
      auto load = [&](long long i, int b) {
        const long long row = row_of(i);
        const uint32_t full = bar(&h.full[b]);
        if (a.row_weight && a.row_weight[row] == 0.f) {
          mbar_arrive(full);
          return;
        }
        const int begin = begin_of(i);
        const T* src = logits_at(row, begin);
        const Slice<T> s(src, slice_n(begin));
        const uint32_t bytes = s.whole_bytes();
        if (!bytes) {
          mbar_arrive(full);
          return;
        }
        mbar_arrive_expect_tx(full, bytes);
        bulk_load_1d(smem_u32(ring + b * plan.buffer_bytes + s.c0 * 16), src - s.lead + s.c0 * Slice<T>::kN, bytes, full);
      };
      long long ahead = first;
      int loads = 0;
      for (; loads < plan.buffers && ahead < items; ++loads, ahead += step) load(ahead, loads);
      int b = 0;
      uint32_t phase = 0;
      for (long long i = first; i < items; i += step) {
        if (!mbar_wait_backoff(bar(&h.empty[b]), phase, 64)) {
          report_error(a.err, kErrWaitOperand);
          break;
        }
        if (kMode != kLoss) {
          const int begin = begin_of(i);
          const Slice<T> s(logits_at(row_of(i), begin), slice_n(begin));
          T* dst = grad_at(row_of(i), begin) - s.lead + s.c0 * Slice<T>::kN;
          if (s.whole_bytes() && (reinterpret_cast<uintptr_t>(dst) & 15) == 0) {
            bulk_store_1d(dst, smem_u32(ring + b * plan.buffer_bytes + s.c0 * 16), s.whole_bytes());
            bulk_commit_group();
            bulk_wait_group_read<0>();
          }
        }
        if (ahead < items) {
          load(ahead, b);
          ahead += step;
          ++loads;
        }
        if (++b == plan.buffers) b = 0, phase ^= 1;
      }
      bulk_wait_group<0>();
      // no copy is in flight when the block ends, also where a wait ran out (else: all are complete)
      for (int l = max(0, loads - plan.buffers); l < loads; ++l)
        if (!mbar_wait(bar(&h.full[l % plan.buffers]), (l / plan.buffers) & 1)) report_error(a.err, kErrWaitOperand);
    }
  } else if (warp == plan.warps + 1) {   // ------------------------------------ teacher
    const float inv_t = 1.f / a.d.temperature;
    int n = 0;
    for (long long i = first; i < items; i += step, ++n) {
      const int slot = n & 1;
      if (n >= 2 && !__all_sync(0xffffffffu, mbar_wait_backoff(bar(&h.t_free[slot]), ((n >> 1) & 1) ^ 1, 64))) {
        if (lane == 0) report_error(a.err, kErrWaitOperand);
        break;
      }
      teach(a, row_of(i), inv_t, ids0 + slot * plan.kp, p0 + slot * plan.kp, lp0 + slot * plan.kp, h.teacher[slot]);
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(&h.t_full[slot]));
    }
  } else {   // ---------------------------------------------------------------- consumers
    const int tid = threadIdx.x, threads = plan.warps * 32, k_n = (int)a.d.topk;
    const float inv_t = 1.f / a.d.temperature, c = inv_t * 1.4426950408889634f;
    int n = 0, b = 0, exchanges = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (long long i = first; i < items; i += step, ++n) {
      const long long row = row_of(i);
      const int begin = begin_of(i), slot = n & 1;
      const T* src = logits_at(row, begin);
      const Slice<T> s(src, slice_n(begin));
      T* const buf = reinterpret_cast<T*>(ring + b * plan.buffer_bytes);
      const uint32_t buf_at = smem_u32(buf);
      int* const ids = ids0 + slot * plan.kp;
      const float* const p = p0 + slot * plan.kp;
      const float* const lp = lp0 + slot * plan.kp;
      if (!mbar_wait(bar(&h.t_full[slot]), (n >> 1) & 1)) {
        ok = false;
        if (lane == 0) report_error(a.err, kErrWaitWeights);
      }
      const int state = (int)h.teacher[slot][kState];
      const float weight = h.teacher[slot][kWeight];
      const int place = s.edge_place(tid);
      T edge = from_f<T>(-INFINITY);
      if (state != kDead && place >= s.lead && place < s.lead + s.n) edge = src[place - s.lead];
      if (ok && !mbar_wait(bar(&h.full[b]), phase)) {
        ok = false;
        if (lane == 0) report_error(a.err, kErrWaitHalo);
      }
      if (state != kDead && place >= 0) buf[place] = edge;
      // every thread or none goes on: those of a block stay together at the barriers below
      if (!(ok = named_bar_and(1, threads, ok))) break;
      bool live = state == kLive, repeated = false;
      float top = 0.f, total = 0.f, unlisted = 0.f;
      if (kMode == kGradient) {
        top = a.stats[row * 3], total = a.stats[row * 3 + 1], unlisted = a.stats[row * 3 + 2];
        live = live && !(total == 0.f);
      }
      float* const sk = sk0 + (kAcross ? (exchanges & 1) : slot) * plan.kp;
      if (live) {
        // Take the listed logits out: the first thread to fill a place with ones has its logit (an
        // id listed again, or a NaN of all ones, finds ones), and once all have, puts -infinity there.
        Running r;
        for (int k = tid; k < k_n; k += threads) {
          const int at = ids[k] - begin;
          if (ids[k] < 0 || at < 0 || at >= s.n) continue;
          const int e = s.lead + at;
          float v;
          bool had;
          if constexpr (sizeof(T) == 4) {
            const uint32_t old = atomicExch(reinterpret_cast<uint32_t*>(buf) + e, 0xffffffffu);
            had = old == 0xffffffffu;
            v = __uint_as_float(old);
          } else {
            const int sh = (e & 1) * 16;
            const uint16_t old = (uint16_t)(atomicOr(reinterpret_cast<uint32_t*>(buf) + (e >> 1), 0xffffu << sh) >> sh);
            had = old == 0xffffu;
            T t;
            *reinterpret_cast<uint16_t*>(&t) = old;
            v = to_f(t);
          }
          if (had) {
            ids[k] |= kRepeated;
            h.repeated = n;
          } else {
            sk[k] = v;
            if (rank) st_cluster(map_to_rank(smem_u32(sk + k), 0), v);
            if (kAcross) {
              raise<T>(r, v, c);
              r.listed += r.top == -INFINITY ? 0.f : ex2<T>((v - r.top) * c);
            }
          }
        }
        named_bar_sync(1, threads);
        repeated = h.repeated == n;   // the next row's marks come after another barrier
        for (int k = tid; k < k_n; k += threads) {
          const int at = ids[k] - begin;
          if (ids[k] >= 0 && at >= 0 && at < s.n) buf[s.lead + at] = from_f<T>(-INFINITY);
        }
        if (repeated) {   // a repeated id has the logit of its first entry (or a NaN that was there)
          for (int k = tid; k < k_n; k += threads) {
            if (ids[k] < 0 || !(ids[k] & kRepeated)) continue;
            float v = __int_as_float(0x7fffffff);
            for (int j = 0; j < k_n; ++j)
              if (ids[j] == (ids[k] & ~kRepeated)) v = sk[j];
            sk[k] = v;
            if (rank) st_cluster(map_to_rank(smem_u32(sk + k), 0), v);
          }
        }
        named_bar_sync(1, threads);
        if constexpr (kAcross) {
          float base = r.top == -INFINITY ? 0.f : r.top;
          for (int q = tid; q < s.chunks; q += threads) {
            const Chunk<T> x(ld_shared_v4(buf_at + q * 16));
            const float m = x.largest();
            if (!(m <= r.top)) {
              raise<T>(r, m, c);
              base = r.top == -INFINITY ? 0.f : r.top;
            }
            float e = 0.f;
#pragma unroll
            for (int j = 0; j < Chunk<T>::n; ++j) e += ex2<T>((x.v[j] - base) * c);
            r.unlisted += e;
          }
          r = merge_warp<T>(r, c);
          if (lane == 0) h.red[warp][0] = r.top, h.red[warp][1] = r.unlisted, h.red[warp][2] = r.listed;
          named_bar_sync(1, threads);
          r = Running{};
          if (lane < plan.warps) r = Running{h.red[lane][0], h.red[lane][1], h.red[lane][2]};
          r = merge_warp<T>(r, c);
          if (across > 1) {
            const int x = exchanges & 1;
            if (warp == 0 && lane < across) {
              const uint32_t to = map_to_rank(smem_u32(h.xch[x][rank]), lane);
              st_cluster(to, r.top);
              st_cluster(to + 4, r.unlisted);
              st_cluster(to + 8, r.listed);
              arrive_cluster(map_to_rank(bar(&h.x_full[x]), lane));
            }
            if (!wait_cluster(bar(&h.x_full[x]), (exchanges >> 1) & 1)) {
              ok = false;
              if (lane == 0) report_error(a.err, kErrWaitAccum);
            }
            if (!(ok = named_bar_and(1, threads, ok))) break;
            r = Running{};
            if (lane < across) r = Running{h.xch[x][lane][0], h.xch[x][lane][1], h.xch[x][lane][2]};
            r = merge_warp<T>(r, c);
          }
          ++exchanges;
          top = r.top;
          unlisted = r.unlisted;
          total = r.unlisted + r.listed;
          live = top != -INFINITY;
        }
      }
      const float mass = h.teacher[slot][kMass], inv = 1.f / total, q_rest = unlisted * inv;
      float rest = h.teacher[slot][kRest];
      if (q_rest == 0.f) rest = 0.f;
      if (kAcross && rank == 0 && warp == plan.warps - 1) {   // the row's loss, by one warp
        float l = 0.f;
        if (live) {
          const float log_total = logf(total);
          for (int k = lane; k < k_n; k += 32)
            if (ids[k] >= 0 && !(p[k] == 0.f)) l += p[k] * (lp[k] - ((sk[k] - top) * inv_t - log_total));
          l = warp_reduce<Sum>(l);
          if (rest != 0.f) l += rest * (logf(rest) - logf(q_rest));
        }
        if (lane == 0) {
          a.loss[row] = live ? l * weight * a.d.temperature * a.d.temperature : 0.f;
          if (a.stats) {
            a.stats[row * 3] = live ? top : 0.f;
            a.stats[row * 3 + 1] = live ? total : 0.f;
            a.stats[row * 3 + 2] = live ? unlisted : 0.f;
          }
        }
      }
      if constexpr (kMode != kLoss) {
        const float scale = weight * a.d.temperature * (kMode == kGradient && a.dloss ? a.dloss[row] : 1.f);
        const float all = mass + rest;
        if (live) {
          const float coef = scale * (rest != 0.f ? all - rest / q_rest : all) * inv;
          for (int q = tid; q < s.chunks; q += threads) {
            Chunk<T> x(ld_shared_v4(buf_at + q * 16));
#pragma unroll
            for (int j = 0; j < Chunk<T>::n; ++j) x.v[j] = ex2<T>((x.v[j] - top) * c) * coef;
            st_shared_v4(buf_at + q * 16, x.packed());
          }
          named_bar_sync(1, threads);
          for (int k = tid; k < k_n; k += threads) {
            const int id = ids[k] & ~kRepeated, at = id - begin;
            if (ids[k] < 0 || at < 0 || at >= s.n) continue;
            float pk = p[k];
            if (repeated) {
              pk = 0.f;
              for (int j = 0; j < k_n; ++j)
                if (ids[j] >= 0 && (ids[j] & ~kRepeated) == id) pk += p[j];
            }
            buf[s.lead + at] = from_f<T>(scale * (ex2<T>((sk[k] - top) * c) * inv * all - pk));
          }
        } else {
          for (int q = tid; q < s.chunks; q += threads) st_shared_v4(buf_at + q * 16, make_uint4(0, 0, 0, 0));
        }
        T* dst = grad_at(row, begin);
        const bool apart = (reinterpret_cast<uintptr_t>(dst - s.lead) & 15) != 0;
        if (s.ragged() || apart) {
          named_bar_sync(1, threads);
          if (apart) {   // the gradient's rows start at other phases than the logits'
            for (int j = tid; j < s.n; j += threads) dst[j] = buf[s.lead + j];
          } else if (place >= s.lead && place < s.lead + s.n) {
            dst[place - s.lead] = buf[place];
          }
        }
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(bar(&h.empty[b]));
        mbar_arrive(bar(&h.t_free[slot]));
      }
      if (++b == plan.buffers) b = 0, phase ^= 1;
    }
  }
  // no block leaves while another may still write to its shared memory
  if (across > 1) {
    __syncwarp();
    cluster_sync();
  }
}

Plan make_plan(const DistillArgs& a, int elt, int num_sms) {
  Plan p{};
  const long long v = a.d.vocab;
  // Slices of at most 32 KB, so that two blocks with three buffers each share an SM; more slices
  // while there are rows for fewer than that many blocks and a slice keeps 2 KB.
  p.slices = 1;
  while (p.slices < kMaxCluster && (v + p.slices - 1) / p.slices * elt > 32 * 1024) p.slices *= 2;
  while (p.slices < kMaxCluster && a.d.rows * p.slices * 2 <= 2 * num_sms && v * elt / (2 * p.slices) >= 2048) p.slices *= 2;
  p.width = (int)(((v + p.slices - 1) / p.slices + 127) / 128 * 128);
  p.buffer_bytes = (p.width * elt + 32 + 127) / 128 * 128;
  p.kp = (int)((a.d.topk + 31) / 32 * 32);
  const int fixed = (int)((sizeof(Header) + 15) / 16 * 16 + (size_t)p.kp * 32 + 127) / 128 * 128;
  const int half = 113 * 1024 - fixed, whole = 226 * 1024 - fixed;
  p.buffers = half / p.buffer_bytes >= 2 ? half / p.buffer_bytes : whole / p.buffer_bytes;
  p.buffers = std::max(1, std::min(p.buffers, kMaxBuffers));
  p.smem = fixed + p.buffers * p.buffer_bytes;
  const int chunks = p.width * elt / 16;
  p.warps = std::max(1, std::min(kMaxWarps, (chunks + 63) / 64));
  return p;
}

template <typename T, int kMode>
int launch(const DistillArgs& a, int num_sms, cudaStream_t st) {
  auto kernel = distill_kernel<T, kMode>;
  constexpr bool kAcross = kMode != kGradient;
  Plan p = make_plan(a, sizeof(T), num_sms);
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kernel), 227 * 1024)) return CBR_ERR_CUDA;
  const int across = kAcross ? p.slices : 1;
  const long long items = kAcross ? a.d.rows : a.d.rows * p.slices;
  const int threads = (p.warps + 2) * 32;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = across;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  cfg.blockDim = dim3(threads);
  cfg.gridDim = dim3(across);
  cfg.dynamicSmemBytes = p.smem;
  cfg.stream = st;
  // how many clusters run at once: asked once for each launch shape
  static std::mutex mu;
  static std::map<std::tuple<int, int, int>, int> at_once;
  int clusters = 0;
  {
    std::lock_guard<std::mutex> lk(mu);
    int& n = at_once[{threads, p.smem, across}];
    if (!n && cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
      return CBR_ERR_CUDA;
    }
    clusters = n;
  }
  if (clusters < 1) return CBR_ERR_CUDA;
  cfg.gridDim = dim3((unsigned)(std::min<long long>(items, clusters) * across));
  if (cudaLaunchKernelEx(&cfg, kernel, a, p) != cudaSuccess) {
    cudaGetLastError();
    return CBR_ERR_CUDA;
  }
  return CBR_OK;
}

template <typename T>
int launch_of(const DistillArgs& a, bool backward, int num_sms, cudaStream_t st) {
  if (backward) return launch<T, kGradient>(a, num_sms, st);
  return a.dlogits ? launch<T, kBoth>(a, num_sms, st) : launch<T, kLoss>(a, num_sms, st);
}

int launch_any(const DistillArgs& a, bool backward, int num_sms, cudaStream_t st) {
  if (a.d.dtype == CBR_F32) return launch_of<float>(a, backward, num_sms, st);
  if (a.d.dtype == CBR_BF16) return launch_of<__nv_bfloat16>(a, backward, num_sms, st);
  return launch_of<__half>(a, backward, num_sms, st);
}

}  // namespace

int launch_distill(const DistillArgs& a, int num_sms, cudaStream_t st) { return launch_any(a, false, num_sms, st); }

int launch_distill_backward(const DistillArgs& a, int num_sms, cudaStream_t st) { return launch_any(a, true, num_sms, st); }

}  // namespace cbr
