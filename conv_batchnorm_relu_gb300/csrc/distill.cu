// Distillation from a teacher's top logits, forward and backward (formulas: include/cbr.h).
//
// A block takes a row (or, where rows are few, one of a cluster's slices of it) through a ring of
// shared-memory buffers: a first pass for the largest logit and the sums of exponentials, a second
// one that turns logits into gradients in place.  The ring keeps the chunks that came last, the
// second pass begins with them, and only what did not fit is fetched again, from L2; so the logits
// cross HBM once.  Warps have their own jobs and meet at barriers in shared memory, chunk by chunk:
//   loader     one thread: bulk copies of chunks into the ring;
//   consumers  both passes, each warp on its own part of every chunk.  A warp takes the listed logits
//              of its part out first (-infinity stands there from then on, so that the sweep sums
//              unlisted words alone, with no test in it) and puts the listed words' gradients in last.
//              Between the passes they merge their sums, and exchange them with the cluster;
//   storer     one thread: bulk copies of finished chunks out of the ring;
//   teachers   two warps, for every other row: some rows ahead the ids and log p of the row's entries,
//              behind the others its loss.
// Exponentials, c = log2(e) / T.  16-bit logits: 2^((s - largest) c), the difference in 32 bits by an add
// that takes the 16-bit operand as it is, which needs no instruction to convert it (conversions by shifts
// and masks kept the integer pipe busiest: 2048 rows of 32000 bf16 took 64.1 us with them, 58.4 without).
// 32-bit ones: 2^(s c - b), with b the largest logit's s c, rounded: one fused multiply-add whose product
// and difference are exact, and b itself, being the same everywhere, drops out of every quotient; where
// b is so large that its rounding would count (a row masked with -1e9 or the type's lowest value), the
// difference as for 16-bit logits.
// Measured: 4096x131072 bf16 362 us, bound by data movement (with the second pass's reload from L2; the
// kernel without its arithmetic takes as long); 2048x32000 54 us, of which a steady state at 86% of the
// copy rate, 5 us until the first chunks are there, and the last round of rows, which not every block has.
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
constexpr int kMaxBuffers = 16;
constexpr int kMaxCluster = 8;
constexpr int kFewRows = 4;         // rows of a call whose rows are each shared by a cluster (make_plan)
constexpr int kRows = 4;            // whose entries are held at once; a multiple of kTeachers
constexpr int kBatch = 4;           // 16-byte vectors that a consumer has in hand at once (2: 57 us for 55)
constexpr int kTeachers = 2;        // warps, for a row each in turn (one: 56 us for 55)
constexpr int kOthers = 2 + kTeachers;  // warps that are not consumers
constexpr int kAbsent = -(1 << 30); // the id of an absent entry

struct Plan {
  int slices;       // of a row: the cluster's blocks (kGradient: independent work items)
  int width;        // elements of a slice, a multiple of 128
  int part;         // log2 of the 16-byte vectors of a chunk that one consumer warp works on
  int warps;        // consumers; a power of two
  int buffers;      // of the ring
  int kp;           // room for entries
  int smem;
  bool ragged;      // a row may start or end inside a 16-byte vector
  float c, c_low;   // log2(e) / T, and what its rounding left: that grows with the distance from the largest logit
};

struct Header {
  // chunk by chunk: copied in; worked through; copied out
  uint64_t full[kMaxBuffers], done[kMaxBuffers], free[kMaxBuffers];
  // row by row: teacher's entries; its probabilities (kGradient: and the row's sums); no longer needed;
  // row's sums; the consumers' own sums; the cluster's sums
  uint64_t t_full[kRows], m_full[kRows], t_free[kRows], r_full[kRows], c_full[2], x_full[2];
  float red[2][kMaxWarps][4];       // (largest, unlisted, listed) of each consumer
  float xch[2][kMaxCluster][4];     // and of each block of the cluster
  float teacher[kRows][4];          // mass, rest, weight, state
  float result[kRows][4];           // of the row: largest, total, unlisted (as `dim_share` has it); live (kGradient: dloss)
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
// Bulk copies that tell L2 what to keep: the chunks that will be read again, and nothing else.
__device__ __forceinline__ uint64_t l2_keep() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ uint64_t l2_pass() {
  uint64_t p;
  asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(p));
  return p;
}
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar, uint64_t policy) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes.L2::cache_hint [%0], [%1], %2, [%3], %4;" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(src)), "r"(bytes), "r"(bar), "l"(policy)
      : "memory");
}
__device__ __forceinline__ void bulk_store(void* dst, uint32_t src, uint32_t bytes, uint64_t policy) {
  asm volatile("cp.async.bulk.global.shared::cta.bulk_group.L2::cache_hint [%0], [%1], %2, %3;" ::"l"(dst), "r"(src),
               "r"(bytes), "l"(policy)
               : "memory");
}

// 2^x.  With 16-bit logits results below 2^-126 are taken as 0: too little for a sum of exponentials
// relative to its own largest, and a bf16 gradient that small, before its scale, becomes 0.  32-bit
// gradients keep their subnormal range.  For them, too, it is the hardware's estimate: with the row's sums
// it is 1.3e-7 off the 64-bit form at 8x1000 (8.5e-8 with a full exponential).
template <typename T>
__device__ __forceinline__ float ex2(float x) {
  float r;
  if constexpr (sizeof(T) == 2) asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  else asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Two floats in one register pair, and arithmetic on both at once.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 unpair(uint64_t v) {
  float2 f;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(f.x), "=f"(f.y) : "l"(v));
  return f;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// A 16-bit logit (the lower or upper half of w) plus m.
template <typename T, bool kUpper>
__device__ __forceinline__ float plus(uint32_t w, float m) {
  float r;
  if constexpr (std::is_same_v<T, __nv_bfloat16>) {
    if constexpr (kUpper) asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tadd.rn.f32.bf16 %0, h, %2;}" : "=f"(r) : "r"(w), "f"(m));
    else asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tadd.rn.f32.bf16 %0, l, %2;}" : "=f"(r) : "r"(w), "f"(m));
  } else {
    if constexpr (kUpper) asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tadd.rn.f32.f16 %0, h, %2;}" : "=f"(r) : "r"(w), "f"(m));
    else asm("{.reg .b16 l, h;\n\tmov.b32 {l, h}, %1;\n\tadd.rn.f32.f16 %0, l, %2;}" : "=f"(r) : "r"(w), "f"(m));
  }
  return r;
}

// The exponentials of the logits of 16 bytes, in pairs.
template <typename T>
struct Chunk {
  static constexpr int kPairs = 8 / sizeof(T);
  uint64_t v[kPairs];
  // minus: -b, or (far) minus the largest logit
  __device__ __forceinline__ Chunk(uint4 w, float minus, float c, bool far) {
    const uint32_t u[4] = {w.x, w.y, w.z, w.w};
    const uint64_t mm = pair(minus, minus), cc = pair(c, c);
#pragma unroll
    for (int i = 0; i < kPairs; ++i) {
      if constexpr (sizeof(T) == 4) {
        const uint64_t x = pair(__uint_as_float(u[2 * i]), __uint_as_float(u[2 * i + 1]));
        v[i] = far ? mul2(add2(x, mm), cc) : fma2(x, cc, mm);
      } else {
        v[i] = mul2(pair(plus<T, false>(u[i], minus), plus<T, true>(u[i], minus)), cc);
      }
      const float2 f = unpair(v[i]);
      v[i] = pair(ex2<T>(f.x), ex2<T>(f.y));
    }
  }
  __device__ __forceinline__ uint4 packed() const {
    uint32_t u[4];
    if constexpr (sizeof(T) == 4) {
      const float2 a = unpair(v[0]), b = unpair(v[1]);
      return make_uint4(__float_as_uint(a.x), __float_as_uint(a.y), __float_as_uint(b.x), __float_as_uint(b.y));
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = unpair(v[i]);
        u[i] = pack2<std::is_same_v<T, __nv_bfloat16>>(f.x, f.y);
      }
      return make_uint4(u[0], u[1], u[2], u[3]);
    }
  }
};

// The exponent's b (not to be fused with what it meets: it has to be the same everywhere), and whether
// exponentials are relative to the logit itself instead: where b's rounding may pass 2^-3, so that sums
// relative to b stay within a tenth of those relative to the logit, and always for 16-bit logits, whose
// difference comes with their conversion to 32 bits.
constexpr float kFar = 4194304.f;   // 2^22
__device__ __forceinline__ float base_of(float top, float c) { return __fmul_rn(top, c); }
template <typename T>
__device__ __forceinline__ bool is_far(float top, float c) {
  return sizeof(T) == 2 || !(fabsf(base_of(top, c)) < kFar);
}
template <typename T>
__device__ __forceinline__ float minus_base(float top, float c) {
  return is_far<T>(top, c) ? -top : -base_of(top, c);
}
template <typename T>
__device__ __forceinline__ float exponential(float s, float top, float c) {
  return ex2<T>(is_far<T>(top, c) ? (s - top) * c : __fmaf_rn(s, c, -base_of(top, c)));
}
// What a sum relative to `from` is multiplied by to be relative to `to`, the larger: either may be far, and
// then the exponent is what is between a base and a logit.
template <typename T>
__device__ __forceinline__ float rebase(float from, float to, float c) {
  float e = (from - to) * c;
  if constexpr (sizeof(T) == 4) {
    const float x = base_of(from, c), y = base_of(to, c);
    const bool near_x = fabsf(x) < kFar, near_y = fabsf(y) < kFar;
    const float from_y = near_x ? __fsub_rn(x, y) : __fmaf_rn(from, c, -y);   // to near
    const float to_x = -__fmaf_rn(to, c, -x);
    e = near_y ? from_y : near_x ? to_x : e;
  }
  return from == -INFINITY ? 0.f : ex2<T>(e);
}
// The logarithm to base 2 of what a sum relative to `from` is multiplied by to be relative to the logit `to`.
template <typename T>
__device__ __forceinline__ float exponent(float from, float to, float c) {
  return is_far<T>(from, c) ? (from - to) * c : -__fmaf_rn(to, c, -base_of(from, c));
}
// 2^(top c - b), b's rounding: what a sum relative to the largest logit is multiplied by to be relative to b.
template <typename T>
__device__ __forceinline__ float rounding_of_base(float top, float c) {
  return is_far<T>(top, c) ? 1.f : exp2f(__fmaf_rn(top, c, -base_of(top, c)));
}

// The largest of `n` vectors of logits, NaN if one is.
template <typename T, int n>
__device__ __forceinline__ float largest(const uint4 (&w)[n]) {
  if constexpr (sizeof(T) == 4) {
    float m = -INFINITY;
#pragma unroll
    for (int i = 0; i < n; ++i)
      m = Max::of(m, Max::of(Max::of(__uint_as_float(w[i].x), __uint_as_float(w[i].y)),
                             Max::of(__uint_as_float(w[i].z), __uint_as_float(w[i].w))));
    return m;
  } else {
    using T2 = std::conditional_t<std::is_same_v<T, __half>, __half2, __nv_bfloat162>;
    T2 m;
#pragma unroll
    for (int i = 0; i < n; ++i) {
      const uint32_t u[4] = {w[i].x, w[i].y, w[i].z, w[i].w};
      T2 a[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) a[k] = *reinterpret_cast<const T2*>(&u[k]);
      const T2 x = __hmax2_nan(__hmax2_nan(a[0], a[1]), __hmax2_nan(a[2], a[3]));
      m = i ? __hmax2_nan(m, x) : x;
    }
    const float2 f = unpack2<std::is_same_v<T, __nv_bfloat16>>(*reinterpret_cast<uint32_t*>(&m));
    return Max::of(f.x, f.y);
  }
}

// A running (largest, sum of exponentials relative to it) pair, the sum in three parts: two of unlisted
// words, one of listed.
struct Running {
  float top = -INFINITY, listed = 0.f;
  uint64_t sum = 0;
};
template <typename T>
__device__ __forceinline__ void raise(Running& r, float m, float c) {
  if (!(m <= r.top)) {   // NaN gets in, too, and stays
    m = Max::of(m, r.top);
    const float f = rebase<T>(r.top, m, c);
    r.listed *= f;
    r.sum = m == m ? mul2(r.sum, pair(f, f)) : pair(m, m);
    r.top = m;
  }
}
// The same, merged over threads.
struct Sums {
  float top = -INFINITY, unlisted = 0.f, listed = 0.f;
};
// The lanes' sums as one.
template <typename T>
__device__ __forceinline__ Sums merge_warp(Sums r, float c) {
  const float m = warp_max(r.top);
  const float f = rebase<T>(r.top, m, c);
  uint64_t s = pair(r.unlisted * f, r.listed * f);
#pragma unroll
  for (int o = 16; o; o >>= 1) {
    const float2 v = unpair(s);
    s = add2(s, pair(__shfl_xor_sync(0xffffffffu, v.x, o), __shfl_xor_sync(0xffffffffu, v.y, o)));
  }
  const float2 v = unpair(s);
  return Sums{m, v.x, v.y};
}

// `rebase`, with the roundings of the exponent, which grow with the distance, put right: a row's unlisted
// share is a result.
template <typename T>
__device__ __forceinline__ float rebase_far_down(float from, float to, float c, float c_low) {
  const float f = rebase<T>(from, to, c);
  if (is_far<T>(from, c) != is_far<T>(to, c)) return f;
  const bool far = is_far<T>(to, c);
  const float x = far ? from : base_of(from, c), y = far ? to : base_of(to, c);
  const float d = __fsub_rn(x, y), z = __fsub_rn(d, x);
  const float low = __fsub_rn(__fsub_rn(x, __fsub_rn(d, z)), __fadd_rn(y, z));   // d + low = x - y
  const float r = far ? __fmaf_rn(d, c, -__fmul_rn(d, c)) + __fmaf_rn(d, c_low, low * c) : __fmaf_rn(from - to, c_low, low);
  return f * (1.f + (fabsf(r) < 1.f ? r * 0.69314718f : 0.f));
}
// The unlisted words' part of a row's sum, relative to the row's largest logit `top`: as it is, or, where it
// is below 2^-64 and a tail needs it, its logarithm to base 2 (negative), 0 below 2^-1074.  Words masked
// with the type's lowest value are below that as are those at -infinity, and their row has no tail.  From
// 2^-32 down it is made from a sum of its own, relative to the largest unlisted logit: this is that.
constexpr float kDim = 0x1p-32f, kFaint = 0x1p-64f, kLeast = -1074.f;
template <typename T>
__device__ __noinline__ float dim_share(Sums r, float top, float c, float c_low) {
  const float u = r.unlisted * rebase_far_down<T>(r.top, top, c, c_low);
  if (u >= kFaint) return u;
  const float l = log2f(r.unlisted) + exponent<T>(r.top, top, c);
  return l < kLeast ? 0.f : l;
}
// What the gradients of unlisted words are made with where their share is small: exponentials relative to
// `base`, near the largest of them, whose sum `sum` is near 1, and from there to the row's largest logit, `down`.
// Factors of their exponentials relative to the row's largest would pass the range of 32 bits.
constexpr float kSmall = 0x1p-20f;
struct Base {
  float base, sum, down;
};
template <typename T>
__device__ __noinline__ Base base_of_share(float share, float top, float c, float temperature) {
  Base b;
  const float l = share < 0.f ? share : log2f(share);
  b.base = __fmaf_rn(l, temperature * 0.69314718f, top);
  b.down = rebase<T>(b.base, top, c);
  b.sum = share < 0.f ? exp2f(l - exponent<T>(b.base, top, c)) : share / b.down;
  return b;
}

// Where a slice's elements lie in its chunks: element j at place lead + j, so that global and shared
// addresses agree modulo 16.  16-byte vectors [v0, v1) are whole and are copied in bulk; the first and
// the last may not be, and their elements go one by one.
template <typename T>
struct Slice {
  static constexpr int kN = 16 / sizeof(T);
  int n, lead, v0, v1, vectors;
  __device__ __forceinline__ Slice(const T* p, int n_) : n(n_) {
    lead = (int)((reinterpret_cast<uintptr_t>(p) & 15) / sizeof(T));
    v0 = lead ? 1 : 0;
    v1 = max(v0, (lead + n) / kN);
    vectors = n ? (lead + n + kN - 1) / kN : 0;
  }
  // Lane i holds a place of the first vector (0 .. kN - 1) or of the last (kN .. 2 kN - 1), or -1.
  __device__ __forceinline__ int edge_place(int i) const {
    if (i >= 2 * kN || !n) return -1;
    if (i < kN) return v0 ? i : -1;
    if (v1 >= vectors || (vectors == 1 && v0)) return -1;
    return (vectors - 1) * kN + i - kN;
  }
  __device__ __forceinline__ bool inside(int place) const { return place >= lead && place < lead + n; }
};

// What the teacher warp reads of a row, some rows ahead of its use: the entries of the first kAhead rounds
// of 32 as they are in memory.  Nothing is made of them before, so that all are in flight at once.
constexpr int kAhead = 4;
struct Fetched {
  float weight, lse, stats[3], up;   // the last two: of kGradient
  uint2 id[kAhead];
  uint32_t logit[kAhead];
};
__device__ __forceinline__ uint2 raw_id(const DistillArgs& a, long long row, int k) {
  const long long i = row * a.d.ids_stride + k;
  return a.d.id_bytes == 8 ? static_cast<const uint2*>(a.top_ids)[i]
                           : make_uint2(static_cast<const uint32_t*>(a.top_ids)[i], 0);
}
__device__ __forceinline__ long long id_of(const DistillArgs& a, uint2 raw) {
  return a.d.id_bytes == 8 ? (long long)((unsigned long long)raw.y << 32 | raw.x) : (long long)(int)raw.x;
}
__device__ __forceinline__ uint32_t raw_logit(const DistillArgs& a, long long row, int k) {
  const long long i = row * a.d.top_stride + k;
  return a.d.top_dtype == CBR_F32 ? static_cast<const uint32_t*>(a.top_logits)[i]
                                  : (uint32_t)static_cast<const uint16_t*>(a.top_logits)[i];
}
__device__ __forceinline__ float logit_of(const DistillArgs& a, uint32_t raw) {
  if (a.d.top_dtype == CBR_F32) return __uint_as_float(raw);
  if (a.d.top_dtype == CBR_BF16) return __uint_as_float(raw << 16);
  return unpack2<false>(raw).x;
}
template <int kMode>
__device__ __forceinline__ void fetch(const DistillArgs& a, long long row, Fetched& f) {
  const int lane = threadIdx.x & 31, k_n = (int)a.d.topk;
  if (a.d.id_bytes == 8) {
    const uint2* p = static_cast<const uint2*>(a.top_ids) + row * a.d.ids_stride + lane;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (lane + i * 32 < k_n) f.id[i] = p[i * 32];
  } else {
    const uint32_t* p = static_cast<const uint32_t*>(a.top_ids) + row * a.d.ids_stride + lane;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (lane + i * 32 < k_n) f.id[i].x = p[i * 32];
  }
  if (a.d.top_dtype == CBR_F32) {
    const uint32_t* p = static_cast<const uint32_t*>(a.top_logits) + row * a.d.top_stride + lane;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (lane + i * 32 < k_n) f.logit[i] = p[i * 32];
  } else {
    const uint16_t* p = static_cast<const uint16_t*>(a.top_logits) + row * a.d.top_stride + lane;
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (lane + i * 32 < k_n) f.logit[i] = p[i * 32];
  }
  f.weight = a.row_weight ? a.row_weight[row] : 1.f;
  f.lse = a.teacher_lse ? a.teacher_lse[row] : 0.f;
  if constexpr (kMode == kGradient) {
#pragma unroll
    for (int i = 0; i < 3; ++i) f.stats[i] = a.stats[row * 3 + i];
    f.up = a.dloss ? a.dloss[row] : 1.f;
  }
}

// The teacher's distribution of a row, by one warp: `begun` is called once the ids and the row's state
// are there, which is all that the first pass needs.  Without a log-sum-exp, log p is of differences from the
// largest logit, before 1 / T, so its roundings go by how far the entries are from one another, not by how
// large they are (a common offset of 300 at T = 2 cost 6e-6 of the loss when it went through t / T).  With one,
// t / T carries its rounding along: the difference is good to its own.
template <typename F>
__device__ void teach(const DistillArgs& a, long long row, const Fetched& f, float inv_t, int* ids, float* lp, float* out,
                      F begun) {
  const int lane = threadIdx.x & 31, k_n = (int)a.d.topk;
  float top = -INFINITY;
  bool any = false;
  auto put = [&](int k, uint2 raw_id, uint32_t logit) {
    const long long raw = id_of(a, raw_id);
    const int id = raw >= 0 && raw < a.d.vocab ? (int)raw : kAbsent;
    const float x = id < 0 ? -INFINITY : logit_of(a, logit);
    ids[k] = id;
    lp[k] = x;
    top = Max::of(top, x);
    any |= id >= 0;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i)
    if (lane + i * 32 < k_n) put(lane + i * 32, f.id[i], f.logit[i]);
#pragma unroll 1
  for (int k = lane + kAhead * 32; k < k_n; k += 32) put(k, raw_id(a, row, k), raw_logit(a, row, k));
  any = __any_sync(0xffffffffu, any);
  top = warp_max(top);
  if (!a.teacher_lse) any = any && top != -INFINITY;
  if (lane == 0) {
    out[kWeight] = f.weight;
    out[kState] = (float)(f.weight == 0.f ? kDead : any ? kLive : kEmpty);
  }
  __syncwarp();
  begun();
  float mass = 1.f;
  if (!a.teacher_lse) {
    float s = 0.f;
#pragma unroll 1
    for (int k = lane; k < k_n; k += 32) {
      const float l = (lp[k] - top) * inv_t;
      lp[k] = l;
      s += expf(l);   // 0 for an absent entry
    }
    const float norm = logf(warp_reduce<Sum>(s));
#pragma unroll 1
    for (int k = lane; k < k_n; k += 32) lp[k] -= norm;
  } else {
    mass = 0.f;
#pragma unroll 1
    for (int k = lane; k < k_n; k += 32) {
      const float t = lp[k], x = t * inv_t, low = __fmaf_rn(-x, a.d.temperature, t) * inv_t;
      const float l = (x - f.lse) + (fabsf(x) < INFINITY ? low : 0.f);   // an infinity leaves no remainder
      lp[k] = l;
      mass += expf(l);
    }
    mass = warp_reduce<Sum>(mass);
  }
  if (lane == 0) {
    out[kMass] = mass;
    out[kRest] = a.teacher_lse ? fmaxf(0.f, 1.f - mass) : 0.f;
  }
}

// 80 registers: two blocks of 12 warps on an SM.  Loops stay rolled but for the vectors of a batch: unrolled,
// a kernel of 100 KB of instructions (70 now) waited for them (the loss alone, 2048x32000 bf16: 34.5 us, 31.7
// rolled; 32-bit 57.5, 55.3).
template <typename T, int kMode>
__global__ void __maxnreg__(80)
    distill_kernel(const __grid_constant__ DistillArgs a, const __grid_constant__ Plan plan) {
  extern __shared__ __align__(128) uint8_t smem[];
  Header& h = *reinterpret_cast<Header*>(smem);
  int* const ids0 = reinterpret_cast<int*>(smem + (sizeof(Header) + 15) / 16 * 16);
  float* const lp0 = reinterpret_cast<float*>(ids0 + kRows * plan.kp);
  float* const sk0 = lp0 + kRows * plan.kp;                                  // the listed logits
  uint16_t* const mine0 = reinterpret_cast<uint16_t*>(sk0 + kRows * plan.kp);  // each consumer's entries
  const int buffers = plan.buffers, chunk_bits = plan.part + 31 - __clz(plan.warps);
  const int per_chunk = 1 << chunk_bits, buffer_bytes = per_chunk * 16;
  uint8_t* const ring = smem + plan.smem - buffers * buffer_bytes;
  const uint32_t bars = smem_u32(&h);
  auto bar = [&](const uint64_t* b) { return bars + (uint32_t)(reinterpret_cast<const uint8_t*>(b) - smem); };

  constexpr bool kAcross = kMode != kGradient;   // whether a row's blocks exchange their sums
  constexpr int kN = Slice<T>::kN;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int across = kAcross ? plan.slices : 1;
  const int rank = across > 1 ? (int)(blockIdx.x % across) : 0;
  if (threadIdx.x == 0) {
#pragma unroll 1
    for (int i = 0; i < buffers; ++i) {
      mbar_init(bar(&h.full[i]), 1);
      mbar_init(bar(&h.done[i]), plan.warps);
      mbar_init(bar(&h.free[i]), 1);
    }
    for (int i = 0; i < kRows; ++i) {
      mbar_init(bar(&h.t_full[i]), 1);
      mbar_init(bar(&h.m_full[i]), 1);
      mbar_init(bar(&h.t_free[i]), plan.warps);
      mbar_init(bar(&h.r_full[i]), 1);
    }
    for (int i = 0; i < 2; ++i) mbar_init(bar(&h.c_full[i]), plan.warps);
    for (int i = 0; i < 2; ++i) mbar_init(bar(&h.x_full[i]), across);
    fence_mbarrier_init();
  }
  if (across > 1) cluster_sync();
  else __syncthreads();

  // Work item i of this block: a row and a slice of it.  A cluster of several blocks has one row.
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
  auto chunks_of = [&](const Slice<T>& s) { return (s.vectors + per_chunk - 1) >> chunk_bits; };
  // Chunks of a row that do not stay for the second pass and are loaded again after the others.
  auto again_of = [&](int chunks) { return kMode == kBoth ? max(0, chunks - buffers) : 0; };
  auto dead_row = [&](long long row) { return a.row_weight && a.row_weight[row] == 0.f; };
  // A wait that runs out is reported, and its warp leaves its loop; the others' waits then run out,
  // too, so that every block comes to its end.
  bool ok = true;

  if (warp == plan.warps) {   // ------------------------------------------------ loader
    if (lane == 0) {
      const uint64_t keep = l2_keep(), pass = l2_pass();
      Turn t;
      long long loads = 0;
      bool next_dead = first < items && dead_row(row_of(first));
#pragma unroll 1
      for (long long i = first; ok && i < items; i += step) {
        const long long row = row_of(i);
        const bool dead = next_dead;
        next_dead = i + step < items && dead_row(row_of(i + step));
        if (dead && kMode == kLoss) continue;
        const int begin = begin_of(i);
        const T* src = logits_at(row, begin);
        const Slice<T> s(src, slice_n(begin));
        const int chunks = chunks_of(s), again = dead ? 0 : again_of(chunks);
#pragma unroll 1
        for (int q = 0; q < chunks + again; ++q) {
          // the buffer's last chunk was copied out before this one comes in
          if (loads >= buffers && !(ok = mbar_wait(bar(&h.free[t.slot]), t.parity ^ 1))) break;
          const int c = q < chunks ? q : q - chunks, from = max(s.v0, c << chunk_bits), to = min(s.v1, (c + 1) << chunk_bits);
          const uint32_t full = bar(&h.full[t.slot]);
          if (dead || from >= to) {
            mbar_arrive(full);
          } else {
            const uint32_t bytes = (uint32_t)(to - from) * 16u;
            mbar_arrive_expect_tx(full, bytes);
            bulk_load(smem_u32(ring + t.slot * buffer_bytes + (from - (c << chunk_bits)) * 16),
                      src - s.lead + (long long)from * kN, bytes, full, q < again ? keep : pass);
          }
          ++loads;
          t.next(buffers);
        }
      }
      // no copy is in flight when the block ends, also where a wait ran out (else: all are complete)
#pragma unroll 1
      for (long long l = max(0ll, loads - buffers); l < loads; ++l)
        ok &= mbar_wait(bar(&h.full[l % buffers]), (uint32_t)(l / buffers) & 1);
    }
  } else if (warp == plan.warps + 1) {   // ------------------------------------ storer
    if (lane == 0) {
      const uint64_t pass = l2_pass();
      Turn t;
      int leaving = -1;   // the buffer whose copy out was started last
      auto all_left = [&] {
        bulk_wait_group_read<0>();
        if (leaving >= 0) mbar_arrive(bar(&h.free[leaving]));
        leaving = -1;
      };
      bool next_dead = first < items && dead_row(row_of(first));
#pragma unroll 1
      for (long long i = first; ok && i < items; i += step) {
        const long long row = row_of(i);
        const bool dead = next_dead;
        next_dead = i + step < items && dead_row(row_of(i + step));
        if (dead && kMode == kLoss) continue;
        const int begin = begin_of(i);
        const Slice<T> s(logits_at(row, begin), slice_n(begin));
        const int chunks = chunks_of(s), again = dead ? 0 : again_of(chunks);
        const int passing = kMode == kLoss ? chunks : again, total = kMode == kLoss ? chunks : chunks + again;
        T* const dst = kMode == kLoss ? nullptr : grad_at(row, begin) - s.lead;
        const bool apart = (reinterpret_cast<uintptr_t>(dst) & 15) != 0;
#pragma unroll 1
        for (int j = 0; j < total; ++j) {
          // the buffers go back as soon as they can, unless the next chunk is there already
          if (leaving >= 0 && !mbar_test(bar(&h.done[t.slot]), t.parity)) all_left();
          if (!(ok = mbar_wait(bar(&h.done[t.slot]), t.parity))) break;
          // chunks that do not stay for the second pass, those that did, those that came again
          const int q = j < chunks ? j : j - chunks;
          const int from = max(s.v0, q << chunk_bits), to = min(s.v1, (q + 1) << chunk_bits);
          if (j >= passing && !apart && from < to) {
            bulk_store(dst + (long long)from * kN, smem_u32(ring + t.slot * buffer_bytes + (from - (q << chunk_bits)) * 16),
                       (uint32_t)(to - from) * 16u, pass);
            bulk_commit_group();
            bulk_wait_group_read<1>();
            if (leaving >= 0) mbar_arrive(bar(&h.free[leaving]));
            leaving = t.slot;
          } else {
            mbar_arrive(bar(&h.free[t.slot]));
          }
          t.next(buffers);
        }
      }
      all_left();
      bulk_wait_group<0>();
    }
  } else if (warp >= plan.warps + 2) {   // ------------------------------------ teachers
    const float inv_t = 1.f / a.d.temperature, c = plan.c;
    // The loss of the block's n-th row, once its sums are there.
    auto settle = [&](long long row, int n) {
      if (!kAcross) return true;
      const int slot = n % kRows;
      if (!__all_sync(0xffffffffu, mbar_wait(bar(&h.r_full[slot]), n / kRows & 1))) return ok = false;
      if (rank) return true;
      const int* const ids = ids0 + slot * plan.kp;
      const float* const lp = lp0 + slot * plan.kp;
      const float* const sk = sk0 + slot * plan.kp;
      const float top = h.result[slot][0], total = h.result[slot][1], part = h.result[slot][2];
      const bool live = h.result[slot][3] != 0.f;
      const float to_top = 1.f / rounding_of_base<T>(top, c);
      float l = 0.f;
      if (live) {
        const float log_total = logf(total * to_top);
        const float rest = part == 0.f ? 0.f : h.teacher[slot][kRest];
#pragma unroll 1
        for (int k = lane; k < (int)a.d.topk; k += 32) {
          const float p = ids[k] >= 0 ? expf(lp[k]) : 0.f;
          if (!(p == 0.f)) l += p * (lp[k] - ((sk[k] - top) * inv_t - log_total));
        }
        l = warp_reduce<Sum>(l);
        if (rest != 0.f) l += rest * (logf(rest) - (part < 0.f ? part * 0.69314718f - log_total : logf(part / total)));
      }
      if (lane == 0) {
        a.loss[row] = live ? l * h.teacher[slot][kWeight] * a.d.temperature * a.d.temperature : 0.f;
        if (a.stats) {
          a.stats[row * 3] = live ? top : 0.f;
          a.stats[row * 3 + 1] = live ? total * to_top : 0.f;
          a.stats[row * 3 + 2] = !live ? 0.f : part < 0.f ? part : part * to_top;
        }
      }
      return true;
    };
    const int start = warp - plan.warps - 2;
    int n = start;   // of the block's rows
    Fetched next;
    if (first + n * step < items) fetch<kMode>(a, row_of(first + n * step), next);
#pragma unroll 1
    for (long long i = first + n * step; ok && i < items; i += kTeachers * step, n += kTeachers) {
      const int slot = n % kRows;
      const Fetched now = next;
      if (i + kTeachers * step < items) fetch<kMode>(a, row_of(i + kTeachers * step), next);
      if (n >= kRows) {
        if (!settle(row_of(i - kRows * step), n - kRows)) break;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(&h.t_free[slot]), (n / kRows & 1) ^ 1));
        if (!ok) break;
      }
      teach(a, row_of(i), now, inv_t, ids0 + slot * plan.kp, lp0 + slot * plan.kp, h.teacher[slot], [&] {
        if (lane == 0) mbar_arrive(bar(&h.t_full[slot]));
      });
      if (kMode == kGradient && lane == 0) {
        const float from_top = rounding_of_base<T>(now.stats[0], c);
        h.result[slot][0] = now.stats[0];
        h.result[slot][1] = now.stats[1] * from_top;
        h.result[slot][2] = now.stats[2] < 0.f ? now.stats[2] : now.stats[2] * from_top;
        h.result[slot][3] = now.up;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(&h.m_full[slot]));
    }
#pragma unroll 1
    for (int m = max(start, n - kRows); ok && m < n; m += kTeachers) settle(row_of(first + m * step), m);
  } else {   // ---------------------------------------------------------------- consumers
    const int part = 1 << plan.part, k_n = (int)a.d.topk;
    const float c = plan.c;
    uint16_t* const mine = mine0 + warp * plan.kp;
    Turn t;
    int n = 0, merges = 0;
    auto wait = [](uint32_t b, uint32_t parity) { return (bool)__all_sync(0xffffffffu, mbar_wait(b, parity)); };
    // Part of a chunk's places that are this warp's, and whose ragged elements (the row's first and last,
    // which a bulk copy cannot move) it puts in; they are read a row ahead of their use.
    constexpr int kLog = sizeof(T) == 4 ? 2 : 3;
    auto is_mine = [&](int place) { return (place >> (plan.part + kLog) & (plan.warps - 1)) == warp; };
    auto edge_of = [&](long long i) {
      const int begin = begin_of(i);
      const T* src = logits_at(row_of(i), begin);
      const Slice<T> s(src, slice_n(begin));
      const int place = s.edge_place(lane);
      return place >= 0 && is_mine(place) && s.inside(place) ? src[place - s.lead] : from_f<T>(-INFINITY);
    };
    T next_edge = from_f<T>(0.f);
    if (plan.ragged && first < items) next_edge = edge_of(first);
#pragma unroll 1
    for (long long i = first; i < items; i += step, ++n) {
      const long long row = row_of(i);
      const int begin = begin_of(i), slot = n % kRows;
      const Slice<T> s(logits_at(row, begin), slice_n(begin));
      const int chunks = chunks_of(s);
      int edge_at = -1;
      const T edge = next_edge;
      if (plan.ragged) {
        edge_at = s.edge_place(lane);
        if (edge_at >= 0 && !is_mine(edge_at)) edge_at = -1;
        if (i + step < items) next_edge = edge_of(i + step);
      }
      if (!(ok = wait(bar(&h.t_full[slot]), n / kRows & 1))) break;
      const int state = (int)h.teacher[slot][kState];
      const int* const ids = ids0 + slot * plan.kp;
      const float* const lp = lp0 + slot * plan.kp;
      float* const sk = sk0 + slot * plan.kp;
      const int shift = s.lead - begin;   // a listed id's place: id + shift
      bool live = state == kLive;
      // This warp's entries.
      int count = 0;
      if (live) {
#pragma unroll 1
        for (int k = lane; k < plan.kp; k += 32) {
          const int place = k < k_n ? ids[k] + shift : -1;
          const bool hit = s.inside(place) && is_mine(place);
          const uint32_t mask = __ballot_sync(0xffffffffu, hit);
          if (hit) mine[count + __popc(mask & ((1u << lane) - 1))] = (uint16_t)k;
          count += __popc(mask);
        }
        __syncwarp();
      }
      const int k0 = lane < count ? mine[lane] : -1;   // the first 32 stay in registers
      const int place0 = k0 >= 0 ? ids[k0] + shift : -1;
      // Calls f(entry, place, round) for this warp's entries in chunk q.
      auto entries = [&](int q, auto f) {
        if (place0 >= 0 && place0 >> (chunk_bits + kLog) == q) f(k0, place0, 0);
#pragma unroll 1
        for (int i = lane + 32, round = 1; i < count; i += 32, ++round) {
          const int k = mine[i], place = ids[k] + shift;
          if (place >> (chunk_bits + kLog) == q) f(k, place, round);
        }
      };
      bool repeated = false;   // whether an id is among them twice, and the rounds of such entries
      uint32_t twice = 0;
      Running run;
      // Puts the ragged elements of a loaded chunk in.
      auto mend = [&](int q, T* buf) {
        if (!plan.ragged) return;
        if (edge_at >= 0 && edge_at >> (chunk_bits + kLog) == q) buf[edge_at - (q << (chunk_bits + kLog))] = edge;
        __syncwarp();
      };
      // Takes the listed logits out.  The first lane to fill a place with ones has its logit (an id
      // listed again, or a NaN of all ones, finds ones), and once all have, -infinity goes there.
      auto extract = [&](int q, T* buf) {
        const int origin = q << (chunk_bits + kLog);
        bool hit = false;
        uint32_t found = 0;
        entries(q, [&](int k, int place, int round) {
          const int e = place - origin;
          float v;
          hit = true;
          bool had;
          if constexpr (sizeof(T) == 4) {
            const uint32_t old = atomicExch(reinterpret_cast<uint32_t*>(buf) + e, 0xffffffffu);
            had = old == 0xffffffffu;
            v = __uint_as_float(old);
          } else {
            const int sh = (e & 1) * 16;
            const uint16_t old = (uint16_t)(atomicOr(reinterpret_cast<uint32_t*>(buf) + (e >> 1), 0xffffu << sh) >> sh);
            had = old == 0xffffu;
            T x;
            *reinterpret_cast<uint16_t*>(&x) = old;
            v = to_f(x);
          }
          if (had) {
            found |= 1u << round;   // at most kMaxTopk / 32 rounds
          } else {
            sk[k] = v;
            if (rank) st_cluster(map_to_rank(smem_u32(sk + k), 0), v);
          }
        });
        if (!__any_sync(0xffffffffu, hit)) return;
        __syncwarp();
        entries(q, [&](int k, int place, int round) {
            if (!(found >> round & 1)) buf[place - origin] = from_f<T>(-INFINITY);
          });
        if (__any_sync(0xffffffffu, found != 0)) {   // the logit of the id's first entry, or that NaN
          repeated = true;
          twice |= found;
          entries(q, [&](int k, int place, int round) {
            if (found >> round & 1) sk[k] = __int_as_float(0x7fffffff);
          });
          __syncwarp();
          // sk of a later entry is that NaN so far, and its first entry's is not, or both are
          entries(q, [&](int k, int place, int round) {
            if (!(found >> round & 1)) return;
            float v = __int_as_float(0x7fffffff);
#pragma unroll 1
            for (int m = 0; m < count; ++m)
              if (ids[mine[m]] == ids[k] && __float_as_int(sk[mine[m]]) != 0x7fffffff) v = sk[mine[m]];
            sk[k] = v;
            if (rank) st_cluster(map_to_rank(smem_u32(sk + k), 0), v);
          });
        }
        __syncwarp();
      };

      const bool two = kAcross && state != kDead;   // passes; else the second alone
      const int again = two ? again_of(chunks) : 0;
      Turn u = t;   // where the second pass begins: the first chunk that stays
      float up = 1.f, top = -INFINITY, total = 0.f, part_u = 0.f;   // of the row; the unlisted share
      if (two) {
        float based = -INFINITY, minus = 0.f;   // no base yet: every logit so far is -infinity
        bool far = false;
#pragma unroll 1
        for (int q = 0; q < chunks; ++q) {
          if (!(ok = wait(bar(&h.full[t.slot]), t.parity))) break;
          if (live) {
            T* const buf = reinterpret_cast<T*>(ring + t.slot * buffer_bytes);
            mend(q, buf);
            extract(q, buf);
            const uint32_t at = smem_u32(buf);
            const int from = warp << plan.part, to = min(from + part, s.vectors - (q << chunk_bits));
            // kBatch vectors at a time: their loads and exponentials overlap, and one look at the largest
            auto add = [&](const auto& w) {
              constexpr int kCount = sizeof(w) / sizeof(uint4);
              const float m = largest<T>(w);
              raise<T>(run, m, c);
              if (run.top != based) {
                based = run.top;
                minus = minus_base<T>(run.top, c);
                far = is_far<T>(run.top, c);
              }
              uint64_t e[kCount];
#pragma unroll
              for (int k = 0; k < kCount; ++k) {
                const Chunk<T> x(w[k], minus, c, far);
                e[k] = x.v[0];
#pragma unroll
                for (int j = 1; j < Chunk<T>::kPairs; ++j) e[k] = add2(e[k], x.v[j]);
              }
#pragma unroll
              for (int k = 0; k < kCount; ++k) run.sum = add2(run.sum, e[k]);
            };
            int v = from + lane;
#pragma unroll 1
            for (; v + (kBatch - 1) * 32 < to; v += kBatch * 32) {
              uint4 w[kBatch];
#pragma unroll
              for (int k = 0; k < kBatch; ++k) w[k] = ld_shared_v4(at + (v + k * 32) * 16);
              add(w);
            }
#pragma unroll 1
            for (; v < to; v += 32) {
              const uint4 w[1] = {ld_shared_v4(at + v * 16)};
              add(w);
            }
          }
          if (kMode == kLoss || q < again) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) mbar_arrive(bar(&h.done[t.slot]));
          }
          t.next(buffers);
          if (q + 1 == again) u = t;
        }
        if (!ok) break;
        const float2 f = unpair(run.sum);
        const Sums own{run.top, f.x + f.y, 0.f};
#pragma unroll 1
        for (int i = lane, round = 0; i < count; i += 32, ++round) {   // the listed words, each id once
          const float v = sk[mine[i]];
          if (!live || (twice >> round & 1) || v == -INFINITY) continue;
          raise<T>(run, v, c);
          run.listed += exponential<T>(v, run.top, c);
        }
        const float2 g = unpair(run.sum);
        Sums r{run.top, g.x + g.y, run.listed};
        // The consumers' sums as one, and the cluster's, for everyone; where the unlisted share is dim, once
        // more for the unlisted words alone.  A cluster's blocks may be one exchange apart: each has its barrier.
#pragma unroll 1
        for (int exchange = 0;; ++exchange) {
          r = merge_warp<T>(r, c);
          float(*const red)[4] = h.red[merges & 1];   // the last merge's may still be read
          if (lane == 0) {
            red[warp][0] = r.top;
            red[warp][1] = r.unlisted;
            red[warp][2] = r.listed;
            mbar_arrive(bar(&h.c_full[merges & 1]));
          }
          if (!(ok = wait(bar(&h.c_full[merges & 1]), merges >> 1 & 1))) break;
          ++merges;
          r = Sums{};
          if (lane < plan.warps) r = Sums{red[lane][0], red[lane][1], red[lane][2]};
          r = merge_warp<T>(r, c);
          if (across > 1 && live) {
            float(*const xch)[4] = h.xch[exchange];
            if (warp == 0 && lane < across) {
              const uint32_t to = map_to_rank(smem_u32(xch[rank]), lane);
              st_cluster(to, r.top);
              st_cluster(to + 4, r.unlisted);
              st_cluster(to + 8, r.listed);
              arrive_cluster(map_to_rank(bar(&h.x_full[exchange]), lane));
            }
            if (!(ok = __all_sync(0xffffffffu, wait_cluster(bar(&h.x_full[exchange]), 0)))) break;
            r = Sums{};
            if (lane < across) r = Sums{xch[lane][0], xch[lane][1], xch[lane][2]};
            r = merge_warp<T>(r, c);
          }
          if (exchange == 0) {
            top = r.top;
            total = r.unlisted + r.listed;
            part_u = r.unlisted;
            live = live && top != -INFINITY;
            if (!(a.teacher_lse && live && part_u < kDim)) break;   // the same for every consumer of the cluster
            r = own;
          } else {
            part_u = dim_share<T>(r, top, c, plan.c_low);
            break;
          }
        }
        if (!ok) break;
      }
      if (kAcross && threadIdx.x == 0) {
        h.result[slot][0] = top;
        h.result[slot][1] = total;
        h.result[slot][2] = part_u;
        h.result[slot][3] = live ? 1.f : 0.f;
        mbar_arrive(bar(&h.r_full[slot]));
      }
      if constexpr (kMode != kLoss) {
        if (!(ok = wait(bar(&h.m_full[slot]), n / kRows & 1))) break;
        if (!kAcross) {
          top = h.result[slot][0];
          total = h.result[slot][1];
          part_u = h.result[slot][2];
          live = live && !(total == 0.f);
          up = h.result[slot][3];
          // an id listed twice, where the lanes hold all of the entries
          repeated = count > 32;
          if (live && !repeated) {
            const uint32_t same = __match_any_sync(0xffffffffu, k0 >= 0 ? place0 : -1 - lane);
            repeated = __any_sync(0xffffffffu, (same & (same - 1)) != 0);
          }
        }
        const float inv = 1.f / total, mass = h.teacher[slot][kMass];
        const float rest = part_u == 0.f ? 0.f : h.teacher[slot][kRest];
        const float scale = h.teacher[slot][kWeight] * a.d.temperature * up, all = mass + rest;
        float base = top, coef;   // an unlisted word's gradient: coef times its exponential relative to base
        if (rest != 0.f && part_u < kSmall) {
          const Base b = base_of_share<T>(part_u, top, c, a.d.temperature);
          base = b.base;
          coef = scale * (all * inv * b.down - rest / b.sum);
        } else {
          coef = scale * (rest != 0.f ? all - rest / (part_u * inv) : all) * inv;
        }
        T* const dst = grad_at(row, begin) - s.lead;
        const bool apart = (reinterpret_cast<uintptr_t>(dst) & 15) != 0, far = is_far<T>(base, c);
        const float minus = minus_base<T>(base, c);
        const uint64_t kk = pair(coef, coef);
        // The teacher's part of an entry's gradient; an id listed twice has the sum at each of its entries.
        auto entry_p = [&](int k) {
          if (!repeated) return expf(lp[k]);
          float pk = 0.f;
#pragma unroll 1
          for (int m = 0; m < count; ++m)
            if (ids[mine[m]] == ids[k]) pk += expf(lp[mine[m]]);
          return pk;
        };
        auto entry_gradient = [&](float s, float pk) {
          return from_f<T>(scale * (exponential<T>(s, top, c) * inv * all - pk));
        };
        const float p0 = live && k0 >= 0 ? entry_p(k0) : 0.f;
        const T g0 = kMode == kBoth && live && k0 >= 0 ? entry_gradient(sk[k0], p0) : from_f<T>(0.f);
#pragma unroll 1
        for (int j = 0; j < chunks; ++j) {
          const int q = j < chunks - again ? j + again : j - (chunks - again);   // those that stayed come first
          const bool came = !two || j >= chunks - again;
          if (came && !(ok = wait(bar(&h.full[u.slot]), u.parity))) break;
          T* const buf = reinterpret_cast<T*>(ring + u.slot * buffer_bytes);
          const uint32_t at = smem_u32(buf);
          const int from = warp << plan.part, to = min(from + part, s.vectors - (q << chunk_bits));
          const int origin = q << (chunk_bits + kLog);
          if (came && state != kDead) mend(q, buf);
          if (kMode == kGradient && live) {
            entries(q, [&](int k, int place, int round) { sk[k] = to_f(buf[place - origin]); });
            __syncwarp();
          }
          auto turn = [&](uint4 w) {
            if (!live) return make_uint4(0, 0, 0, 0);
            Chunk<T> x(w, minus, c, far);
#pragma unroll
            for (int k = 0; k < Chunk<T>::kPairs; ++k) x.v[k] = mul2(x.v[k], kk);
            return x.packed();
          };
          int v = from + lane;
          if (!apart)
#pragma unroll 1
            for (; v + (kBatch - 1) * 32 < to; v += kBatch * 32) {
              uint4 w[kBatch];
#pragma unroll
              for (int k = 0; k < kBatch; ++k) w[k] = ld_shared_v4(at + (v + k * 32) * 16);
#pragma unroll
              for (int k = 0; k < kBatch; ++k) st_shared_v4(at + (v + k * 32) * 16, turn(w[k]));
            }
#pragma unroll 1
          for (; v < to; v += 32) {
            const uint4 w = turn(ld_shared_v4(at + v * 16));
            if (!apart) {
              st_shared_v4(at + v * 16, w);
            } else {   // the gradient's rows start at other phases than the logits'
              const T* g = reinterpret_cast<const T*>(&w);
#pragma unroll
              for (int k = 0; k < kN; ++k) {
                const int place = ((q << chunk_bits) + v) * kN + k;
                if (s.inside(place)) dst[place] = g[k];
              }
            }
          }
          __syncwarp();
          if (live) {
            entries(q, [&](int k, int place, int round) {
              const T g = kMode == kBoth && round == 0 ? g0 : entry_gradient(sk[k], round == 0 ? p0 : entry_p(k));
              if (apart) dst[place] = g;
              else buf[place - origin] = g;
            });
            __syncwarp();
          }
          if (!apart && edge_at >= 0 && edge_at >> (chunk_bits + kLog) == q && s.inside(edge_at))
            dst[edge_at] = buf[edge_at - origin];
          fence_proxy_async_smem();
          __syncwarp();
          if (lane == 0) mbar_arrive(bar(&h.done[u.slot]));
          u.next(buffers);
        }
        t = u;
      }
      if (!ok) break;
      __syncwarp();
      if (lane == 0) mbar_arrive(bar(&h.t_free[slot]));
    }
  }
  if (!ok) report_error(a.err, kErrWaitOperand);
  // no block leaves while another may still write to its shared memory
  if (across > 1) {
    __syncwarp();
    cluster_sync();
  }
}

Plan make_plan(const DistillArgs& a, int elt) {
  Plan p{};
  const long long v = a.d.vocab;
  // A block for each row.  In calls of a few rows a cluster shares each, while a slice keeps 2 KB; its
  // sums are added in another order, so the rule goes by the rows alone and its bound is low: other calls
  // give a row the same result whatever rows are beside it.  One or four rows of 131072 bf16: 8.1 us, a
  // block each 19.8; of 32000: 7.5, 8.5.
  p.slices = 1;
  if (a.d.rows <= kFewRows)
    while (p.slices < kMaxCluster && v * elt / (2 * p.slices) >= 2048) p.slices *= 2;
  p.width = (int)(((v + p.slices - 1) / p.slices + 127) / 128 * 128);
  const bool aligned = reinterpret_cast<uintptr_t>(a.logits) % 16 == 0 && a.d.logits_stride * elt % 16 == 0;
  p.ragged = !aligned || v * elt % 16 != 0;
  const double c = 1.4426950408889634 / (double)a.d.temperature;
  p.c = (float)c;
  p.c_low = (float)(c - (double)p.c);
  const int vectors = (int)(std::min<long long>(p.width, v) * elt + 15) / 16 + !aligned;
  // Chunks of 32 KB for eight warps, two batches of vectors for each lane (2048x32000 bf16: 55 us; of 16
  // KB, one batch between waits: 64); smaller where the row is.
  p.part = 8;
  p.warps = kMaxWarps;
  while (p.warps > 1 && (p.warps << p.part) / 2 >= vectors) p.warps /= 2;
  while (p.part > 5 && (p.warps << p.part) / 2 >= vectors) --p.part;
  const int chunk = p.warps << p.part << 4;
  p.kp = (int)((a.d.topk + 31) / 32 * 32);
  const int fixed = (int)((sizeof(Header) + 15) / 16 * 16 + (size_t)p.kp * (kRows * 12 + p.warps * 2) + 127) / 128 * 128;
  // Two blocks an SM: while one waits for loads or for its sums, the other computes (55 us; one block with
  // twice the ring: 78).
  p.buffers = std::max(2, std::min((113 * 1024 - fixed) / chunk, kMaxBuffers));
  p.smem = fixed + p.buffers * chunk;
  return p;
}

template <typename T, int kMode>
int launch(const DistillArgs& a, cudaStream_t st) {
  auto kernel = distill_kernel<T, kMode>;
  constexpr bool kAcross = kMode != kGradient;
  Plan p = make_plan(a, sizeof(T));
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kernel), 227 * 1024)) return CBR_ERR_CUDA;
  const int across = kAcross ? p.slices : 1;
  const long long items = kAcross ? a.d.rows : a.d.rows * p.slices;
  const int threads = (p.warps + kOthers) * 32;
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
  // how many clusters run at once: asked once for each launch shape and device
  static std::mutex mu;
  static std::map<std::tuple<int, int, int, int>, int> at_once;
  int clusters = 0, dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return CBR_ERR_CUDA;
  {
    std::lock_guard<std::mutex> lk(mu);
    int& n = at_once[{threads, p.smem, across, dev}];
    if (!n && cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) {
      cudaGetLastError();
      n = 0;
      return CBR_ERR_CUDA;
    }
    clusters = n;
  }
  if (clusters < 1) return CBR_ERR_CUDA;
  cfg.gridDim = dim3((unsigned)((across > 1 ? items : std::min<long long>(items, clusters)) * across));
  if (cudaLaunchKernelEx(&cfg, kernel, a, p) != cudaSuccess) {
    cudaGetLastError();
    return CBR_ERR_CUDA;
  }
  return CBR_OK;
}

template <typename T>
int launch_of(const DistillArgs& a, bool backward, cudaStream_t st) {
  if (backward) return launch<T, kGradient>(a, st);
  return a.dlogits ? launch<T, kBoth>(a, st) : launch<T, kLoss>(a, st);
}

int launch_any(const DistillArgs& a, bool backward, cudaStream_t st) {
  if (a.d.dtype == CBR_F32) return launch_of<float>(a, backward, st);
  if (a.d.dtype == CBR_BF16) return launch_of<__nv_bfloat16>(a, backward, st);
  return launch_of<__half>(a, backward, st);
}

}  // namespace

int launch_distill(const DistillArgs& a, cudaStream_t st) { return launch_any(a, false, st); }

int launch_distill_backward(const DistillArgs& a, cudaStream_t st) { return launch_any(a, true, st); }

}  // namespace cbr
