// Rotary positions over several axes (formulas: include/cbr.h).
//
// A block takes a few consecutive tokens: the cosines and sines of their pairs once, into shared memory,
// then the heads of q and k, a 16-byte vector (and, with pairs in halves, its partner) a thread and step.
// The angle is a product modulo 2^64 of the position and the frequency in turns, so it is reduced to one
// turn without rounding; its top 32 bits, as a signed fraction of half a turn, go to sincospif.  Bound by
// HBM, each element of q and k read and written once: 65536 tokens of 40 heads of 128 bf16 in 197 us, 6.8
// TB/s; calls that fit in L2 by the index arithmetic of each vector (12544 tokens of 24 heads of 80 f16: 21
// us, 4.6 TB/s).
#include <algorithm>
#include <type_traits>

#include "cbr_internal.h"
#include "common.cuh"
#include "token_ops.cuh"

namespace cbr {
namespace {

using namespace tok;

constexpr int kThreads = 128;

// How a call is laid out: `unit` elements a vector (kUnit, or 1), in items of one vector (neighbours, or a
// copied part) or two (the halves of pairs).
struct Plan {
  int tokens;        // of a block
  int items;         // of one head
  int rotated;       // of them, those that are rotated; the others are copied
  int heads;
  FastDiv per_head;  // by items
  FastDiv per_token; // by heads * items
  long long blocks_a_batch;
};

__device__ __forceinline__ uint32_t fast_div(uint32_t n, FastDiv f) {
  const uint32_t t = __umulhi(f.m, n);
  return (t + ((n - t) >> f.s1)) >> f.s2;
}

template <typename T, int kUnit>
struct Vector {
  float v[kUnit];
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kUnit == 1) {
      v[0] = to_f(*p);
    } else {
      uint4 w;
      asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w)
                   : "l"(p));
      const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) {
          v[i] = __uint_as_float(u[i]);
        } else {
          const float2 f = unpack2<std::is_same_v<T, __nv_bfloat16>>(u[i]);
          v[2 * i] = f.x, v[2 * i + 1] = f.y;
        }
      }
    }
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kUnit == 1) {
      *p = from_f<T>(v[0]);
    } else {
      uint32_t u[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 4) u[i] = __float_as_uint(v[i]);
        else u[i] = pack2<std::is_same_v<T, __nv_bfloat16>>(v[2 * i], v[2 * i + 1]);
      }
      st_global_v4(p, make_uint4(u[0], u[1], u[2], u[3]));
    }
  }
};

// n turns of the table, two at a time (vectors of elements start at even pairs).
template <int n>
__device__ __forceinline__ void turns(const float2* p, float2 (&w)[n]) {
  if constexpr (n == 1) {
    w[0] = *p;
  } else {
#pragma unroll
    for (int k = 0; k < n; k += 2) {
      const float4 f = *reinterpret_cast<const float4*>(p + k);
      w[k] = make_float2(f.x, f.y), w[k + 1] = make_float2(f.z, f.w);
    }
  }
}

template <typename T, int kUnit, bool kHalves>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a,
                                                          const __grid_constant__ Plan plan) {
  extern __shared__ __align__(16) float2 turn[];   // [tokens][pairs]: cosine, sine
  const cbr_rotary_desc_t& d = a.d;
  const int pairs = d.rot_dim / 2;
  const long long b = blockIdx.x / plan.blocks_a_batch;
  const long long t0 = (blockIdx.x - b * plan.blocks_a_batch) * plan.tokens;
  const int tokens = (int)min((long long)plan.tokens, d.tokens - t0);

  for (int i = threadIdx.x; i < tokens * pairs; i += kThreads) {
    const int t = i / pairs, p = i - t * pairs;
    const int axis = min((int)__ldg(a.axis + p), d.axes - 1);
    const long long pos = a.positions[b * d.pos_stride[0] + (t0 + t) * d.pos_stride[1] + axis * d.pos_stride[2]];
    const unsigned long long f = (unsigned long long)pos * (unsigned long long)__ldg(a.freq + p);
    float sn, cs;
    sincospif((float)(int)(f >> 32) * 0x1p-31f, &sn, &cs);
    turn[i] = make_float2(cs, a.backward ? -sn : sn);
  }
  __syncthreads();

  const int per_token = plan.heads * plan.items;
  for (int i = threadIdx.x; i < tokens * per_token; i += kThreads) {
    const int t = fast_div(i, plan.per_token), j = i - t * per_token;
    const int head = fast_div(j, plan.per_head), item = j - head * plan.items;
    const bool is_q = head < d.heads_q;
    const int h = is_q ? head : head - d.heads_q;
    const int64_t* si = is_q ? d.q_stride : d.k_stride;
    const int64_t* so = is_q ? d.q_out_stride : d.k_out_stride;
    const T* in = static_cast<const T*>(is_q ? a.q : a.k) + b * si[0] + (t0 + t) * si[1] + h * si[2];
    T* out = static_cast<T*>(is_q ? a.q_out : a.k_out) + b * so[0] + (t0 + t) * so[1] + h * so[2];
    const float2* cs = turn + t * pairs;
    const bool copied = item >= plan.rotated;
    if (copied && in == out) continue;
    if constexpr (kHalves || kUnit == 1) {
      if (copied) {
        const int c = d.rot_dim + (item - plan.rotated) * kUnit;
        Vector<T, kUnit> x;
        x.load(in + c);
        x.store(out + c);
        continue;
      }
      // a pair's two elements are in two vectors (or are two single ones)
      const int c = kHalves ? item * kUnit : item * 2, partner = kHalves ? pairs : 1;
      Vector<T, kUnit> x, y;
      x.load(in + c);
      y.load(in + c + partner);
      float2 w[kUnit];
      turns<kUnit>(cs + item * kUnit, w);
#pragma unroll
      for (int k = 0; k < kUnit; ++k) {
        const float u = x.v[k], v = y.v[k];
        x.v[k] = u * w[k].x - v * w[k].y;
        y.v[k] = v * w[k].x + u * w[k].y;
      }
      x.store(out + c);
      y.store(out + c + partner);
    } else {
      const int c = item * kUnit;   // the copied part comes right after the rotated one
      Vector<T, kUnit> x;
      x.load(in + c);
      if (!copied) {
        float2 w[kUnit / 2];
        turns<kUnit / 2>(cs + c / 2, w);
#pragma unroll
        for (int k = 0; k < kUnit; k += 2) {
          const float u = x.v[k], v = x.v[k + 1];
          x.v[k] = u * w[k / 2].x - v * w[k / 2].y;
          x.v[k + 1] = v * w[k / 2].x + u * w[k / 2].y;
        }
      }
      x.store(out + c);
    }
  }
}

template <typename T, int kUnit, bool kHalves>
int launch(const RotaryArgs& a, int num_sms, cudaStream_t st) {
  const cbr_rotary_desc_t& d = a.d;
  const int pairs = d.rot_dim / 2;
  Plan p{};
  p.rotated = kHalves ? pairs / kUnit : kUnit > 1 ? d.rot_dim / kUnit : pairs;
  p.items = p.rotated + (d.head_dim - d.rot_dim) / kUnit;
  p.heads = d.heads_q + d.heads_k;
  const long long per_token = (long long)p.heads * p.items;
  // About four items a thread, so that the table is a small part of a block's work, while there are
  // blocks for every SM (us, the two calls above: 197 and 21; one item 197 and 23, eight 201 and 22; blocks
  // of 256 threads 198 and 21); at most 16 KB of table.
  const long long all = d.batch * d.tokens;
  long long want = std::max(1ll, 4ll * kThreads / per_token);
  want = std::min(want, std::max(1ll, all / (4ll * num_sms)));
  p.tokens = (int)std::min(want, std::max(1ll, 2048ll / pairs));
  p.per_head = make_fastdiv((uint32_t)p.items);
  p.per_token = make_fastdiv((uint32_t)per_token);
  p.blocks_a_batch = (d.tokens + p.tokens - 1) / p.tokens;
  const long long blocks = p.blocks_a_batch * d.batch;
  if (blocks > 0x7fffffffll) return CBR_ERR_UNSUPPORTED;
  rotary_kernel<T, kUnit, kHalves><<<(unsigned)blocks, kThreads, p.tokens * pairs * sizeof(float2), st>>>(a, p);
  return cudaGetLastError() == cudaSuccess ? CBR_OK : CBR_ERR_CUDA;
}

// Whether every head that is read or written starts on a 16-byte boundary and splits into whole vectors.
bool vectors(const RotaryArgs& a, int n) {
  const cbr_rotary_desc_t& d = a.d;
  auto fits = [&](const void* p, const int64_t* s) {
    return reinterpret_cast<uintptr_t>(p) % 16 == 0 && s[0] % n == 0 && s[1] % n == 0 && s[2] % n == 0;
  };
  const int part = d.layout == CBR_ROTARY_HALVES ? d.rot_dim / 2 : d.rot_dim;
  return part % n == 0 && (d.head_dim - d.rot_dim) % n == 0 &&
         (!d.heads_q || (fits(a.q, d.q_stride) && fits(a.q_out, d.q_out_stride))) &&
         (!d.heads_k || (fits(a.k, d.k_stride) && fits(a.k_out, d.k_out_stride)));
}

template <typename T>
int by_layout(const RotaryArgs& a, int num_sms, cudaStream_t st) {
  constexpr int kUnit = 16 / sizeof(T);
  const bool halves = a.d.layout == CBR_ROTARY_HALVES;
  if (vectors(a, kUnit))
    return halves ? launch<T, kUnit, true>(a, num_sms, st) : launch<T, kUnit, false>(a, num_sms, st);
  return halves ? launch<T, 1, true>(a, num_sms, st) : launch<T, 1, false>(a, num_sms, st);
}

}  // namespace

int launch_rotary(const RotaryArgs& a, int num_sms, cudaStream_t st) {
  if (a.d.dtype == CBR_F32) return by_layout<float>(a, num_sms, st);
  if (a.d.dtype == CBR_BF16) return by_layout<__nv_bfloat16>(a, num_sms, st);
  return by_layout<__half>(a, num_sms, st);
}

}  // namespace cbr
