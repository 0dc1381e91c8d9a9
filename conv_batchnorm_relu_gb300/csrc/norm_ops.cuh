// What the block norms' forward and backward kernels share: how a row is laid over a team of threads,
// its loads and stores, and sums over a team.
//
// A team is a part of a warp (narrow rows) or a whole block.  A thread holds kEpt elements of a row in
// registers, in 16-byte vectors a team's width apart (kVec elements each), or, where a row does not
// divide into aligned vectors, one by one (kVec = 1), a team's width apart too, so that a warp's loads
// are consecutive either way.
#pragma once
#include "common.cuh"
#include "token_ops.cuh"

namespace cbr {
namespace norm {

using namespace tok;

// A thread's share of a row.  `left`: the elements from its first column to the row's end.
// Pointers to rows are given at the first of its columns.
template <typename T, int kVec, int kEpt>
struct Row {
  static constexpr int kSteps = kEpt / kVec;
  // single elements: a register each (16-bit ones in pairs would be packed, and waited for, at once)
  using Raw = std::conditional_t<kVec == 1, uint32_t, uint4>;
  Raw raw[kSteps];

  static __device__ __forceinline__ int column(int step, int team) { return step * team * kVec; }
  static __device__ __forceinline__ bool inside(int i, int team, int left) { return column(i / kVec, team) < left; }

  // Streaming loads: nothing of a row is read twice.  Columns past the row read as zero.
  __device__ __forceinline__ void load(const T* p, int team, int left) {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int c = column(j, team);
      if constexpr (kVec == 1) {
        raw[j] = 0;
        if (c < left) {
          if constexpr (sizeof(T) == 4) asm volatile("ld.global.b32 %0, [%1];" : "=r"(raw[j]) : "l"(p + c));
          else asm volatile("ld.global.u16 %0, [%1];" : "=r"(raw[j]) : "l"(p + c));
        }
      } else {
        raw[j] = make_uint4(0, 0, 0, 0);
        if (c < left)
          asm volatile("ld.global.L1::no_allocate.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(raw[j].x), "=r"(raw[j].y), "=r"(raw[j].z), "=r"(raw[j].w)
                       : "l"(p + c));
      }
    }
  }
  // From a row in shared memory.
  __device__ __forceinline__ void load_shared(uint32_t p, int team, int left) {
    if constexpr (kVec > 1) {
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const int c = column(j, team);
        raw[j] = c < left ? ld_shared_v4(p + c * (uint32_t)sizeof(T)) : make_uint4(0, 0, 0, 0);
      }
    }
  }
  __device__ __forceinline__ void get(float (&v)[kEpt]) const {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      if constexpr (kVec == 1) {
        if constexpr (sizeof(T) == 4) v[j] = __uint_as_float(raw[j]);
        else if constexpr (std::is_same_v<T, __nv_bfloat16>) v[j] = __uint_as_float(raw[j] << 16);
        else v[j] = unpack2<false>(raw[j]).x;
      } else if constexpr (sizeof(T) == 4) {
        v[4 * j] = __uint_as_float(raw[j].x), v[4 * j + 1] = __uint_as_float(raw[j].y);
        v[4 * j + 2] = __uint_as_float(raw[j].z), v[4 * j + 3] = __uint_as_float(raw[j].w);
      } else {
        const uint32_t u[4] = {raw[j].x, raw[j].y, raw[j].z, raw[j].w};
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = unpack2<std::is_same_v<T, __nv_bfloat16>>(u[k]);
          v[8 * j + 2 * k] = f.x, v[8 * j + 2 * k + 1] = f.y;
        }
      }
    }
  }
  static __device__ __forceinline__ void store(T* p, const float (&v)[kEpt], int team, int left) {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int c = column(j, team);
      if (c >= left) continue;
      if constexpr (kVec == 1) {
        p[c] = from_f<T>(v[j]);
      } else if constexpr (sizeof(T) == 4) {
        st_global_v4(p + c, make_uint4(__float_as_uint(v[4 * j]), __float_as_uint(v[4 * j + 1]),
                                       __float_as_uint(v[4 * j + 2]), __float_as_uint(v[4 * j + 3])));
      } else {
        uint32_t u[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) u[k] = pack2<std::is_same_v<T, __nv_bfloat16>>(v[8 * j + 2 * k], v[8 * j + 2 * k + 1]);
        st_global_v4(p + c, make_uint4(u[0], u[1], u[2], u[3]));
      }
    }
  }
  // fp32 parameters of this thread's columns; zero past the row.
  static __device__ __forceinline__ void params(const float* p, float (&v)[kEpt], int team, int left) {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int c = column(j, team);
      if constexpr (kVec == 1) {
        v[j] = c < left ? __ldg(p + c) : 0.f;
      } else {
#pragma unroll
        for (int k = 0; k < kVec; k += 4) {
          const float4 f = c < left ? __ldg(reinterpret_cast<const float4*>(p + c + k)) : make_float4(0, 0, 0, 0);
          v[kVec * j + k] = f.x, v[kVec * j + k + 1] = f.y, v[kVec * j + k + 2] = f.z, v[kVec * j + k + 3] = f.w;
        }
      }
    }
  }
  static __device__ __forceinline__ void put(float* p, const float (&v)[kEpt], int team, int left) {
#pragma unroll
    for (int j = 0; j < kSteps; ++j) {
      const int c = column(j, team);
      if (c >= left) continue;
      if constexpr (kVec == 1) {
        p[c] = v[j];
      } else {
#pragma unroll
        for (int k = 0; k < kVec; k += 4)
          *reinterpret_cast<float4*>(p + c + k) =
              make_float4(v[kVec * j + k], v[kVec * j + k + 1], v[kVec * j + k + 2], v[kVec * j + k + 3]);
      }
    }
  }
};

__device__ __forceinline__ float from_lane(float v, int o) { return __shfl_xor_sync(0xffffffffu, v, o); }

// Sums over a team, the same for every one of its threads; a block has at most 16 warps.  Its warps leave
// theirs in shared memory, in one of two places in turn: whoever writes a place for the second time has
// been through the barrier that follows its last reads.  Of several values (four, in effect), each
// quarter of a warp comes to hold one, which takes a shuffle or two a step for all of them together.
constexpr int kMaxTeamWarps = 16;
template <bool kBlock, int kValues>
struct TeamSum {
  static_assert(kValues <= 4, "a quarter of a warp for each");
  float (*red)[kValues == 1 ? 1 : 4][kMaxTeamWarps];   // two of them, zero past the block's warps
  int turn = 0;
  __device__ __forceinline__ void operator()(float (&v)[kValues], int team) {
    if constexpr (!kBlock) {
#pragma unroll
      for (int o = 16; o; o >>= 1)
        if (o < team) {
#pragma unroll
          for (int i = 0; i < kValues; ++i) v[i] += from_lane(v[i], o);
        }
    } else if constexpr (kValues == 1) {
#pragma unroll
      for (int o = 16; o; o >>= 1) v[0] += from_lane(v[0], o);
      float* r = red[turn][0];
      turn ^= 1;
      if ((threadIdx.x & 31) == 0) r[threadIdx.x >> 5] = v[0];
      __syncthreads();
      float s = r[threadIdx.x & 15];
#pragma unroll
      for (int o = 8; o; o >>= 1) s += from_lane(s, o);
      v[0] = s;
    } else {
      const int lane = threadIdx.x & 31;
      const float v2 = kValues > 2 ? v[2] : 0.f, v3 = kValues > 3 ? v[3] : 0.f;
      const bool a = lane & 16, b = lane & 8;
      const float k0 = (a ? v2 : v[0]) + from_lane(a ? v[0] : v2, 16);
      const float k1 = (a ? v3 : v[1]) + from_lane(a ? v[1] : v3, 16);
      float x = (b ? k1 : k0) + from_lane(b ? k0 : k1, 8);
#pragma unroll
      for (int o = 4; o; o >>= 1) x += from_lane(x, o);
      float(*r)[kMaxTeamWarps] = red[turn];
      turn ^= 1;
      if ((lane & 7) == 0) r[lane >> 3][threadIdx.x >> 5] = x;
      __syncthreads();
      x = r[lane >> 3][lane & 7] + r[lane >> 3][(lane & 7) + 8];
#pragma unroll
      for (int o = 4; o; o >>= 1) x += from_lane(x, o);
#pragma unroll
      for (int i = 0; i < kValues; ++i) v[i] = __shfl_sync(0xffffffffu, x, 8 * i);
    }
  }
};

// 1 / sqrt(x), x > 0: the hardware's estimate and a Newton step, which leaves about a rounding (a square
// root and a division would be a fifth of a row's instructions).  0 for infinity, whose step would be
// infinity times 0.
__device__ __forceinline__ float inverse_root(float x) {
  const float y = rsqrtf(x);
  return x == INFINITY ? 0.f : y * fmaf(-0.5f * x * y, y, 1.5f);
}

inline bool aligned16(const void* p) { return reinterpret_cast<uintptr_t>(p) % 16 == 0; }

}  // namespace norm
}  // namespace cbr
