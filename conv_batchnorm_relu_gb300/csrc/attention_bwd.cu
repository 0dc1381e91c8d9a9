// Attention backward (declared in include/cbr.h) on the tensor cores: the probabilities are computed again.
//
// Two launches.  prepare_kernel takes D_i = do_i . o_i and the exponents' offsets.  backward_kernel has blocks of two
// kinds.  One holds a tile of 128 queries and walks over the keys: S = Q K^T, dP = dO V^T, dQ += dS K.  The other
// holds a tile of 128 keys and walks over the queries of all heads that read it: S' = K Q^T, dP' = V dO^T,
// dV += P' dO, dK += dS' Q.  Scores and dP are taken twice (seven products instead of five), and in return every sum
// stays in TMEM to its end, in a fixed order: no atomics, no sums in memory.
//   P and dS go from registers over their scores in TMEM and enter the second products from there; each rounded to the
// storage type for that.  A thread has a row of a tile and 64 of its columns.
//   f16: p is taken 2^12 times as large, and dS a power of two times as large that a bound on |do| |v| gives
// for each key head, so that small ones keep their digits; the results are scaled back.
//   Queries past the last one have the offset -infinity (p = 0), keys past theirs are cut off at the outputs.
//   Bound by the products with heads of 128 (2 of 8192 tokens, 16 heads, bf16: 1.13 ms; the seven products alone take
// 1.02 at the rate that a library's matrix product has here); with heads of 64 a step's chain of products and
// exponentials, the tensor cores busy 35% of the time (16 of 784, 12 heads, f16: 177 us).
#include <algorithm>

#include "attention.cuh"
#include "cbr_internal.h"

namespace cbr {
namespace att {
namespace {

// By the head: kN, the tokens that a step of a walk takes (what stays has 128), and the warps.  Warps 0-3 (and 4-7) have the
// 128 rows of a tile of scores, 64 columns of each to a thread; one loads, one issues the products.  Heads of 64 take
// half of TMEM, and two blocks to an SM, one's start and end over the other's walk (16x784 tokens, 12 heads of 64: one block
// and kN = 128, in two launches, took 1.46 times as long; 32 columns to a thread and twice the warps 1.05 times).
template <int kDim>
struct Form {
  static constexpr int kN = kDim, kRowWarps = kN / 16, kHalves = kN / 64, kThreads = 32 * (kRowWarps + 2), kBlocks = 128 / kDim;
  static constexpr int kLoadWarp = kRowWarps, kMmaWarp = kRowWarps + 1;
  static constexpr int kStep = kN * kDim * 2;   // bytes of a step's tile
  static constexpr uint32_t kColumns = 4 * kN;  // of TMEM, in quarters
};

// Where a kind of block puts its results.
struct Results {
  void* out[2];
  int64_t stride[2][3];
  float* part;            // splits > 1: [split][out][rows of the outputs][head_dim]
  int64_t part_rows;
  int32_t splits;
  int32_t blocks;         // of one split
};

struct BackwardParams {
  Params p;
  const float* offset;    // [batch * packs][rows]: shift - lse log2(e) of a row, -infinity where p is 0
  const float* delta;     // the same of -D
  const uint32_t* norms;  // f16: [batch][heads_k][2] bits of the largest |do|^2 and |v|^2
  int64_t rows;           // of a pack of heads, a multiple of 128
  int64_t batch;
  Results queries, keys;  // dq; dv, dk
};

template <bool BF16>
constexpr float kShift = BF16 ? 0.f : 12.f;

// f16: the power of two that takes |dP - D| <= 2 max|do| max|v| to at most 2^14; 1 where that bound says nothing.
template <bool BF16>
__device__ __forceinline__ float ds_scale(const BackwardParams& f, int batch, int key_head) {
  if constexpr (BF16) return 1.f;
  const uint32_t* n = f.norms + 2 * ((int64_t)batch * f.p.heads_k + key_head);
  const float bound = 2.f * sqrtf(__uint_as_float(n[0])) * sqrtf(__uint_as_float(n[1]));
  if (!(bound > 0.f && bound < INFINITY)) return 1.f;
  return __int_as_float((127 + 14 - (ilogbf(bound) + 1)) << 23);
}

// ---------------------------------------------------------------- D, offsets, bounds

constexpr int kTurns = 4;   // rows of a thread in a block of 256
template <int kDim>
constexpr int kLanes = kDim / 8;                             // of a row
template <int kDim>
constexpr int kPrepareRows = kTurns * 256 / kLanes<kDim>;    // of a block: 64 or 128

struct PrepareParams {
  BackwardParams f;
  const void* d_o;
  const void* o;
  const void* v;
  int64_t do_stride[3], o_stride[3], v_stride[3];
  const float* lse;
  float* offset;
  float* delta;
  uint32_t* norms;
  int64_t query_blocks;   // blocks of queries; the others (f16) take values
};

template <int kDim>
__device__ __forceinline__ float row_sum(float v) {
#pragma unroll
  for (int o = kLanes<kDim> / 2; o; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// |a|^2 of a thread's eight elements, and a . b.
template <bool BF16>
__device__ __forceinline__ float dot8(const uint4& a, const uint4& b) {
  const uint32_t x[4] = {a.x, a.y, a.z, a.w}, y[4] = {b.x, b.y, b.z, b.w};
  float s = 0.f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 u = unpack2<BF16>(x[i]), w = unpack2<BF16>(y[i]);
    s = fmaf(u.x, w.x, s);
    s = fmaf(u.y, w.y, s);
  }
  return s;
}

template <int kDim, bool BF16>
__global__ void __launch_bounds__(256) prepare_kernel(const __grid_constant__ PrepareParams g) {
  const Params& a = g.f.p;
  __shared__ float largest[8];
  let_next_kernel_start();
  constexpr int kSubs = 256 / kLanes<kDim>;
  const int lane = threadIdx.x % kLanes<kDim>, sub = threadIdx.x / kLanes<kDim>, e = lane * 8;
  const bool queries = blockIdx.x < g.query_blocks;
  float most = 0.f;
  int64_t batch, key_head;
  if (queries) {
    const uint32_t packs = a.heads_q / a.pack, per = (uint32_t)(g.f.rows / kPrepareRows<kDim>), place = blockIdx.x / per;
    const int64_t at = place, first = (int64_t)(blockIdx.x - place * per) * kPrepareRows<kDim>;
    const uint32_t head = place % packs;
    batch = place / packs;
    const int shift = 31 - __clz(a.pack);   // a power of two
    key_head = a.pack > 1 ? head : head / a.group;
    uint4 u[kTurns], w[kTurns];
    float lse[kTurns];
#pragma unroll
    for (int r = 0; r < kTurns; ++r) {
      const int64_t row = first + r * kSubs + sub, token = row >> shift, h = (head << shift) + (row & (a.pack - 1));
      u[r] = w[r] = make_uint4(0, 0, 0, 0);
      lse[r] = -INFINITY;
      if (token >= a.q_tokens) continue;
      if (e < a.head_dim) {
        u[r] = ld_global_nc_v4(static_cast<const uint16_t*>(g.d_o) + batch * g.do_stride[0] + token * g.do_stride[1] + h * g.do_stride[2] + e);
        w[r] = ld_global_nc_v4(static_cast<const uint16_t*>(g.o) + batch * g.o_stride[0] + token * g.o_stride[1] + h * g.o_stride[2] + e);
      }
      if (lane == 0) lse[r] = g.lse[(batch * a.heads_q + h) * a.q_tokens + token];
    }
#pragma unroll
    for (int r = 0; r < kTurns; ++r) {
      const float d = row_sum<kDim>(dot8<BF16>(u[r], w[r]));
      if constexpr (!BF16) most = tok::Max::of(most, row_sum<kDim>(dot8<BF16>(u[r], u[r])));
      if (lane == 0) {
        const int64_t to = at * g.f.rows + first + r * kSubs + sub;
        g.offset[to] = lse[r] == -INFINITY ? -INFINITY : kShift<BF16> - lse[r] * kLog2e;
        g.delta[to] = -d;
      }
    }
  } else {
    const uint32_t per = (a.k_tokens + kPrepareRows<kDim> - 1) / kPrepareRows<kDim>, block = blockIdx.x - (uint32_t)g.query_blocks;
    const uint32_t place = block / per;
    const int64_t first = (int64_t)(block - place * per) * kPrepareRows<kDim>;
    key_head = place % a.heads_k;
    batch = place / a.heads_k;
    const int keys = keys_of(a, (int)batch);
    uint4 u[kTurns];
#pragma unroll
    for (int r = 0; r < kTurns; ++r) {
      const int64_t row = first + r * kSubs + sub;
      u[r] = make_uint4(0, 0, 0, 0);
      if (row < keys && e < a.head_dim)
        u[r] = ld_global_nc_v4(static_cast<const uint16_t*>(g.v) + batch * g.v_stride[0] + row * g.v_stride[1] + key_head * g.v_stride[2] + e);
    }
#pragma unroll
    for (int r = 0; r < kTurns; ++r) most = tok::Max::of(most, row_sum<kDim>(dot8<BF16>(u[r], u[r])));
  }
  if constexpr (!BF16) {
    most = tok::warp_max(most);
    if ((threadIdx.x & 31) == 0) largest[threadIdx.x >> 5] = most;
    __syncthreads();
    if (threadIdx.x == 0) {
      for (int i = 1; i < 8; ++i) most = tok::Max::of(most, largest[i]);
      // bits of floats that are not negative are in their order, those of a NaN above all: the largest does not
      // depend on the order of the blocks
      atomicMax(g.norms + 2 * (batch * a.heads_k + key_head) + !queries, __float_as_uint(fabsf(most)));
    }
  }
}

// ---------------------------------------------------------------- a row's results

// 32 columns of a row from TMEM, scaled: whole results in the storage type, parts of them in 32 bits.
//   any: the accumulator was written (the same in the whole warp); use: the row has a result, else 0.
template <bool BF16>
__device__ __forceinline__ void store32(uint32_t taddr, int col, int dim, bool any, bool use, bool live, float scale, uint8_t* out,
                                        float* part) {
  uint32_t r[32];
  float v[32];
  if (any) {
    tmem_ld32(taddr + col, r);
    tmem_ld_wait();
  }
#pragma unroll
  for (int e = 0; e < 32; ++e) v[e] = any && use ? __uint_as_float(r[e]) * scale : 0.f;
  if (!live) return;
#pragma unroll
  for (int e = 0; e < 32; e += 8) {
    if (col + e >= dim) continue;
    if (!part) {
      st_global_v4(out + 2 * (col + e), pack8<BF16>(v + e));
    } else {
      *reinterpret_cast<float4*>(part + col + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      *reinterpret_cast<float4*>(part + col + e + 4) = make_float4(v[e + 4], v[e + 5], v[e + 6], v[e + 7]);
    }
  }
}

__device__ __forceinline__ uint8_t* row_of(const Results& f, int which, int64_t batch, int64_t token, int64_t head) {
  return static_cast<uint8_t*>(f.out[which]) + 2 * (batch * f.stride[which][0] + token * f.stride[which][1] + head * f.stride[which][2]);
}

// ---------------------------------------------------------------- dQ

template <int kDim>
struct QuerySmem {
  static constexpr int kK = 3, kV = 2;   // stages: a tile of keys stays for two products, one of values for one
  static constexpr int kQ = 0, kDo = tile_bytes(kDim), kKeys = 2 * tile_bytes(kDim), kValues = kKeys + kK * Form<kDim>::kStep;
  static constexpr int kBar = kValues + kV * Form<kDim>::kStep;
  // Q and dO; K full, empty; V full, empty; scores, dS (two each); dP full, empty; dQ; tail; drain
  static constexpr int kBars = 1 + 2 * kK + 2 * kV + 4 + 2 + 3, kTotal = kBar + kBars * 8 + 16 + 1024;
};

// TMEM by quarters: dQ, S in two buffers (dS over them), dP.
template <int kDim, bool BF16>
__device__ __forceinline__ void by_queries(const CUtensorMap& map_q, const CUtensorMap& map_k, const CUtensorMap& map_v, const CUtensorMap& map_do,
                                           const BackwardParams& f, const Results& out, const int index, const int split) {
  using L = QuerySmem<kDim>;
  using F = Form<kDim>;
  constexpr int kN = F::kN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_q = sbase + L::kBar, bar_kf = bar_q + 8, bar_ke = bar_kf + 8 * L::kK, bar_vf = bar_ke + 8 * L::kK;
  const uint32_t bar_ve = bar_vf + 8 * L::kV, bar_s = bar_ve + 8 * L::kV, bar_ds = bar_s + 16, bar_dpf = bar_ds + 16;
  const uint32_t bar_dpe = bar_dpf + 8, bar_dq = bar_dpe + 8, bar_tail = bar_dq + 8, bar_drain = bar_tail + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kBar + L::kBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const Params& a = f.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int packs = a.heads_q / a.pack;
  const int head = index % packs, batch = index / packs % (int)f.batch;
  const int block = a.q_blocks - 1 - index / (packs * (int)f.batch);   // the longest rows first
  const int key_head = a.pack > 1 ? head : head / a.group;
  const int token0 = block * a.tile_tokens;
  const int keys = keys_of(a, batch), start = start_of(a, batch);
  const int see = a.causal ? min(keys, max(0, start + min(token0 + a.tile_tokens, a.q_tokens))) : keys;
  const int tiles = (see + kN - 1) / kN, share = (tiles + out.splits - 1) / out.splits;
  const int first = min(tiles, split * share), n = min(tiles, first + share) - first;

  if (threadIdx.x == 0) {
    for (uint32_t b = bar_q; b <= bar_drain; b += 8)
      mbar_init(b, (b >= bar_ds && b < bar_dpf) || b == bar_dpe ? F::kRowWarps : 1);   // dS, dP empty: one arrival for each row warp
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == F::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), F::kColumns);
    tmem_relinquish();
  }
  tc_fence_before();
  wait_for_kernel_ahead();
  let_next_kernel_start();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto give_up = [&](uint32_t bits) {
    *abort_flag = 1;
    report_error(a.err, bits);
  };

  if (warp == F::kLoadWarp) {
    if (n > 0) {
      if (lane == 0) {
        mbar_arrive_expect_tx(bar_q, 2 * query_bytes<kDim>(a));
        load_queries<kDim, kTile, kN>(sbase + L::kQ, &map_q, a, a.q, token0, head, batch, bar_q);
        load_queries<kDim, kTile, kN>(sbase + L::kDo, &map_do, a, a.d_o, token0, head, batch, bar_q);
      }
      int kn = 0, vn = 0;   // tiles asked for
      for (int j = 0; j < n && !__any_sync(0xffffffffu, *abort_flag); ++j) {
        const int row = (first + j) * kN;
        const uint32_t ks = j % L::kK, vs = j % L::kV;
        if (!__all_sync(0xffffffffu, mbar_wait_backoff(bar_ke + 8 * ks, ((j / L::kK) & 1) ^ 1, 32))) {
          give_up(kErrWaitOperand);
          break;
        }
        const bool tail = row + kN > keys && keys < a.k_tokens;
        const uint32_t dst = sbase + L::kKeys + ks * F::kStep;
        if (lane == 0) load_keys<kDim, kN>(dst, &map_k, a.k, row, key_head, batch, tail ? bar_tail : bar_kf + 8 * ks);
        if (tail) {
          // keys behind the last one may be anything: dS is 0 there, and 0 times NaN is not
          if (!__all_sync(0xffffffffu, mbar_wait(bar_tail, 0))) {
            give_up(kErrWaitOperand);
            break;
          }
          clear_rows<kDim, kN>(dst, keys - row, lane);
          __syncwarp();
          if (lane == 0) mbar_arrive(bar_kf + 8 * ks);
        }
        ++kn;
        if (!__all_sync(0xffffffffu, mbar_wait_backoff(bar_ve + 8 * vs, ((j / L::kV) & 1) ^ 1, 32))) {
          give_up(kErrWaitOperand);
          break;
        }
        if (lane == 0) load_keys<kDim, kN>(sbase + L::kValues + vs * F::kStep, &map_v, a.v, row, key_head, batch, bar_vf + 8 * vs);
        ++vn;
        __syncwarp();
      }
      if (lane == 0) {   // never leave with a copy in flight
        mbar_wait(bar_q, 0);
        for (int i = max(0, kn - L::kK); i < kn; ++i) mbar_wait(bar_kf + 8 * (i % L::kK), (i / L::kK) & 1);
        for (int i = max(0, vn - L::kV); i < vn; ++i) mbar_wait(bar_vf + 8 * (i % L::kV), (i / L::kV) & 1);
      }
    }
  } else if (warp == F::kMmaWarp) {
    if (n > 0) {
      constexpr uint32_t kIdS = make_idesc_f16(128, kN, BF16, false, false), kIdQ = make_idesc_f16(128, kDim, BF16, false, true);
      bool bad = false;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!bad) bad = !__all_sync(0xffffffffu, mbar_wait(bar, parity));
        tc_fence_after();
        return !bad;
      };
      auto product = [&](uint32_t d, uint32_t x, uint32_t y) {
        const uint64_t xd = k_major(x), yd = k_major(y);
#pragma unroll
        for (int k = 0; k < kDim / 16; ++k) mma_f16_ss_warp(tmem + d, xd + k_major_step(k), yd + k_major_step(k), kIdS, k != 0);
      };
      auto scores = [&](int i) {
        if (!wait(bar_kf + 8 * (i % L::kK), (i / L::kK) & 1)) return;
        product(kN + (i & 1) * kN, sbase + L::kQ, sbase + L::kKeys + (i % L::kK) * F::kStep);
        mma_commit_warp(bar_s + 8 * (i & 1));
      };
      auto dp = [&](int i) {
        if (!wait(bar_vf + 8 * (i % L::kV), (i / L::kV) & 1)) return;
        product(3 * kN, sbase + L::kDo, sbase + L::kValues + (i % L::kV) * F::kStep);
        mma_commit_warp(bar_dpf);
        mma_commit_warp(bar_ve + 8 * (i % L::kV));
      };
      if (wait(bar_q, 0)) scores(0);
      if (!bad) dp(0);
      if (!bad && n > 1) scores(1);
      for (int j = 0; j < n && !bad; ++j) {
        if (j + 1 < n) {
          if (!wait(bar_dpe, j & 1)) break;
          dp(j + 1);
          if (bad) break;
        }
        if (!wait(bar_ds + 8 * (j & 1), (j >> 1) & 1)) break;
        const uint64_t kd = mn_major(sbase + L::kKeys + (j % L::kK) * F::kStep);
        const uint32_t ds = tmem + kN + (j & 1) * kN;
#pragma unroll
        for (int k = 0; k < kN / 16; ++k)   // 64 columns of dS at the start of each half of its scores
          mma_f16_ts_warp(tmem, ds + (k >> 2) * 64 + (k & 3) * 8, kd + mn_major_step(k), kIdQ, (k != 0) | (j != 0));
        mma_commit_warp(bar_ke + 8 * (j % L::kK));
        if (j + 2 < n) scores(j + 2);
        if (__any_sync(0xffffffffu, *abort_flag)) break;
      }
      mma_commit_warp(bar_dq);
      if (bad) give_up(kErrWaitMma);
      mma_commit_warp(bar_drain);
      mbar_wait(bar_drain, 0);
    }
  } else {
    const int half = warp >> 2, row = threadIdx.x & 127;
    const int token = token0 + row / a.pack;
    const int q_head = a.pack > 1 ? head * a.pack + row % a.pack : head;
    const bool live = row < a.tile_tokens * a.pack && token < a.q_tokens;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const float c = exponent_scale(a), sc = ds_scale<BF16>(f, batch, key_head), sc2 = sc * ex2(-kShift<BF16>);
    const int64_t at = ((int64_t)batch * packs + head) * f.rows + (int64_t)block * kTile + row;
    const float offset = f.offset[at], dsc = f.delta[at] * sc2;
    const uint64_t c2 = pair(c, c), offset2 = pair(offset, offset), sc22 = pair(sc2, sc2), dsc2 = pair(dsc, dsc);
    const int limit = a.causal ? min(keys, max(0, start + token + 1)) : keys;
    const int least = a.causal ? min(keys, max(0, start + token0 + 1)) : keys;
    bool bad = false;
    for (int j = 0; j < n; ++j) {
      const uint32_t ts = trow + kN + (j & 1) * kN + half * 64;
      const int key = (first + j) * kN + half * 64;
      const bool edge = key + 64 > least;
      bad = !__all_sync(0xffffffffu, mbar_wait(bar_s + 8 * (j & 1), (j >> 1) & 1));
      if (bad) break;
      tc_fence_after();
      uint32_t r[64];
      float p[64];
#pragma unroll
      for (int i = 0; i < 2; ++i) tmem_ld32(ts + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(r + 32 * i));
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 64; i += 2) {
        const uint64_t x = fma2(pair(r[i], r[i + 1]), c2, offset2);
        p[i] = ex2(low(x));
        p[i + 1] = ex2(high(x));
      }
      bad = !__all_sync(0xffffffffu, mbar_wait(bar_dpf, j & 1));
      if (bad) break;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 2; ++i) tmem_ld32(trow + 3 * kN + half * 64 + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(r + 32 * i));
      tmem_ld_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_dpe);
      if (edge) {
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (key + i >= limit) p[i] = 0.f, r[i] = 0u;
      }
      uint32_t ds[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const uint64_t x = mul2(pair(p[2 * i], p[2 * i + 1]), fma2(pair(r[2 * i], r[2 * i + 1]), sc22, dsc2));
        ds[i] = pack2<BF16>(low(x), high(x));
      }
      tmem_st32(ts, ds);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ds + 8 * (j & 1));
    }
    if (!bad && n > 0) bad = !__all_sync(0xffffffffu, mbar_wait(bar_dq, 0));
    if (bad) give_up(kErrWaitAccum);
    tc_fence_after();
    const int64_t out_row = ((int64_t)batch * a.heads_q + q_head) * a.q_tokens + token;
    uint8_t* to = row_of(out, 0, batch, token, q_head);
    float* part = out.splits > 1 ? out.part + (split * out.part_rows + out_row) * a.head_dim : nullptr;
#pragma unroll 1
    for (int i = half * 64; i < (half + 1) * 64; i += 32)
      store32<BF16>(trow, i, a.head_dim, n > 0 && !bad, true, live, a.scale / sc, to, part);
    tc_fence_before();
  }
  __syncthreads();
  if (warp == F::kMmaWarp) tmem_dealloc(tmem, F::kColumns);
}

// ---------------------------------------------------------------- dK, dV

template <int kDim>
struct KeySmem {
  static constexpr int kStep = Form<kDim>::kStep, kRowStep = Form<kDim>::kN * 8;
  static constexpr int kK = 0, kV = tile_bytes(kDim), kQ = 2 * tile_bytes(kDim), kDo = kQ + 2 * kStep;   // Q, dO: two stages
  static constexpr int kRow = kDo + 2 * kStep;   // two stages of offsets and D
  static constexpr int kBar = kRow + 2 * kRowStep;
  // K and V; Q full, empty; dO full, empty (two each); scores, p, dP, dS; out; drain
  static constexpr int kBars = 1 + 8 + 4 + 2, kTotal = kBar + kBars * 8 + 16 + 1024;
};

__device__ __forceinline__ float4 ld_shared_v4(uint32_t from) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(from));
  return v;
}

// Rows are keys here, columns queries.  TMEM by quarters: dV, dK, S (P over it), dP (dS over it).
template <int kDim, bool BF16>
__device__ __forceinline__ void by_keys(const CUtensorMap& map_q, const CUtensorMap& map_k, const CUtensorMap& map_v, const CUtensorMap& map_do,
                                        const BackwardParams& f, const Results& out, const int index, const int split) {
  using L = KeySmem<kDim>;
  using F = Form<kDim>;
  constexpr int kN = F::kN;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_kv = sbase + L::kBar, bar_qf = bar_kv + 8, bar_qe = bar_qf + 16, bar_of = bar_qe + 16, bar_oe = bar_of + 16;
  const uint32_t bar_s = bar_oe + 16, bar_p = bar_s + 8, bar_dp = bar_p + 8, bar_ds = bar_dp + 8, bar_out = bar_ds + 8;
  const uint32_t bar_drain = bar_out + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kBar + L::kBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const Params& a = f.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  const int key_head = index % a.heads_k, batch = index / a.heads_k % (int)f.batch;
  const int tile = index / (a.heads_k * (int)f.batch);   // causal: the first keys have the most queries, and come first
  const int key0 = tile * kTile, keys = keys_of(a, batch), start = start_of(a, batch);
  // tiles of queries: those from the first that sees one of the keys, of every pack of heads that reads them
  const int q_tiles = (int)(f.rows / kN);
  const int q_first = a.causal ? (int)min((int64_t)q_tiles, (int64_t)min(max(0, key0 - start), a.q_tokens) * a.pack / kN) : 0;
  const int each = key0 < keys ? q_tiles - q_first : 0, all = each * (a.group / a.pack);
  const int share = (all + out.splits - 1) / out.splits;
  const int first = min(all, split * share), n = min(all, first + share) - first;
  const int head0 = a.pack > 1 ? key_head : key_head * a.group;   // the first pack of heads

  if (threadIdx.x == 0) {
    for (uint32_t b = bar_kv; b <= bar_drain; b += 8) mbar_init(b, b == bar_p || b == bar_ds ? F::kRowWarps : b == bar_kv ? 2 : 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == F::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), F::kColumns);
    tmem_relinquish();
  }
  tc_fence_before();
  wait_for_kernel_ahead();
  let_next_kernel_start();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto give_up = [&](uint32_t bits) {
    *abort_flag = 1;
    report_error(a.err, bits);
  };

  if (warp == F::kLoadWarp) {
    if (n > 0) {
      if (lane == 0) {
        load_keys<kDim, kTile, kN>(sbase + L::kK, &map_k, a.k, key0, key_head, batch, bar_kv);
        // (the barrier counts two arrivals: each of the loads announces its own bytes)
        load_keys<kDim, kTile, kN>(sbase + L::kV, &map_v, a.v, key0, key_head, batch, bar_kv);
      }
      int qn = 0, on = 0;   // tiles asked for
      for (int j = 0; j < n && !__any_sync(0xffffffffu, *abort_flag); ++j) {
        const int head = head0 + (first + j) / each, qt = q_first + (first + j) % each;
        const uint32_t s = j & 1, parity = ((j >> 1) & 1) ^ 1;
        if (!__all_sync(0xffffffffu, mbar_wait_backoff(bar_qe + 8 * s, parity, 32))) {
          give_up(kErrWaitOperand);
          break;
        }
        if (lane == 0) {
          const int64_t at = ((int64_t)batch * (a.heads_q / a.pack) + head) * f.rows + (int64_t)qt * kN;
          mbar_arrive_expect_tx(bar_qf + 8 * s, query_bytes<kDim, kN>(a) + L::kRowStep);
          load_queries<kDim, kN>(sbase + L::kQ + s * F::kStep, &map_q, a, a.q, qt * (kN / a.pack), head, batch, bar_qf + 8 * s);
          bulk_load_1d(sbase + L::kRow + s * L::kRowStep, f.offset + at, L::kRowStep / 2, bar_qf + 8 * s);
          bulk_load_1d(sbase + L::kRow + s * L::kRowStep + L::kRowStep / 2, f.delta + at, L::kRowStep / 2, bar_qf + 8 * s);
        }
        ++qn;
        if (!__all_sync(0xffffffffu, mbar_wait_backoff(bar_oe + 8 * s, parity, 32))) {
          give_up(kErrWaitOperand);
          break;
        }
        if (lane == 0) {
          mbar_arrive_expect_tx(bar_of + 8 * s, query_bytes<kDim, kN>(a));
          load_queries<kDim, kN>(sbase + L::kDo + s * F::kStep, &map_do, a, a.d_o, qt * (kN / a.pack), head, batch, bar_of + 8 * s);
        }
        ++on;
        __syncwarp();
      }
      if (lane == 0) {   // never leave with a copy in flight
        mbar_wait(bar_kv, 0);
        for (int i = max(0, qn - 2); i < qn; ++i) mbar_wait(bar_qf + 8 * (i & 1), (i >> 1) & 1);
        for (int i = max(0, on - 2); i < on; ++i) mbar_wait(bar_of + 8 * (i & 1), (i >> 1) & 1);
      }
    }
  } else if (warp == F::kMmaWarp) {
    if (n > 0) {
      constexpr uint32_t kIdS = make_idesc_f16(128, kN, BF16, false, false), kIdK = make_idesc_f16(128, kDim, BF16, false, true);
      bool bad = false;
      auto wait = [&](uint32_t bar, uint32_t parity) {
        if (!bad) bad = !__all_sync(0xffffffffu, mbar_wait(bar, parity));
        tc_fence_after();
        return !bad;
      };
      // keys (values) times queries (dO): a tile of scores
      auto scores = [&](uint32_t d, uint32_t x, uint32_t y, uint32_t bar) {
        const uint64_t xd = k_major(sbase + x), yd = k_major(sbase + y);
#pragma unroll
        for (int k = 0; k < kDim / 16; ++k) mma_f16_ss_warp(tmem + d, xd + k_major_step(k), yd + k_major_step(k), kIdS, k != 0);
        mma_commit_warp(bar);
      };
      // what lies over the scores at `x` times queries (dO), added to the accumulator at `d`
      auto gather = [&](uint32_t d, uint32_t x, uint32_t y, int j) {
        const uint64_t yd = mn_major(sbase + y);
#pragma unroll
        for (int k = 0; k < kN / 16; ++k)
          mma_f16_ts_warp(tmem + d, tmem + x + (k >> 2) * 64 + (k & 3) * 8, yd + mn_major_step(k), kIdK, (k != 0) | (j != 0));
      };
      if (wait(bar_kv, 0) && wait(bar_qf, 0)) scores(2 * kN, L::kK, L::kQ, bar_s);
      if (!bad && wait(bar_of, 0)) scores(3 * kN, L::kV, L::kDo, bar_dp);
      for (int j = 0; j < n && !bad; ++j) {
        const uint32_t s = j & 1, next = s ^ 1, parity = ((j + 1) >> 1) & 1;
        if (!wait(bar_p, j & 1)) break;
        gather(0, 2 * kN, L::kDo + s * F::kStep, j);
        mma_commit_warp(bar_oe + 8 * s);
        if (j + 1 < n) {
          if (!wait(bar_qf + 8 * next, parity)) break;
          scores(2 * kN, L::kK, L::kQ + next * F::kStep, bar_s);
        }
        if (!wait(bar_ds, j & 1)) break;
        gather(kN, 3 * kN, L::kQ + s * F::kStep, j);
        mma_commit_warp(bar_qe + 8 * s);
        if (j + 1 < n) {
          if (!wait(bar_of + 8 * next, parity)) break;
          scores(3 * kN, L::kV, L::kDo + next * F::kStep, bar_dp);
        }
        if (__any_sync(0xffffffffu, *abort_flag)) break;
      }
      mma_commit_warp(bar_out);
      if (bad) give_up(kErrWaitMma);
      mma_commit_warp(bar_drain);
      mbar_wait(bar_drain, 0);
    }
  } else {
    const int half = warp >> 2, row = threadIdx.x & 127, key = key0 + row;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = trow + 2 * kN + half * 64, tdp = trow + 3 * kN + half * 64;
    const float c = exponent_scale(a), sc = ds_scale<BF16>(f, batch, key_head), sc2 = sc * ex2(-kShift<BF16>);
    const uint64_t c2 = pair(c, c), sc22 = pair(sc2, sc2);
    bool bad = false;
    for (int j = 0; j < n; ++j) {
      const int qt = q_first + (first + j) % each;
      // causal: the first of the tile's columns (queries, of several heads where packed) that sees this row's key
      int hidden = 0;
      if (a.causal) {
        const int64_t from = (int64_t)max(0, key - start) * a.pack - (int64_t)qt * kN - half * 64;
        hidden = (int)max((int64_t)0, min((int64_t)64, from));
      }
      const bool edge = __any_sync(0xffffffffu, hidden > 0);
      const uint32_t offset = sbase + L::kRow + (j & 1) * L::kRowStep + half * 256, delta = offset + 4 * kN;
      bad = !__all_sync(0xffffffffu, mbar_wait(bar_qf + 8 * (j & 1), (j >> 1) & 1) && mbar_wait(bar_s, j & 1));
      if (bad) break;
      tc_fence_after();
      uint32_t r[64];
      float p[64];
#pragma unroll
      for (int i = 0; i < 2; ++i) tmem_ld32(ts + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(r + 32 * i));
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 o = ld_shared_v4(offset + 16 * i);   // negative
        const uint64_t x = fma2(pair(r[4 * i], r[4 * i + 1]), c2, pair(o.x, o.y));
        const uint64_t y = fma2(pair(r[4 * i + 2], r[4 * i + 3]), c2, pair(o.z, o.w));
        p[4 * i] = ex2(low(x));
        p[4 * i + 1] = ex2(high(x));
        p[4 * i + 2] = ex2(low(y));
        p[4 * i + 3] = ex2(high(y));
      }
      if (edge) {
#pragma unroll
        for (int i = 0; i < 64; ++i)
          if (i < hidden) p[i] = 0.f;
      }
      uint32_t w[32];
#pragma unroll
      for (int i = 0; i < 32; ++i) w[i] = pack2<BF16>(p[2 * i], p[2 * i + 1]);
      tmem_st32(ts, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_p);
      bad = !__all_sync(0xffffffffu, mbar_wait(bar_dp, j & 1));
      if (bad) break;
      tc_fence_after();
#pragma unroll
      for (int i = 0; i < 2; ++i) tmem_ld32(tdp + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(r + 32 * i));
      tmem_ld_wait();
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float4 d = ld_shared_v4(delta + 16 * i);   // negative
        uint64_t x = add2(pair(r[4 * i], r[4 * i + 1]), pair(d.x, d.y)), y = add2(pair(r[4 * i + 2], r[4 * i + 3]), pair(d.z, d.w));
        if constexpr (!BF16) x = mul2(x, sc22), y = mul2(y, sc22);
        x = mul2(x, pair(p[4 * i], p[4 * i + 1]));
        y = mul2(y, pair(p[4 * i + 2], p[4 * i + 3]));
        w[2 * i] = pack2<BF16>(low(x), high(x));
        w[2 * i + 1] = pack2<BF16>(low(y), high(y));
      }
      tmem_st32(tdp, w);
      tmem_st_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(bar_ds);
    }
    if (!bad && n > 0) bad = !__all_sync(0xffffffffu, mbar_wait(bar_out, 0));
    if (bad) give_up(kErrWaitAccum);
    tc_fence_after();
    // with two warpgroups the first stores dV, the second dK
#pragma unroll 1
    for (int which = half; which < 2; which += F::kHalves) {
      uint8_t* to = row_of(out, which, batch, key, key_head);
      const int64_t out_row = ((int64_t)batch * a.heads_k + key_head) * a.k_tokens + key;
      float* part = out.splits > 1 ? out.part + ((2 * split + which) * out.part_rows + out_row) * a.head_dim : nullptr;
      const float scale = which ? a.scale / sc : ex2(-kShift<BF16>);
#pragma unroll 1
      for (int i = 0; i < kDim; i += 32)
        store32<BF16>(trow + which * kN, i, a.head_dim, n > 0 && !bad, key < keys, key < a.k_tokens, scale, to, part);
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == F::kMmaWarp) tmem_dealloc(tmem, F::kColumns);
}

// Blocks of both kinds in one launch, so that neither's last ones leave SMs idle: those by keys, whose walks over several
// heads' queries are the longest, come first.
template <int kDim, bool BF16>
__global__ void __launch_bounds__(Form<kDim>::kThreads, Form<kDim>::kBlocks)
    backward_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                    const __grid_constant__ CUtensorMap map_v, const __grid_constant__ CUtensorMap map_do,
                    const __grid_constant__ BackwardParams f) {
  const int by_key = f.keys.blocks * f.keys.splits, i = (int)blockIdx.x - by_key;
  if (i < 0)
    by_keys<kDim, BF16>(map_q, map_k, map_v, map_do, f, f.keys, blockIdx.x % f.keys.blocks, blockIdx.x / f.keys.blocks);
  else
    by_queries<kDim, BF16>(map_q, map_k, map_v, map_do, f, f.queries, i % f.queries.blocks, i / f.queries.blocks);
}

// ---------------------------------------------------------------- parts

// Parts added up in their order: a warp for each row of `outs` results of [batch][heads][tokens], four elements to a lane.
template <bool BF16>
__global__ void __launch_bounds__(128) sum_kernel(const __grid_constant__ Results f, int dim, int outs, int64_t heads, int64_t tokens) {
  const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  wait_for_kernel_ahead();
  if (at >= outs * f.part_rows) return;
  const int64_t which = at / f.part_rows, row = at % f.part_rows;
  using T = std::conditional_t<BF16, __nv_bfloat16, __half>;
  T* out = reinterpret_cast<T*>(row_of(f, (int)which, row / tokens / heads, row % tokens, row / tokens % heads));
  if (4 * lane >= dim) return;
  const float4* part = reinterpret_cast<const float4*>(f.part + (which * f.part_rows + row) * dim + 4 * lane);
  const int64_t step = outs * f.part_rows * dim / 4;
  float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 8
  for (int s = 0; s < f.splits; ++s) {
    const float4 u = part[s * step];
    v.x += u.x, v.y += u.y, v.z += u.z, v.w += u.w;
  }
  reinterpret_cast<uint2*>(out)[lane] = make_uint2(pack2<BF16>(v.x, v.y), pack2<BF16>(v.z, v.w));
}

// ---------------------------------------------------------------- host side

struct Shape {
  int pack, query_splits, key_splits;
  int64_t packs, rows, q_blocks, key_tiles;
  size_t offsets, norms, q_parts, parts;   // bytes of the workspace's regions; q_parts is the first of the parts
};

// Heads that share a key head are packed into a tile of queries where they fill it evenly.  Where blocks leave
// SMs idle a long walk is shared among several, four steps at least to each.
Shape shape_of(const cbr_attention_desc_t& d, bool may_pack) {
  Shape s{};
  const int64_t group = d.heads_q / d.heads_k;
  const int step = d.head_dim > 64 ? 128 : 64, blocks_to_sm = 128 / step;
  s.pack = may_pack && group <= step && (group & (group - 1)) == 0 ? (int)group : 1;
  s.packs = d.heads_q / s.pack;
  s.rows = (d.q_tokens * s.pack + kTile - 1) / kTile * kTile;
  s.q_blocks = s.rows / kTile;
  s.key_tiles = (d.k_tokens + kTile - 1) / kTile;
  const int64_t blocks = s.q_blocks * s.packs * d.batch + s.key_tiles * d.heads_k * d.batch;
  auto splits = [&](int64_t walk) {
    if (walk < 12 * step) return 1;   // the sum of the parts costs about as much as a few steps
    return (int)std::max<int64_t>(1, std::min<int64_t>(kSms * blocks_to_sm / std::max<int64_t>(blocks, 1), walk / step / 4));
  };
  s.query_splits = splits(d.k_tokens);
  s.key_splits = splits(s.rows * (group / s.pack));
  s.offsets = (size_t)d.batch * s.packs * s.rows * 4;
  s.norms = align256((size_t)d.batch * d.heads_k * 8);
  const size_t q_part = s.query_splits > 1 ? (size_t)s.query_splits * d.batch * d.heads_q * d.q_tokens : 0;
  const size_t k_part = s.key_splits > 1 ? (size_t)s.key_splits * 2 * d.batch * d.heads_k * d.k_tokens : 0;
  s.q_parts = q_part * d.head_dim * 4;
  s.parts = s.q_parts + k_part * d.head_dim * 4;
  return s;
}

// (heads of q or dO that repeat have no axis to pack)
bool may_pack(const cbr_attention_desc_t& d) { return d.q_stride[2] != 0 && d.do_stride[2] != 0; }

size_t total(const Shape& s) { return 2 * align256(s.offsets) + s.norms + s.parts; }

template <int kDim, bool BF16>
int launch(const AttentionArgs& g, cudaStream_t st) {
  const cbr_attention_desc_t& d = g.d;
  const Shape s = shape_of(d, may_pack(d));
  uint8_t* ws = static_cast<uint8_t*>(g.ws);
  PrepareParams pre{};
  BackwardParams& f = pre.f;
  f.p = params_of(g, s.pack);
  f.p.q_blocks = (int)s.q_blocks;
  pre.offset = reinterpret_cast<float*>(ws);
  pre.delta = reinterpret_cast<float*>(ws + align256(s.offsets));
  pre.norms = reinterpret_cast<uint32_t*>(ws + 2 * align256(s.offsets));
  f.offset = pre.offset;
  f.delta = pre.delta;
  f.norms = pre.norms;
  f.rows = s.rows;
  f.batch = d.batch;
  if (d.q_tokens && d.k_tokens) {
    pre.d_o = g.d_o;
    pre.o = g.o;
    pre.v = g.v;
    pre.lse = g.lse;
    for (int i = 0; i < 3; ++i) pre.do_stride[i] = d.do_stride[i], pre.o_stride[i] = d.o_stride[i], pre.v_stride[i] = d.v_stride[i];
    pre.query_blocks = d.batch * s.packs * (s.rows / kPrepareRows<kDim>);
    int64_t blocks = pre.query_blocks;
    if constexpr (!BF16) {
      if (cudaMemsetAsync(pre.norms, 0, (size_t)d.batch * d.heads_k * 8, st) != cudaSuccess) return CBR_ERR_CUDA;
      blocks += d.batch * d.heads_k * ((d.k_tokens + kPrepareRows<kDim> - 1) / kPrepareRows<kDim>);
    }
    prepare_kernel<kDim, BF16><<<(unsigned)blocks, 256, 0, st>>>(pre);
  }
  // where one side is empty nothing is loaded, and the maps of the other stand in for its own
  CUtensorMap q, k, v, d_o;
  cbr_attention_desc_t e = d;
  const void *pq = g.q, *pdo = g.d_o, *pk = g.k, *pv = g.v;
  if (!d.q_tokens) {
    e.q_tokens = 1, pq = pdo = g.k;
    for (int i = 0; i < 3; ++i) e.q_stride[i] = e.do_stride[i] = 0;
  }
  if (!d.k_tokens) {
    pk = pv = g.q;
    for (int i = 0; i < 3; ++i) e.k_stride[i] = e.v_stride[i] = 0;
  }
  constexpr int kN = Form<kDim>::kN, kThreads = Form<kDim>::kThreads;
  if (!query_map(&q, e, pq, e.q_stride, s.pack, kN) || !query_map(&d_o, e, pdo, e.do_stride, s.pack, kN) ||
      !key_map(&k, e, pk, e.k_stride, kN) || !key_map(&v, e, pv, e.v_stride, kN))
    return CBR_ERR_CUDA;
  uint8_t* parts = ws + 2 * align256(s.offsets) + s.norms;
  f.queries = Results{{g.dq, nullptr}, {}, reinterpret_cast<float*>(parts), d.batch * d.heads_q * d.q_tokens, s.query_splits,
                      (int)(s.q_blocks * s.packs * d.batch)};
  f.keys = Results{{g.dv, g.dk}, {}, reinterpret_cast<float*>(parts + s.q_parts), d.batch * d.heads_k * d.k_tokens, s.key_splits,
                   (int)(s.key_tiles * d.heads_k * d.batch)};
  for (int i = 0; i < 3; ++i) f.queries.stride[0][i] = d.dq_stride[i], f.keys.stride[0][i] = d.dv_stride[i], f.keys.stride[1][i] = d.dk_stride[i];
  const auto kern = &backward_kernel<kDim, BF16>;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), 227 * 1024)) return CBR_ERR_CUDA;
  constexpr int kSmem = std::max(QuerySmem<kDim>::kTotal, KeySmem<kDim>::kTotal);
  bool fine = launch_behind(kern, dim3((unsigned)(f.keys.blocks * f.keys.splits + f.queries.blocks * f.queries.splits)), kThreads, kSmem, st,
                            q, k, v, d_o, f);
  auto sum = [&](const Results& r, int outs, int64_t heads, int64_t tokens) {
    if (r.splits > 1 && fine)
      fine = launch_behind(&sum_kernel<BF16>, dim3((unsigned)((outs * r.part_rows + 3) / 4)), 128, 0, st, r, d.head_dim, outs, heads, tokens);
  };
  sum(f.queries, 1, d.heads_q, d.q_tokens);
  sum(f.keys, 2, d.heads_k, d.k_tokens);
  if (!fine) return CBR_ERR_CUDA;
  return cudaGetLastError() == cudaSuccess ? CBR_OK : CBR_ERR_CUDA;
}

}  // namespace
}  // namespace att

size_t attention_backward_ws(const cbr_attention_desc_t& d) {
  return std::max(att::total(att::shape_of(d, true)), att::total(att::shape_of(d, false)));
}

int launch_attention_backward(const AttentionArgs& a, cudaStream_t st) {
  const bool bf16 = a.d.dtype == CBR_BF16;
  if (a.d.head_dim > 64) return bf16 ? att::launch<128, true>(a, st) : att::launch<128, false>(a, st);
  return bf16 ? att::launch<64, true>(a, st) : att::launch<64, false>(a, st);
}

}  // namespace cbr
