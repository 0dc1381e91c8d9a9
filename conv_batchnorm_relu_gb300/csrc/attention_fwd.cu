// Attention forward (declared in include/cbr.h) on the tensor cores.
//
// A block takes one or two tiles of 128 queries of a head (or of the heads that share a key head) and walks
// over the keys in tiles of 128, once: S = Q K^T into TMEM; a warpgroup for each query tile, a thread for each
// query, takes the scores to registers, keeps the running maximum m and the sum l of exp2((s - m) c),
// c = scale log2(e), and writes these p, rounded to the storage type, over S; O += P V with P read from
// TMEM.  While one tile's scores are exponentiated the tensor cores work on the other's products.
//   m moves only when a score passes it by 8 in the exponent (p stays below 2^8): O is rescaled then, which is
// rare after the first tiles.  In f16 p is 2^6 times as large, which keeps small p's out of the subnormals.
//   Few queries on long keys: the walk is shared among blocks, whose results a second kernel joins by their sums.
//   Warps: four for each tile's rows, one loads (TMA), one issues the products.  TMEM: the tiles' scores (128 columns
// each; P in the first 64 of each), then their O.
//   Bound by the products where rows are long (2 of 8192 tokens, 16 heads of 128, bf16: 340 us, 85% of the rate that a
// library's matrix product has here).  Heads of 64 and less: by the row warps' chain of a tile (scores to registers,
// maximum, exponentials, p back), two warps to a scheduler: tensor cores, the exponentials' pipe and the issue slots
// are busy 35, 35 and 41% of the time (1 of 16384, 2 heads, bf16: 174 us), and with rows of 196 tokens 13, 15 and 31%.  Few
// queries: the keys' and values' bytes, a tile ahead at most, and the join (4 of 16384: 27 us, 3.7 TB/s).
#include <algorithm>

#include "attention.cuh"
#include "cbr_internal.h"

namespace cbr {
namespace att {
namespace {

constexpr float kMove = 8.f;   // how far a score may pass the running maximum, as an exponent of 2

// By the tiles of queries that a block takes.  Two: the block has an SM to itself, and its row warps take registers from
// the others (two warps only give theirs).  One: half of TMEM, two blocks to an SM, one's exponentials over the
// other's products.
template <int kTiles>
struct Form {
  static constexpr int kRowWarps = 4 * kTiles, kLoadWarp = kRowWarps, kMmaWarp = kRowWarps + 1;
  static constexpr int kThreads = kTiles == 2 ? 384 : 192, kBlocks = 3 - kTiles;
  static constexpr uint32_t kColumns = 256 * kTiles, kO = 128 * kTiles;   // of TMEM: all, and where O is
};

template <int kDim, int kTiles>
struct Smem {
  static constexpr int kStages = kTiles == 2 ? (kDim == 128 ? 5 : 8) : (kDim == 128 ? 2 : 5);   // of keys and values in turn
  static constexpr int kQ = 0, kKv = kTiles * tile_bytes(kDim), kBar = kKv + kStages * tile_bytes(kDim);
  // barriers: Q; K/V full, empty; scores full, p full (two halves), O full for each query tile; tail; drain
  static constexpr int kBars = 1 + 2 * kStages + 4 * kTiles + 2, kTotal = kBar + kBars * 8 + 16 + 1024;
};

struct ForwardParams {
  Params p;
  void* o;
  float* lse;            // may be null
  int64_t o_stride[3];
  float* part_o;         // splits > 1: [split][row][head_dim] normalised partial results, rows as in lse
  float* part_lse;       // [split][row]: log2 of the partial sums
};

template <int kDim, int kTiles, bool BF16>
__global__ void __launch_bounds__(Form<kTiles>::kThreads, Form<kTiles>::kBlocks)
    forward_kernel(const __grid_constant__ CUtensorMap map_q, const __grid_constant__ CUtensorMap map_k,
                   const __grid_constant__ CUtensorMap map_v, const __grid_constant__ ForwardParams f) {
  using L = Smem<kDim, kTiles>;
  using F = Form<kTiles>;
  constexpr float kShift = BF16 ? 0.f : 6.f;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~static_cast<uintptr_t>(1023));
  const uint32_t sbase = smem_u32(smem);
  const uint32_t bar_q = sbase + L::kBar, bar_full = bar_q + 8, bar_empty = bar_full + 8 * L::kStages;
  const uint32_t bar_s = bar_empty + 8 * L::kStages, bar_p = bar_s + 8 * kTiles, bar_o = bar_p + 16 * kTiles, bar_tail = bar_o + 8 * kTiles;
  const uint32_t bar_drain = bar_tail + 8;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + L::kBar + L::kBars * 8);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  const Params& a = f.p;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  // the block's place: heads fastest, so that blocks that run together share keys; the longest rows first
  const int packs = a.heads_q / a.pack;
  const int head = blockIdx.x % packs, batch = blockIdx.x / packs % (gridDim.x / packs / a.q_blocks);
  const int block = a.q_blocks - 1 - blockIdx.x / (gridDim.x / a.q_blocks);
  const int key_head = a.pack > 1 ? head : head / a.group;
  const int token0 = block * kTiles * a.tile_tokens;
  const int keys = keys_of(a, batch), start = start_of(a, batch);
  // tiles of keys that each query tile needs: those that its last query sees
  int end[kTiles], widest = 0;
#pragma unroll
  for (int t = 0; t < kTiles; ++t) {
    const int first = token0 + t * a.tile_tokens;
    int see = 0;
    if (first < a.q_tokens)
      see = a.causal ? min(keys, max(0, start + min(first + a.tile_tokens, a.q_tokens))) : keys;
    end[t] = (see + kTile - 1) / kTile;
    widest = max(widest, end[t]);
  }
  const int share = (widest + a.splits - 1) / a.splits, begin = blockIdx.y * share;
#pragma unroll
  for (int t = 0; t < kTiles; ++t) end[t] = max(begin, min(end[t], begin + share));
  const int last = max(end[0], end[kTiles - 1]);

  if (threadIdx.x == 0) {
    mbar_init(bar_q, 1);
    for (int i = 0; i < L::kStages; ++i) {
      mbar_init(bar_full + 8 * i, 1);
      mbar_init(bar_empty + 8 * i, 1);
    }
    for (int t = 0; t < kTiles; ++t) {
      mbar_init(bar_s + 8 * t, 1);
      mbar_init(bar_p + 16 * t, 4);
      mbar_init(bar_p + 16 * t + 8, 4);
      mbar_init(bar_o + 8 * t, 1);
    }
    mbar_init(bar_tail, 1);
    mbar_init(bar_drain, 1);
    *abort_flag = 0;
    fence_mbarrier_init();
  }
  if (warp == F::kMmaWarp) {
    tmem_alloc(smem_u32(tmem_slot), F::kColumns);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  auto give_up = [&](uint32_t bits) {
    *abort_flag = 1;
    report_error(a.err, bits);
  };

  if (warp >= F::kRowWarps) {
  if constexpr (kTiles == 2) give_registers<80>();
  if (warp == F::kLoadWarp) {
    if (last > begin) {
      if (lane == 0) {
        int tiles = 0;
        for (int t = 0; t < kTiles; ++t) tiles += end[t] > begin;
        mbar_arrive_expect_tx(bar_q, tiles * query_bytes<kDim>(a));
        for (int t = 0; t < kTiles; ++t)
          if (end[t] > begin)
            load_queries<kDim>(sbase + L::kQ + t * tile_bytes(kDim), &map_q, a, a.q, token0 + t * a.tile_tokens, head, batch, bar_q);
      }
      uint32_t it = 0;
      for (int j = begin; j < last && !__any_sync(0xffffffffu, *abort_flag); ++j) {
        for (int kv = 0; kv < 2; ++kv, ++it) {
          const uint32_t s = it % L::kStages, ph = (it / L::kStages) & 1;
          const uint32_t dst = sbase + L::kKv + s * tile_bytes(kDim);
          if (!__all_sync(0xffffffffu, mbar_wait_backoff(bar_empty + 8 * s, ph ^ 1, 32))) {
            give_up(kErrWaitOperand);
            break;
          }
          const bool tail = kv == 1 && (j + 1) * kTile > keys && keys < a.k_tokens;
          const uint32_t bar = tail ? bar_tail : bar_full + 8 * s;
          if (lane == 0) load_keys<kDim>(dst, kv ? &map_v : &map_k, kv ? a.v : a.k, j * kTile, key_head, batch, bar);
          if (tail) {
            // values behind the last key may be anything: p is 0 there, and 0 times NaN is not
            if (!__all_sync(0xffffffffu, mbar_wait(bar_tail, 0))) {
              give_up(kErrWaitOperand);
              break;
            }
            clear_rows<kDim>(dst, keys - j * kTile, lane);
            __syncwarp();
            if (lane == 0) mbar_arrive(bar_full + 8 * s);
          }
          __syncwarp();
        }
      }
      // never leave with a copy in flight
      if (lane == 0) {
        mbar_wait(bar_q, 0);
        for (uint32_t i = it > L::kStages ? it - L::kStages : 0; i < it; ++i)
          mbar_wait(bar_full + 8 * (i % L::kStages), (i / L::kStages) & 1);
      }
    }
  } else if (warp == F::kMmaWarp) {
    if (last > begin) {
      constexpr uint32_t kIdS = make_idesc_f16(128, 128, BF16, false, false), kIdO = make_idesc_f16(128, kDim, BF16, false, true);
      bool bad = !__all_sync(0xffffffffu, mbar_wait(bar_q, 0));
      uint32_t done = 0;   // stages taken
      auto full = [&](uint32_t i) {
        if (bad) return;
        bad = !__all_sync(0xffffffffu, mbar_wait(bar_full + 8 * (i % L::kStages), (i / L::kStages) & 1));
        tc_fence_after();
      };
      auto scores = [&](int t, uint32_t i) {
        const uint64_t qd = k_major(sbase + L::kQ + t * tile_bytes(kDim));
        const uint64_t kd = k_major(sbase + L::kKv + (i % L::kStages) * tile_bytes(kDim));
#pragma unroll
        for (int k = 0; k < kDim / 16; k += 4) mma_f16_ss_slab(tmem + t * 128, qd + k_major_step(k), kd + k_major_step(k), kIdS, k != 0);
        mma_commit_warp(bar_s + 8 * t);
      };
      full(0);
      for (int t = 0; t < kTiles && !bad; ++t)
        if (end[t] > begin) scores(t, 0);
      if (!bad) mma_commit_warp(bar_empty);
      for (int j = begin; j < last && !bad; ++j) {
        const uint32_t v_at = done + 1, k_next = done + 2;
        const uint32_t ph = (j - begin) & 1;
        full(v_at);
        for (int t = 0; t < kTiles && !bad; ++t) {
          if (j >= end[t]) continue;
          const uint64_t vd = mn_major(sbase + L::kKv + (v_at % L::kStages) * tile_bytes(kDim));
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            if (!bad) bad = !__all_sync(0xffffffffu, mbar_wait(bar_p + 16 * t + 8 * half, ph));
            if (bad) break;
            tc_fence_after();
            mma_f16_ts_slab(tmem + F::kO + t * kDim, tmem + t * 128 + 32 * half, vd + mn_major_step(4 * half), kIdO, (half != 0) | (j != begin));
          }
          if (bad) break;
          if (t == kTiles - 1 || j >= end[kTiles - 1]) mma_commit_warp(bar_empty + 8 * (v_at % L::kStages));
          if (j + 1 < end[t]) {
            if (t == 0 || end[0] <= j + 1) full(k_next);
            if (bad) break;
            scores(t, k_next);
          } else {
            mma_commit_warp(bar_o + 8 * t);
          }
        }
        if (bad) break;
        if (j + 1 < last) mma_commit_warp(bar_empty + 8 * (k_next % L::kStages));
        done += 2;
        if (__any_sync(0xffffffffu, *abort_flag)) break;
      }
      if (bad) give_up(kErrWaitMma);
      mma_commit_warp(bar_drain);
      mbar_wait(bar_drain, 0);
    }
  }
  } else {
    if constexpr (kTiles == 2) take_registers<208>();
    const int t = warp >> 2, row = threadIdx.x & 127;
    const int token = token0 + t * a.tile_tokens + row / a.pack;
    const int q_head = a.pack > 1 ? head * a.pack + row % a.pack : head;
    const bool live = row < a.tile_tokens * a.pack && token < a.q_tokens;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t ts = trow + t * 128, to = trow + F::kO + t * kDim;
    const float c = exponent_scale(a);
    // the first key that this query does not see, and one for the whole tile
    const int limit = a.causal ? min(keys, max(0, start + token + 1)) : keys;
    const int least = a.causal ? min(keys, max(0, start + token0 + t * a.tile_tokens + 1)) : keys;
    float m = -INFINITY, l = 0.f;
    bool bad = false;
    for (int j = begin; j < end[t]; ++j) {
      if (!__all_sync(0xffffffffu, mbar_wait(bar_s + 8 * t, (j - begin) & 1))) {
        give_up(kErrWaitAccum);
        bad = true;
        break;
      }
      tc_fence_after();
      uint32_t r[128];
#pragma unroll
      for (int i = 0; i < 4; ++i) tmem_ld32(ts + 32 * i, *reinterpret_cast<uint32_t(*)[32]>(r + 32 * i));
      tmem_ld_wait();
      if ((j + 1) * kTile > least) {
        const int left = limit - j * kTile;
#pragma unroll
        for (int i = 0; i < 128; ++i)
          if (i >= left) r[i] = 0xff800000u;
      }
      float top[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
      for (int i = 0; i < 128; i += 2) top[i / 2 & 3] = max3(top[i / 2 & 3], __uint_as_float(r[i]), __uint_as_float(r[i + 1]));
      const float most = fmaxf(max3(top[0], top[1], top[2]), top[3]);
      const bool move = (most - m) * c > kMove && m != -INFINITY;
      if (__any_sync(0xffffffffu, move)) {
        // O is complete up to the tile before: its products were issued before these scores'
        const float keep = move ? ex2((m - most) * c) : 1.f;
        if (move) m = most;
        l *= keep;
#pragma unroll 1
        for (int i = 0; i < kDim; i += 32) {
          uint32_t v[32];
          tmem_ld32(to + i, v);
          tmem_ld_wait();
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) * keep);
          tmem_st32(to + i, v);
        }
      }
      if (m == -INFINITY) m = most;
      const float base = kShift - (m == -INFINITY ? 0.f : m * c);
      const uint64_t c2 = pair(c, c), base2 = pair(base, base);
      uint64_t sum[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < 2; ++i) {   // the products start with the first half while the second is worked on
        uint32_t p[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          const uint64_t x = fma2(pair(r[64 * i + 2 * e], r[64 * i + 2 * e + 1]), c2, base2);
          const float lo = ex2(low(x)), hi = ex2(high(x));
          sum[e & 1] = add2(sum[e & 1], pair(lo, hi));
          p[e] = pack2<BF16>(lo, hi);
        }
        tmem_st32(ts + 32 * i, p);
        tmem_st_wait();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar_p + 16 * t + 8 * i);
      }
      const uint64_t both = add2(sum[0], sum[1]);
      l += low(both) + high(both);
    }
    const bool any = end[t] > begin && !bad;
    if (any && !mbar_wait(bar_o + 8 * t, 0)) give_up(kErrWaitAccum);
    tc_fence_after();
    const int64_t at = ((int64_t)batch * a.heads_q + q_head) * a.q_tokens + token;
    const bool whole = a.splits == 1;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint8_t* out = static_cast<uint8_t*>(f.o) + 2 * (batch * f.o_stride[0] + (int64_t)token * f.o_stride[1] + q_head * f.o_stride[2]);
    const int64_t rows = (int64_t)gridDim.x / packs / a.q_blocks * a.heads_q * a.q_tokens;
    float* part = whole ? nullptr : f.part_o + (blockIdx.y * rows + at) * a.head_dim;
#pragma unroll 1
    for (int i = 0; i < a.head_dim; i += 32) {
      uint32_t r[32];
      float v[32];
      if (any) {   // the same in the whole warp
        tmem_ld32(to + i, r);
        tmem_ld_wait();
      }
#pragma unroll
      for (int e = 0; e < 32; ++e) v[e] = any && l != 0.f ? __uint_as_float(r[e]) * inv : 0.f;
      if (!live) continue;
#pragma unroll
      for (int e = 0; e < 32; e += 8) {
        if (i + e >= a.head_dim) continue;
        if (whole) {
          st_global_v4(out + 2 * (i + e), pack8<BF16>(v + e));
        } else {
          *reinterpret_cast<float4*>(part + i + e) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
          *reinterpret_cast<float4*>(part + i + e + 4) = make_float4(v[e + 4], v[e + 5], v[e + 6], v[e + 7]);
        }
      }
    }
    if (live) {
      const float log2_sum = l == 0.f ? -INFINITY : m * c + (log2f(l) - kShift);
      if (!whole) f.part_lse[blockIdx.y * rows + at] = log2_sum;
      else if (f.lse) f.lse[at] = log2_sum * kLn2;
    }
    tc_fence_before();
  }
  __syncthreads();
  if (warp == F::kMmaWarp) tmem_dealloc(tmem, F::kColumns);
}

constexpr int kMostSplits = 64;

// The parts of a query's result, joined in their order: a warp for each query, four elements to a lane.
template <bool BF16>
__global__ void __launch_bounds__(128) join_kernel(const __grid_constant__ ForwardParams f, int64_t rows) {
  const Params& a = f.p;
  const int64_t row = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31;
  if (row >= rows) return;
  // the weights by lanes, at most kMostSplits
  float lse[kMostSplits / 32], most = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < kMostSplits / 32; ++i) {
    lse[i] = lane + 32 * i < a.splits ? f.part_lse[(lane + 32 * i) * rows + row] : -INFINITY;
    most = tok::Max::of(most, lse[i]);
  }
  most = tok::warp_max(most);
  const float base = most == -INFINITY ? 0.f : most;
#pragma unroll
  for (int i = 0; i < kMostSplits / 32; ++i) sum += lse[i] = ex2(lse[i] - base);
  sum = tok::warp_reduce<tok::Sum>(sum);
  const bool in = 4 * lane < a.head_dim;
  const float4* part = reinterpret_cast<const float4*>(f.part_o + row * a.head_dim + (in ? 4 * lane : 0));
  const int64_t step = rows * a.head_dim / 4;
  float v[4] = {};
#pragma unroll
  for (int i = 0; i < kMostSplits / 32; ++i) {
    for (int first = 32 * i; first < min(a.splits, 32 * i + 32); first += 8) {   // eight loads at a time
      float4 o[8];
#pragma unroll
      for (int s = 0; s < 8; ++s) o[s] = first + s < a.splits ? part[(first + s) * step] : make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int s = 0; s < 8; ++s) {
        const float w = __shfl_sync(0xffffffffu, lse[i], (first + s) & 31);
        v[0] = fmaf(w, o[s].x, v[0]);
        v[1] = fmaf(w, o[s].y, v[1]);
        v[2] = fmaf(w, o[s].z, v[2]);
        v[3] = fmaf(w, o[s].w, v[3]);
      }
    }
  }
  const float inv = sum == 0.f ? 0.f : 1.f / sum;
  const int64_t token = row % a.q_tokens, h = row / a.q_tokens % a.heads_q, b = row / a.q_tokens / a.heads_q;
  uint8_t* out = static_cast<uint8_t*>(f.o) + 2 * (b * f.o_stride[0] + token * f.o_stride[1] + h * f.o_stride[2] + 4 * lane);
  if (in) *reinterpret_cast<uint2*>(out) = make_uint2(pack2<BF16>(v[0] * inv, v[1] * inv), pack2<BF16>(v[2] * inv, v[3] * inv));
  if (f.lse && lane == 0) f.lse[row] = (base + log2f(sum)) * kLn2;
}

int64_t rows_of(const cbr_attention_desc_t& d) { return d.batch * d.heads_q * d.q_tokens; }

struct Shape {
  int pack, tiles, splits;
  int64_t q_blocks, packs;
};

// How the queries are laid over blocks.  Heads that share a key head are packed into a tile where that leaves at
// most an eighth of its rows empty, or where all the queries there are fit one tile.  Two tiles to a block overlap one's
// exponentials with the other's products; a block has an SM to itself, so one tile each is taken where two would
// leave SMs without a block.  Where blocks leave SMs idle a long walk over the keys is shared among
// several.
// (Heads of q that repeat have no axis to pack.)
Shape shape_of(const cbr_attention_desc_t& d, bool may_pack) {
  Shape s{};
  const int64_t group = d.heads_q / d.heads_k;
  s.pack = group > 1 && group <= kTile && may_pack && (kTile / group * group >= 112 || group * d.q_tokens <= kTile) ? (int)group : 1;
  s.packs = d.heads_q / s.pack;
  const int64_t tiles = (d.q_tokens + kTile / s.pack - 1) / (kTile / s.pack);
  s.tiles = (tiles + 1) / 2 * s.packs * d.batch >= kSms ? 2 : 1;
  s.q_blocks = (tiles + s.tiles - 1) / s.tiles;
  const int64_t blocks = s.q_blocks * s.packs * d.batch, key_tiles = (d.k_tokens + kTile - 1) / kTile;
  // A tile takes a block that is alone about 1.4 us; the join 3 us for a few rows, 6 for ten thousand (8 tiles of one row:
  // 14.6 us in one block, 10.3 in four; 7 tiles of 9408 rows: 12.4 and, in three, 17).
  const bool few = rows_of(d) <= 2048;
  if (s.tiles == 1 && key_tiles >= (few ? 6 : 12))
    s.splits = (int)std::min<int64_t>({2 * kSms / std::max<int64_t>(blocks, 1), key_tiles / (few ? 2 : 4), kMostSplits});
  s.splits = std::max(1, s.splits);
  return s;
}

template <int kDim, int kTiles, bool BF16>
int launch(const AttentionArgs& g, const Shape& s, cudaStream_t st) {
  const cbr_attention_desc_t& d = g.d;
  ForwardParams f{};
  f.p = params_of(g, s.pack);
  f.p.q_blocks = (int)s.q_blocks;
  f.p.splits = s.splits;
  f.o = g.o;
  f.lse = g.lse;
  for (int i = 0; i < 3; ++i) f.o_stride[i] = d.o_stride[i];
  const int64_t rows = rows_of(d);
  if (s.splits > 1) {
    f.part_o = static_cast<float*>(g.ws);
    f.part_lse = f.part_o + s.splits * rows * d.head_dim;
  }
  CUtensorMap q, k, v;
  // no keys: nothing is loaded, and the maps of q stand in for theirs
  if (!query_map(&q, d, g.q, d.q_stride, s.pack) || !key_map(&k, d, d.k_tokens ? g.k : g.q, d.k_tokens ? d.k_stride : d.q_stride) ||
      !key_map(&v, d, d.k_tokens ? g.v : g.q, d.k_tokens ? d.v_stride : d.q_stride))
    return CBR_ERR_CUDA;
  const auto kern = &forward_kernel<kDim, kTiles, BF16>;
  if (!ensure_smem_attr(reinterpret_cast<const void*>(kern), 227 * 1024)) return CBR_ERR_CUDA;
  kern<<<dim3((unsigned)(s.q_blocks * s.packs * d.batch), s.splits), Form<kTiles>::kThreads, Smem<kDim, kTiles>::kTotal, st>>>(q, k, v, f);
  if (s.splits > 1) join_kernel<BF16><<<(unsigned)((rows + 3) / 4), 128, 0, st>>>(f, rows);
  return cudaGetLastError() == cudaSuccess ? CBR_OK : CBR_ERR_CUDA;
}

}  // namespace
}  // namespace att

size_t attention_forward_ws(const cbr_attention_desc_t& d) {
  const int splits = std::max(att::shape_of(d, true).splits, att::shape_of(d, false).splits);
  return splits > 1 ? (size_t)splits * att::rows_of(d) * (d.head_dim + 1) * 4 : 0;
}

int launch_attention(const AttentionArgs& a, cudaStream_t st) {
  const att::Shape s = att::shape_of(a.d, a.d.q_stride[2] != 0);
  auto by_type = [&](auto dim, auto tiles) {
    constexpr int kDim = decltype(dim)::value, kTiles = decltype(tiles)::value;
    return a.d.dtype == CBR_BF16 ? att::launch<kDim, kTiles, true>(a, s, st) : att::launch<kDim, kTiles, false>(a, s, st);
  };
  using One = std::integral_constant<int, 1>;
  using Two = std::integral_constant<int, 2>;
  if (a.d.head_dim > 64) return s.tiles == 2 ? by_type(std::integral_constant<int, 128>{}, Two{}) : by_type(std::integral_constant<int, 128>{}, One{});
  return s.tiles == 2 ? by_type(std::integral_constant<int, 64>{}, Two{}) : by_type(std::integral_constant<int, 64>{}, One{});
}

}  // namespace cbr
