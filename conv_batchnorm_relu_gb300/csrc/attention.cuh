// What the attention kernels share: tiles, masks, the load of keys and values, TMEM rows.
//
// Every kernel works on tiles of 128 tokens of one head (the backward's walks over heads of 64 take steps of 64).  A tile in
// shared memory is kDim / 64 slabs of [its rows][128 bytes] in the 128-byte swizzle, as the tensor maps write them; it serves as a K-major
// operand (rows along M or N, the head's elements along K) and as an MN-major one (rows along K).  Heads of
// up to 64 (128) elements fill kDim = 64 (128); the maps fill the rest with zeros.
#pragma once
#include <cuda.h>

#include <algorithm>

#include "cbr_internal.h"
#include "common.cuh"
#include "follow.cuh"
#include "ptx_rows.cuh"
#include "token_ops.cuh"
#include "trunk_ops.h"

namespace cbr {
namespace att {

constexpr int kTile = 128;
constexpr int64_t kSms = 152;        // of the device that the rules on blocks are made for
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

__host__ __device__ constexpr int tile_bytes(int dim) { return kTile * dim * 2; }
constexpr int kSlab = kTile * 128;   // bytes of a slab

// exp2 in one instruction (relative error 2^-22); 0 below 2^-126.
__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// A tensor map's coordinates of a head: rows of a tile are (token, packed head) pairs, `pack` neighbouring
// query heads to a token, so that the heads that share a key head can share its tiles.  An axis that repeats
// (stride 0) is one step in its map: its factor is 0 and its coordinate stays 0.
struct Place {
  int32_t head, batch;   // factors, 1 or 0
};

// Kernel parameters beside the maps.
struct Params {
  const int32_t* key_lengths;
  const int32_t* query_start;
  int32_t q_tokens, k_tokens, heads_q, heads_k, group, head_dim, causal;
  int32_t pack;          // query heads in a tile's rows: 1 or the group
  int32_t tile_tokens;   // queries in a tile: 128 / pack
  int32_t q_blocks;      // blocks along the queries
  int32_t splits;        // blocks that share a tile's keys
  float scale;
  Place q, k, v, d_o;
  uint32_t* err;
};

// Two 32-bit values in one instruction; the largest of three in one.
__device__ __forceinline__ uint64_t pair(float lo, float hi) { return (uint64_t)__float_as_uint(hi) << 32 | __float_as_uint(lo); }
__device__ __forceinline__ uint64_t pair(uint32_t lo, uint32_t hi) { return (uint64_t)hi << 32 | lo; }
__device__ __forceinline__ float low(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float high(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
  return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
  return d;
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

// Warpgroups of a block trade registers: what some give back others take, together no more than at the launch.
template <int n>
__device__ __forceinline__ void take_registers() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(n));
}
template <int n>
__device__ __forceinline__ void give_registers() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(n));
}

// The place of sequence b's first query, kept within a range in which sums of tokens (up to 2^29) cannot
// overflow: beyond the last key, or so far before the first that no query sees one, all are alike.
__device__ __forceinline__ int start_of(const Params& a, int b) {
  return a.query_start ? min(max(a.query_start[b], -(1 << 30)), a.k_tokens) : 0;
}
// Keys of sequence b: those that there are, and, causal, that its last query sees.  What lies behind them is not looked at.
__device__ __forceinline__ int keys_of(const Params& a, int b) {
  const int there = a.key_lengths ? min(max(a.key_lengths[b], 0), a.k_tokens) : a.k_tokens;
  return a.causal ? min(there, max(0, start_of(a, b) + a.q_tokens)) : there;
}

// scale log2(e); above 0, so that a hidden score's -infinity stays one (2^-149 of any score is 0 beside 1).
__device__ __forceinline__ float exponent_scale(const Params& a) { return fmaxf(a.scale * kLog2e, 0x1p-149f); }

// A tile of keys or values (kRows rows from `row` on of one head), by one thread, in boxes of kBox rows and 64 elements.
template <int kDim, int kRows = kTile, int kBox = kRows>
__device__ __forceinline__ void load_keys(uint32_t dst, const CUtensorMap* map, const Place& p, int row, int head, int batch,
                                          uint32_t bar) {
  mbar_arrive_expect_tx(bar, kRows * kDim * 2);
#pragma unroll
  for (int i = 0; i < kDim / 64; ++i)
#pragma unroll
    for (int r = 0; r < kRows; r += kBox)
      tma_load_4d(dst + (i * kRows + r) * 128, map, 64 * i, row + r, head * p.head, batch * p.batch, bar);
}

// A tile of queries (or of what has their shape), kRows rows of tokens and the `pack` heads of each, in boxes of kBox rows;
// where the pack does not divide them, the rows that are left keep what they held.  head: counted in packs.  The
// barrier's thread has announced query_bytes() for each.
template <int kDim, int kRows = kTile>
__device__ __forceinline__ uint32_t query_bytes(const Params& a) {
  return (kRows == kTile ? a.tile_tokens * a.pack : kRows) * kDim * 2;
}
template <int kDim, int kRows = kTile, int kBox = kRows>
__device__ __forceinline__ void load_queries(uint32_t dst, const CUtensorMap* map, const Params& a, const Place& p, int token,
                                             int head, int batch, uint32_t bar) {
#pragma unroll
  for (int i = 0; i < kDim / 64; ++i)
#pragma unroll
    for (int r = 0; r < kRows; r += kBox)
      tma_load_5d(dst + (i * kRows + r) * 128, map, 64 * i, 0, token + r / a.pack, head * p.head, batch * p.batch, bar);
}

// Rows from `first` on of a tile set to zero by one warp, visible to the tensor cores afterwards.
template <int kDim, int kRows = kTile>
__device__ __forceinline__ void clear_rows(uint32_t dst, int first, int lane) {
  for (int c = first * 8 + lane; c < kRows * 8; c += 32)
#pragma unroll
    for (int i = 0; i < kDim / 64; ++i) st_shared_v4(dst + i * kRows * 128 + c * 16, make_uint4(0, 0, 0, 0));
  fence_proxy_async_smem();
}

// K-major and MN-major descriptors of a tile, and how much further a step of 16 along K is.  (Tiles of 64 rows have one
// slab: heads of 64.)
__device__ __forceinline__ uint64_t k_major(uint32_t tile) { return make_sw128_desc(tile, 16, 1024, 0); }
__device__ __forceinline__ uint64_t mn_major(uint32_t tile) { return make_sw128_desc(tile, kSlab, 1024, 0); }
__device__ __forceinline__ constexpr uint64_t k_major_step(int k) { return (uint64_t)(((k >> 2) * kSlab + (k & 3) * 32) >> 4); }
__device__ __forceinline__ constexpr uint64_t mn_major_step(int k) { return (uint64_t)((k * 2048) >> 4); }

// 16-bit results of a row, eight at a time.
template <bool BF16>
__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack2<BF16>(v[0], v[1]), pack2<BF16>(v[2], v[3]), pack2<BF16>(v[4], v[5]), pack2<BF16>(v[6], v[7]));
}

// ---------------------------------------------------------------- host side

// A map's axis: its steps and bytes between them; one that has a single step, or repeats, is one step.
struct Axis {
  uint64_t steps, bytes;
};
inline Axis axis(int64_t steps, int64_t stride) {
  return steps <= 1 || stride == 0 ? Axis{1, 16} : Axis{(uint64_t)steps, (uint64_t)stride * 2};
}
inline bool map_of(CUtensorMap* map, const cbr_attention_desc_t& d, const void* p, int rank, const Axis* axes, const uint32_t* box) {
  uint64_t dims[5] = {(uint64_t)d.head_dim}, strides[4];
  for (int i = 1; i < rank; ++i) dims[i] = axes[i - 1].steps, strides[i - 1] = axes[i - 1].bytes;
  return encode_tiled(map, d.dtype == CBR_BF16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, rank, p, dims,
                      strides, box);
}

// Keys or values: [batch][heads_k][tokens][head_dim], boxes of `rows` tokens and 64 elements.
inline bool key_map(CUtensorMap* map, const cbr_attention_desc_t& d, const void* p, const int64_t* s, int rows = kTile) {
  const Axis axes[3] = {axis(std::max<int64_t>(d.k_tokens, 1), s[1]), axis(d.heads_k, s[2]), axis(d.batch, s[0])};
  const uint32_t box[4] = {64, (uint32_t)rows, 1, 1};
  return map_of(map, d, p, 4, axes, box);
}

// Queries, or what has their shape: [batch][heads_q / pack][tokens][pack][head_dim].
inline bool query_map(CUtensorMap* map, const cbr_attention_desc_t& d, const void* p, const int64_t* s, int pack, int rows = kTile) {
  const Axis axes[4] = {axis(pack, s[2]), axis(d.q_tokens, s[1]), axis(d.heads_q / pack, s[2] * pack), axis(d.batch, s[0])};
  const uint32_t box[5] = {64, (uint32_t)pack, (uint32_t)(rows / pack), 1, 1};
  return map_of(map, d, p, 5, axes, box);
}

inline Place place(const int64_t* s) { return Place{s[2] != 0, s[0] != 0}; }

inline Params params_of(const AttentionArgs& g, int pack) {
  const cbr_attention_desc_t& d = g.d;
  Params p{};
  p.key_lengths = g.key_lengths;
  p.query_start = g.query_start;
  p.q_tokens = (int32_t)d.q_tokens;
  p.k_tokens = (int32_t)d.k_tokens;
  p.heads_q = d.heads_q;
  p.heads_k = d.heads_k;
  p.group = d.heads_q / d.heads_k;
  p.head_dim = d.head_dim;
  p.causal = d.causal;
  p.pack = pack;
  p.tile_tokens = kTile / pack;
  p.scale = d.scale;
  p.q = place(d.q_stride);
  p.k = place(d.k_stride);
  p.v = place(d.v_stride);
  p.d_o = place(d.do_stride);
  p.err = g.err;
  return p;
}

}  // namespace att
}  // namespace cbr
