// The norms around a gated residual block, forward (formulas: include/cbr.h).
//
// One pass: a team of threads holds a row of x and of the branch in registers, from its loads to its
// stores, with the next row's loads in flight meanwhile; the parameters of its columns stay in registers
// over its run of rows.  Variances are sums of squared differences from the mean, over the registers.
// Bound by HBM, x and the branch in, x_out and h out: 32768x4096 bf16 in 174 us, 6.2 TB/s.  A ring of rows
// in shared memory, as the backward has, is slower here (251 us): one row ahead in registers is enough in
// flight.
#include <algorithm>
#include <map>
#include <mutex>
#include <tuple>
#include <type_traits>

#include "cbr_internal.h"
#include "norm_ops.cuh"

namespace cbr {
namespace {

using namespace norm;

template <typename T, int kVec, int kEpt, bool kBlock, bool kCenter, int kThreads, int kFit>
__global__ void __launch_bounds__(kThreads, kFit) norm_forward_kernel(const __grid_constant__ BlockNormArgs a, int team_) {
  using R = Row<T, kVec, kEpt>;
  __shared__ float red[2][1][kMaxTeamWarps];
  const int team = kBlock ? blockDim.x : team_, at = kBlock ? threadIdx.x : threadIdx.x & (team - 1);
  if (kBlock) {
    if (threadIdx.x < kMaxTeamWarps) red[0][0][threadIdx.x] = red[1][0][threadIdx.x] = 0.f;
    __syncthreads();
  }
  TeamSum<kBlock, 1> sum{red};
  const int dim = (int)a.d.dim, col = at * kVec, left = dim - col;
  const float inv_d = 1.f / (float)dim;
  const bool join = a.branch != nullptr, next = a.pre_weight != nullptr;
  const int teams_a_block = kBlock ? 1 : blockDim.x / team;
  const long long teams = (long long)gridDim.x * teams_a_block;
  const long long mine = (long long)blockIdx.x * teams_a_block + (kBlock ? 0 : threadIdx.x / team);
  const long long run = (a.d.rows + teams - 1) / teams, first = mine * run, last = min(first + run, (long long)a.d.rows);

  // mean and 1 / sqrt(variance + eps) of the row in v
  auto moments = [&](const float(&v)[kEpt], float& m, float& r) __attribute__((always_inline)) {
    float s[1] = {0.f};
    m = 0.f;
    if constexpr (kCenter) {
#pragma unroll
      for (int i = 0; i < kEpt; ++i) s[0] += v[i];
      sum(s, team);
      m = s[0] * inv_d;
      s[0] = 0.f;
    }
#pragma unroll
    for (int i = 0; i < kEpt; ++i) {
      const float d = !kCenter ? v[i] : R::inside(i, team, left) ? v[i] - m : 0.f;   // v: 0 past the row
      s[0] += d * d;
    }
    sum(s, team);
    r = inverse_root(s[0] * inv_d + a.d.eps);
  };

  R x, f;
  const T* xp = static_cast<const T*>(a.x) + first * a.d.x_stride + col;
  const T* fp = join ? static_cast<const T*>(a.branch) + first * a.d.branch_stride + col : nullptr;
  T* op = join ? static_cast<T*>(a.x_out) + first * a.d.x_out_stride + col : nullptr;
  T* hp = next ? static_cast<T*>(a.h) + first * a.d.h_stride + col : nullptr;
  auto fetch = [&](bool here) __attribute__((always_inline)) {
    if (here) {
      x.load(xp, team, left);
      if (join) f.load(fp, team, left);
    }
    xp += a.d.x_stride;
    fp += a.d.branch_stride;
  };
  fetch(first < last);
  float w1[kEpt] = {}, w2[kEpt] = {};   // branch_scale gate post_weight, pre_weight
  if (next) R::params(a.pre_weight + col, w2, team, left);
  long long gate_end = first;           // the first row of another gate
  // a warp's teams go through as many rows as the longest of their runs, for the sums' shuffles
  for (long long i = 0; i < run; ++i) {
    const long long row = first + i;
    if (kBlock && row >= last) break;
    const bool here = kBlock || row < last;
    if (join && here && row == gate_end) {
      R::params(a.post_weight + col, w1, team, left);
      gate_end = last;
      if (a.gate) {
        const long long g = row / a.d.gate_rows;
        float u[kEpt];
        R::params(a.gate + g * dim + col, u, team, left);
#pragma unroll
        for (int k = 0; k < kEpt; ++k) w1[k] *= u[k];
        gate_end = (g + 1) * a.d.gate_rows;
      }
#pragma unroll
      for (int k = 0; k < kEpt; ++k) w1[k] *= a.d.branch_scale;
    }
    float v[kEpt], n[kEpt], m1 = 0.f, r1 = 0.f, m2 = 0.f, r2 = 0.f;
    x.get(v);
    if (join) f.get(n);
    fetch(row + 1 < last);
    if (join) {
      moments(n, m1, r1);
#pragma unroll
      for (int k = 0; k < kEpt; ++k) v[k] = a.d.residual_scale * v[k] + (kCenter ? n[k] - m1 : n[k]) * (r1 * w1[k]);
      if (here) R::store(op, v, team, left);
      op += a.d.x_out_stride;
    }
    if (next) {
      moments(v, m2, r2);
#pragma unroll
      for (int k = 0; k < kEpt; ++k) v[k] = (kCenter ? v[k] - m2 : v[k]) * (r2 * w2[k]);
      if (here) R::store(hp, v, team, left);
      hp += a.d.h_stride;
    }
    if (a.stats && here && at == 0) {
      float* s = a.stats + row * 4;
      s[0] = m1, s[1] = r1, s[2] = m2, s[3] = r2;
    }
  }
}

template <typename T, int kVec, int kEpt, bool kBlock, int kThreads, int kFit>
int launch(const BlockNormArgs& a, int team, int threads, int num_sms, cudaStream_t st) {
  auto kernel = a.d.kind == CBR_NORM_LAYER ? norm_forward_kernel<T, kVec, kEpt, kBlock, true, kThreads, kFit>
                                           : norm_forward_kernel<T, kVec, kEpt, kBlock, false, kThreads, kFit>;
  const int blocks = blocks_that_fit(reinterpret_cast<const void*>(kernel), threads, 0);
  if (blocks < 1) return CBR_ERR_CUDA;
  const int teams = kBlock ? 1 : threads / team;
  const long long want = (a.d.rows + teams - 1) / teams;
  kernel<<<(unsigned)std::min<long long>(want, (long long)blocks * num_sms), threads, 0, st>>>(a, team);
  return cudaGetLastError() == cudaSuccess ? CBR_OK : CBR_ERR_CUDA;
}

template <typename T, int kVec>
int pick(const BlockNormArgs& a, int num_sms, cudaStream_t st) {
  const int dim = (int)a.d.dim;
  // us, what is taken first.  Narrow rows: a warp or less each, eight elements a thread (50176x64 f16 7.4,
  // a block for each row: 24).  Others: a block each, 16 elements a thread, as fewer threads have less to
  // add up (16384x1001 bf16 33, 8192x1024 14; eight a thread 42, 17), and the same at 4096 wide; 32 a thread
  // leave too few in flight (16384x1001: 89) and are for rows that 512 threads cannot hold otherwise.
  if (dim <= 256) {
    int team = 1;
    while (team * 8 < dim) team *= 2;
    return launch<T, kVec, 8, false, 256, 3>(a, team, 256, num_sms, st);
  }
  const int ept = dim <= 8192 ? 16 : 32;
  const int threads = ((dim + ept - 1) / ept + 31) / 32 * 32;
  if (ept == 16) return launch<T, kVec, 16, true, 512, 1>(a, threads, threads, num_sms, st);
  return launch<T, kVec, 32, true, 512, 1>(a, threads, threads, num_sms, st);
}

template <typename T>
int by_alignment(const BlockNormArgs& a, int num_sms, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  const cbr_block_norm_desc_t& d = a.d;
  const bool vec = d.dim % kVec == 0 && d.x_stride % kVec == 0 && aligned16(a.x) && aligned16(a.post_weight) &&
                   aligned16(a.pre_weight) && aligned16(a.gate) &&
                   (!a.branch || (d.branch_stride % kVec == 0 && d.x_out_stride % kVec == 0 && aligned16(a.branch) && aligned16(a.x_out))) &&
                   (!a.h || (d.h_stride % kVec == 0 && aligned16(a.h)));
  return vec ? pick<T, kVec>(a, num_sms, st) : pick<T, 1>(a, num_sms, st);
}

}  // namespace

int blocks_that_fit(const void* kernel, int threads, int smem) {
  static std::mutex mu;
  static std::map<std::tuple<const void*, int, int, int>, int> known;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  std::lock_guard<std::mutex> lk(mu);
  const auto key = std::make_tuple(kernel, threads, smem, dev);
  const auto it = known.find(key);
  if (it != known.end()) return it->second;
  int blocks = 0;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&blocks, kernel, threads, smem) != cudaSuccess) {
    cudaGetLastError();
    return 0;
  }
  return known[key] = blocks;
}

int launch_block_norm(const BlockNormArgs& a, int num_sms, cudaStream_t st) {
  if (a.d.dtype == CBR_F32) return by_alignment<float>(a, num_sms, st);
  if (a.d.dtype == CBR_BF16) return by_alignment<__nv_bfloat16>(a, num_sms, st);
  return by_alignment<__half>(a, num_sms, st);
}

}  // namespace cbr
