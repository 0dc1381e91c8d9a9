// The norms around a gated residual block, backward (formulas: include/cbr.h).
//
// One pass: a team of threads holds a row of x_out, dh, dx_out and the branch in registers, up to the
// stores of dx and dbranch, with coming rows' loads in flight meanwhile: a ring of rows in shared memory,
// filled by bulk copies, where a block is a team and the rows are aligned and of 16-bit elements; else the
// next row, in registers.  The parameters of its columns and their gradients stay in registers over its
// rows; gate and post_weight are constant over a gate's rows, so both take their gradients from one sum,
// of D e.  Blocks leave their sums in the workspace, and a second kernel adds them in a fixed order.
// Bound by HBM, six rows of the storage type: 32768x4096 bf16 in 265 us, 6.1 TB/s; narrow and unaligned
// rows by their instructions (50176x64 f16: 16 us, 2.4 TB/s).
//
// The second norm's means enter the first's linearly.  For RMS, with p = branch_scale gate post_weight
// and q = dx_out + r2 u: D = q - r2 mean(u c) c, so
//   mean(p D e) = mean(p q e) - r2 mean(u c) mean(p c e)
// and one round of sums over the team serves both; for LAYER it would take eight of them: two rounds.
//
// A gate's gradient is complete where its last row is, and goes straight out if all its rows were this
// team's.  Otherwise:
//   a block that is one team (wide rows) works on a run of consecutive rows, of which at most the first
//   and the last gate have rows elsewhere, too: those go to the workspace;
//   a block of several teams shares the rows of each gate of its run among them, where a gate has many
//   rows; where it has few, each team has a run of whole gates.
#include <algorithm>
#include <type_traits>

#include "cbr_internal.h"
#include "norm_ops.cuh"

namespace cbr {
namespace {

using namespace norm;

constexpr int kMaxStages = 8;

struct BwdPlan {
  int team;
  long long run;      // rows of a block (shared: of a block, else of a team)
  bool shared;        // the teams of a block share each gate's rows
  int stages;         // of the ring
  int row_bytes;      // of one of the ring's rows
  int blocks;
};

template <typename T, int kVec, int kEpt, bool kBlock, bool kRing, bool kCenter, int kThreads, int kFit>
__global__ void __launch_bounds__(kThreads, kFit)
    norm_backward_kernel(const __grid_constant__ BlockNormArgs a, const __grid_constant__ BwdPlan plan) {
  using R = Row<T, kVec, kEpt>;
  constexpr int kSums = kCenter ? 2 : 3;
  __shared__ float red[2][4][kMaxTeamWarps];
  __shared__ __align__(16) float fold[kBlock ? 1 : kThreads * kEpt];   // R::put writes 16 bytes at a time
  static_assert(__alignof__(fold) >= 16, "");
  __shared__ __align__(8) uint64_t full[kRing ? kMaxStages : 1];
  extern __shared__ __align__(128) uint8_t ring[];
  const int team = kBlock ? blockDim.x : plan.team, at = kBlock ? threadIdx.x : threadIdx.x & (team - 1);
  if (kBlock) {
    for (int i = threadIdx.x; i < 2 * 4 * kMaxTeamWarps; i += blockDim.x) (&red[0][0][0])[i] = 0.f;
    __syncthreads();
  }
  TeamSum<kBlock, kSums> sum{red};
  const int dim = (int)a.d.dim, col = at * kVec, left = dim - col;
  const float inv_d = 1.f / (float)dim, beta = a.d.branch_scale;
  const bool join = a.branch != nullptr, next = a.pre_weight != nullptr;
  const int teams = kBlock ? 1 : blockDim.x / team, mine = kBlock ? 0 : threadIdx.x / team;
  const bool shared = !kBlock && plan.shared;
  // this team's rows (shared: the block's, of which every teams-th)
  const long long first = (shared ? (long long)blockIdx.x : (long long)blockIdx.x * teams + mine) * plan.run;
  const long long last = min(first + plan.run, (long long)a.d.rows);
  float* const part = a.part + (long long)blockIdx.x * 4 * dim;   // pre_weight, post_weight, two gates

  float p[kEpt] = {}, w2[kEpt] = {};                        // branch_scale gate post_weight, pre_weight
  float de[kEpt] = {}, dw1[kEpt] = {}, dw2[kEpt] = {};      // sum of D e over the gate's rows so far
  if (next) R::params(a.pre_weight + col, w2, team, left);
  // Adds the teams' values of a column and puts them at `to`.
  auto fold_teams = [&](const float(&v)[kEpt], float* to) __attribute__((always_inline)) {
    if constexpr (kBlock) {
      R::put(to + col, v, team, left);
    } else {
      __syncthreads();
      R::put(fold + mine * dim + col, v, team, left);
      __syncthreads();
      for (int c = threadIdx.x; c < dim; c += blockDim.x) {
        float s = 0.f;
        for (int t = 0; t < teams; ++t) s += fold[t * dim + c];
        to[c] = s;
      }
    }
  };
  auto begin_gate = [&](long long g) __attribute__((always_inline)) {
    R::params(a.post_weight + col, p, team, left);
    if (a.gate) {
      float u[kEpt];
      R::params(a.gate + g * dim + col, u, team, left);
#pragma unroll
      for (int k = 0; k < kEpt; ++k) p[k] *= u[k];
    }
#pragma unroll
    for (int k = 0; k < kEpt; ++k) p[k] *= beta;
  };
  // The gradients of gate g from the sum of D e: dw1 has it added, the gate's comes back in u.
  auto end_gate = [&](long long g, float(&u)[kEpt]) __attribute__((always_inline)) {
    R::params(a.gate + g * dim + col, u, team, left);
#pragma unroll
    for (int k = 0; k < kEpt; ++k) dw1[k] += beta * u[k] * de[k];
    R::params(a.post_weight + col, u, team, left);
#pragma unroll
    for (int k = 0; k < kEpt; ++k) u[k] *= beta * de[k], de[k] = 0.f;
  };
  auto gate_at = [&](long long g) {   // where gate g's gradient goes
    const bool whole = g * a.d.gate_rows >= first && (g + 1) * a.d.gate_rows <= last;
    return whole ? a.dgate + g * dim : part + (2 + (g != first / a.d.gate_rows)) * dim;
  };

  // Pointers at this thread's first column of the row that is next to be loaded, and of that at hand.
  R xo, dh, dxo, f;
  float st[4];
  const T *xo_at = nullptr, *dh_at = nullptr, *dxo_at = nullptr, *f_at = nullptr;
  T *dx_at = nullptr, *df_at = nullptr;
  const float* st_at = nullptr;
  auto go_to = [&](long long row) __attribute__((always_inline)) {
    xo_at = static_cast<const T*>(a.x) + row * a.d.x_out_stride + col;
    dh_at = static_cast<const T*>(a.dh) + row * a.d.dh_stride + col;
    dxo_at = static_cast<const T*>(a.dx_out) + row * a.d.dx_out_stride + col;
    f_at = static_cast<const T*>(a.branch) + row * a.d.branch_stride + col;
    dx_at = static_cast<T*>(a.dx) + row * a.d.dx_stride + col;
    df_at = static_cast<T*>(a.dbranch) + row * a.d.dbranch_stride + col;
    st_at = a.stats + row * 4;
  };
  // The ring: thread 0 fills stage n % stages with row n's four parts.  A stage is read before the row's
  // first sum, whose barrier frees it.
  Turn turn{0, 0};
  bool ok = true;
  auto fill = [&](long long row, int stage) __attribute__((always_inline)) {
    const uint32_t bar = smem_u32(&full[stage]), to = smem_u32(ring) + stage * 4 * plan.row_bytes;
    const uint32_t bytes = (uint32_t)(dim * sizeof(T));
    mbar_arrive_expect_tx(bar, bytes * ((next ? 2 : 0) + (a.dx_out ? 1 : 0) + (join ? 1 : 0)));
    if (next) {
      bulk_load_1d(to, static_cast<const T*>(a.x) + row * a.d.x_out_stride, bytes, bar);
      bulk_load_1d(to + plan.row_bytes, static_cast<const T*>(a.dh) + row * a.d.dh_stride, bytes, bar);
    }
    if (a.dx_out) bulk_load_1d(to + 2 * plan.row_bytes, static_cast<const T*>(a.dx_out) + row * a.d.dx_out_stride, bytes, bar);
    if (join) bulk_load_1d(to + 3 * plan.row_bytes, static_cast<const T*>(a.branch) + row * a.d.branch_stride, bytes, bar);
  };
  if constexpr (kRing) {
    if (threadIdx.x == 0) {
      for (int i = 0; i < plan.stages; ++i) mbar_init(smem_u32(&full[i]), 1);
      fence_mbarrier_init();
    }
    __syncthreads();
    if (threadIdx.x == 0)
      for (int i = 0; i < plan.stages && first + i < last; ++i) fill(first + i, i);
  }
  auto read_stats = [&] __attribute__((always_inline)) {
    if constexpr (kVec == 1) {
#pragma unroll
      for (int i = 0; i < 4; ++i) st[i] = __ldg(st_at + i);
    } else {
      const float4 s4 = __ldg(reinterpret_cast<const float4*>(st_at));
      st[0] = s4.x, st[1] = s4.y, st[2] = s4.z, st[3] = s4.w;
    }
  };
  // Starts the loads of the row that the pointers are at, and moves them `rows` on.
  auto fetch = [&](bool here, int rows) __attribute__((always_inline)) {
    if (here) {
      if constexpr (!kRing) {
        if (next) {
          xo.load(xo_at, team, left);
          dh.load(dh_at, team, left);
        }
        if (a.dx_out) dxo.load(dxo_at, team, left);
        if (join) f.load(f_at, team, left);
      }
      read_stats();
    }
    if constexpr (!kRing) {
      xo_at += rows * a.d.x_out_stride;
      dh_at += rows * a.d.dh_stride;
      dxo_at += rows * a.d.dx_out_stride;
      f_at += rows * a.d.branch_stride;
    }
    st_at += rows * 4;
  };

  long long begin = first;
  long long gate = -1, gate_end = first;   // (not shared) the gate at hand and the first row of another
  const int stride = shared ? teams : 1;
  // shared: a stretch of rows of one gate at a time; else all of the team's rows
  while (shared ? begin < last : true) {
    const long long end = shared && a.gate ? min(last, (begin / a.d.gate_rows + 1) * a.d.gate_rows) : last;
    if (shared) begin_gate(begin / a.d.gate_rows);
    // a warp's teams go through as many rows as the longest, for the sums' shuffles
    const long long trips = kBlock ? max(0ll, end - begin) : shared ? (end - begin + teams - 1) / teams : plan.run;
    long long row = begin + (shared ? mine : 0);
    go_to(row);
    fetch(row < end, stride);
    for (long long i = 0; i < trips; ++i, row += stride) {
      const bool here = kBlock || row < end;
      if (!shared && join && here && row == gate_end) {
        if (a.gate) {
          if (gate >= 0) {
            float u[kEpt];
            end_gate(gate, u);
            R::put(gate_at(gate) + col, u, team, left);
          }
          gate = row / a.d.gate_rows;
          gate_end = (gate + 1) * a.d.gate_rows;
        } else {
          gate_end = last;
        }
        begin_gate(gate);
      }
      const float m1 = st[0], r1 = st[1], m2 = st[2], r2 = st[3];
      if constexpr (kRing) {   // a wait that runs out is reported; the rest is done without further ones
        if (ok && !mbar_wait(smem_u32(&full[turn.slot]), turn.parity)) {
          ok = false;
          report_error(a.err, kErrWaitOperand);
        }
        const uint32_t from = smem_u32(ring) + turn.slot * 4 * plan.row_bytes + col * (uint32_t)sizeof(T);
        if (next) {
          xo.load_shared(from, team, left);
          dh.load_shared(from + plan.row_bytes, team, left);
        }
        if (a.dx_out) dxo.load_shared(from + 2 * plan.row_bytes, team, left);
        if (join) f.load_shared(from + 3 * plan.row_bytes, team, left);
      }
      float d[kEpt], n[kEpt], u[kEpt], e[kEpt];
      if (a.dx_out) {
        dxo.get(d);
      } else {
#pragma unroll
        for (int k = 0; k < kEpt; ++k) d[k] = 0.f;
      }
      if (join) f.get(e);
      if (next) {
        xo.get(n);
        dh.get(u);
      }
      fetch(row + stride < end, stride);
      float s[kSums] = {};
      auto sum_first = [&] __attribute__((always_inline)) {
        sum(s, team);
        if constexpr (kRing) {
          if (threadIdx.x == 0 && row + plan.stages < last) fill(row + plan.stages, turn.slot);
          turn.next(plan.stages);
        }
      };
      if (next) {
#pragma unroll
        for (int k = 0; k < kEpt; ++k) {
          n[k] = (kCenter ? n[k] - m2 : n[k]) * r2;
          const float t = u[k] * n[k];
          if (here) dw2[k] += t;
          u[k] *= w2[k];
          s[0] += t * w2[k];
          if constexpr (kCenter) s[1] += u[k];
          else d[k] += r2 * u[k];
        }
      }
      if (join) {
#pragma unroll
        for (int k = 0; k < kEpt; ++k) e[k] = (kCenter ? e[k] - m1 : e[k]) * r1;
      }
      if constexpr (kCenter) {
        if (next) {
          sum_first();
          const float mc = s[0] * inv_d, mu = s[1] * inv_d;
#pragma unroll
          for (int k = 0; k < kEpt; ++k) d[k] += r2 * (u[k] - mu - n[k] * mc);
        }
        if (join) {
          s[0] = s[1] = 0.f;
#pragma unroll
          for (int k = 0; k < kEpt; ++k) {
            const float v = p[k] * d[k];
            s[0] += v * e[k];
            s[1] += v;
          }
          if (next) sum(s, team);
          else sum_first();
        }
      } else {
        if (join) {
#pragma unroll
          for (int k = 0; k < kEpt; ++k) {
            const float v = p[k] * e[k];
            s[1] += v * d[k];
            if (next) s[2] += v * n[k];
          }
        }
        sum_first();
        if (next) {
          const float mc = r2 * s[0] * inv_d;
#pragma unroll
          for (int k = 0; k < kEpt; ++k) d[k] -= mc * n[k];
          s[1] -= mc * s[2];
        }
        s[0] = s[1];
      }
      if (join) {
        const float me = s[0] * inv_d, mv = kCenter ? s[1] * inv_d : 0.f;
#pragma unroll
        for (int k = 0; k < kEpt; ++k) {
          if (here) de[k] += d[k] * e[k];
          e[k] = kCenter ? r1 * (p[k] * d[k] - mv - e[k] * me) : r1 * (p[k] * d[k] - e[k] * me);
          d[k] *= a.d.residual_scale;
        }
        if (here) R::store(df_at, e, team, left);
      }
      if (here) R::store(dx_at, d, team, left);
      dx_at += stride * a.d.dx_stride;
      df_at += stride * a.d.dbranch_stride;
    }
    if (!shared) break;
    const long long g = begin / a.d.gate_rows;
    float u[kEpt];
    end_gate(g, u);
    fold_teams(u, gate_at(g));
    begin = end;
  }
  if (join && !shared) {
    if (a.gate) {
      if (gate >= 0) {
        float u[kEpt];
        end_gate(gate, u);
        R::put(gate_at(gate) + col, u, team, left);
      }
    } else {
#pragma unroll
      for (int k = 0; k < kEpt; ++k) dw1[k] = beta * de[k];
    }
  }
  if constexpr (kRing) {   // no copy is in flight when the block ends, also where a wait ran out
    if (!ok && threadIdx.x == 0)
      for (int i = 0; i < plan.stages; ++i, turn.next(plan.stages)) mbar_wait(smem_u32(&full[turn.slot]), turn.parity);
  }
  if (next) fold_teams(dw2, part);
  if (join) fold_teams(dw1, part + dim);
}

// Adds the blocks' sums: 32 columns a block, kSlices threads a column take every kSlices-th block's and
// are added in their order.  y = 0: the weights; the others: the gates whose rows several blocks had.
constexpr int kSlices = 32;
__global__ void __launch_bounds__(32 * kSlices) norm_reduce_kernel(const __grid_constant__ BlockNormArgs a, int blocks,
                                                                   long long run, bool by_gate) {
  __shared__ float part[2][kSlices][32];
  const int dim = (int)a.d.dim, c = blockIdx.x * 32 + (threadIdx.x & 31), slice = threadIdx.x >> 5;
  const long long stride = 4ll * dim;
  float *to = nullptr, *to2 = nullptr;
  float s = 0.f, t = 0.f;
  if (blockIdx.y == 0) {
    if (a.pre_weight) to = a.dpre_weight;
    if (a.branch) to2 = a.dpost_weight;
    const float* from = a.part + c;
    if (c < dim)
#pragma unroll 8
      for (int b = slice; b < blocks; b += kSlices) {
        if (to) s += __ldg(from + b * stride);
        if (to2) t += __ldg(from + b * stride + dim);
      }
  } else {
    // the gate y - 1, or (gates shorter than a run) the one that has the first row of block y and an
    // earlier one; only its first block may have another gate's rows before it
    const long long g = by_gate ? blockIdx.y - 1 : blockIdx.y * run / a.d.gate_rows;
    const long long b0 = g * a.d.gate_rows / run, b1 = ((g + 1) * a.d.gate_rows - 1) / run;
    if (b0 == b1) return;
    to = a.dgate + g * dim;
    const float* from = a.part + 2 * dim + c;
    const int later = g != b0 * run / a.d.gate_rows ? dim : 0;
    if (c < dim)
#pragma unroll 8
      for (long long b = b0 + slice; b <= b1; b += kSlices) s += __ldg(from + b * stride + (b == b0 ? later : 0));
  }
  part[0][slice][threadIdx.x & 31] = s;
  part[1][slice][threadIdx.x & 31] = t;
  __syncthreads();
  float* const out = slice ? to2 : to;
  if (slice < 2 && c < dim && out) {
    float v = 0.f;
#pragma unroll
    for (int i = 0; i < kSlices; ++i) v += part[slice][i][threadIdx.x & 31];
    out[c] = v;
  }
}

// Blocks at most on an SM: the workspace has room for their sums.
int blocks_per_sm(long long dim) { return (int)std::max(1ll, std::min(8ll, 8192 / dim)); }

template <typename T, int kVec, int kEpt, bool kBlock, bool kRing, bool kCenter, int kThreads, int kFit>
int launch_kind(const BlockNormArgs& a, int team, int threads, int num_sms, cudaStream_t st) {
  auto kernel = norm_backward_kernel<T, kVec, kEpt, kBlock, kRing, kCenter, kThreads, kFit>;
  BwdPlan p{};
  int smem = 0;
  if (kRing) {
    // as many stages as fit beside one another in blocks of half an SM's threads and registers in all
    if (!ensure_smem_attr(reinterpret_cast<const void*>(kernel), 200 * 1024)) return CBR_ERR_CUDA;
    p.row_bytes = (int)((a.d.dim * sizeof(T) + 127) / 128 * 128);
    const int share = std::max(1, std::min(512 / threads, blocks_per_sm(a.d.dim)));
    p.stages = std::max(2, std::min(kMaxStages, 200 * 1024 / share / (4 * p.row_bytes)));
    smem = p.stages * 4 * p.row_bytes;
  }
  const int fit = blocks_that_fit(reinterpret_cast<const void*>(kernel), threads, smem);
  if (fit < 1) return CBR_ERR_CUDA;
  const long long most = (long long)std::min(fit, blocks_per_sm(a.d.dim)) * num_sms;
  const int teams = kBlock ? 1 : threads / team;
  p.team = team;
  // Few rows a gate: teams with runs of gates; 32, or as many as a block has teams: the block shares each.
  // us, 50176x64 f16 with 8, 16, 32, 64 rows a gate: runs 18, 23, 39, 70 (fewer and fewer teams have one),
  // shared 81, 48, 32, 26 (the teams' sums are added up once a gate).
  p.shared = !kBlock && a.gate && a.d.gate_rows >= std::max(32, teams);
  if (p.shared) {
    p.blocks = (int)std::min<long long>(most, (a.d.rows + teams - 1) / teams);
    p.run = (a.d.rows + p.blocks - 1) / p.blocks;
    p.blocks = (int)((a.d.rows + p.run - 1) / p.run);
  } else {
    // runs of whole gates, where a run has several (a block that is a team can do without)
    const long long unit = !a.gate || (kBlock && a.d.gate_rows * 4 > a.d.rows / most) ? 1 : a.d.gate_rows;
    const long long units = a.d.rows / unit, runs = std::min<long long>(units, most * teams);
    p.run = (units + runs - 1) / runs * unit;
    p.blocks = (int)((a.d.rows + p.run * teams - 1) / (p.run * teams));
  }
  kernel<<<p.blocks, threads, smem, st>>>(a, p);
  if (cudaGetLastError() != cudaSuccess) return CBR_ERR_CUDA;
  const bool split = a.gate && (kBlock || p.shared) && p.run % a.d.gate_rows != 0;
  const long long groups = split ? a.d.rows / a.d.gate_rows : 0;
  const bool by_gate = groups < p.blocks;
  const unsigned extra = split ? (unsigned)(by_gate ? groups : p.blocks - 1) : 0;
  norm_reduce_kernel<<<dim3((unsigned)((a.d.dim + 31) / 32), 1 + extra), 32 * kSlices, 0, st>>>(a, p.blocks, p.run, by_gate);
  return cudaGetLastError() == cudaSuccess ? CBR_OK : CBR_ERR_CUDA;
}

template <typename T, int kVec, int kEpt, bool kBlock, bool kRing, int kThreads, int kFit>
int launch(const BlockNormArgs& a, int team, int threads, int num_sms, cudaStream_t st) {
  return a.d.kind == CBR_NORM_LAYER
             ? launch_kind<T, kVec, kEpt, kBlock, kRing, true, kThreads, kFit>(a, team, threads, num_sms, st)
             : launch_kind<T, kVec, kEpt, kBlock, kRing, false, kThreads, kFit>(a, team, threads, num_sms, st);
}

// us, what is taken first.  Narrow rows: teams of a warp or less in blocks of 128 threads at three an SM,
// 168 registers each (50176x64 f16 16.2); 256 at two have 128 and spill (18.5); a block for each row: 57.
// Wide rows: eight elements a thread, 16-bit rows through the ring (32768x4096 bf16 265, 8192x1024 31),
// since without it too little is in flight (648, 45); 32-bit ones in registers, where the next row's four
// parts are as much as the ring holds (8192x4096 135, with the ring 146).  16 elements a thread spill
// (32768x4096: 791) and are left to rows that 512 threads cannot hold otherwise.  Rows of single 16-bit
// elements: four a thread, for more threads on an SM (16384x1001 bf16 62, eight: 102); 32-bit ones keep
// eight (73, four: 80).
template <typename T, int kVec>
int pick(const BlockNormArgs& a, int num_sms, cudaStream_t st) {
  const int dim = (int)a.d.dim;
  auto threads_of = [&](int ept) { return ((dim + ept - 1) / ept + 31) / 32 * 32; };
  if (dim <= 256) {
    int team = 1;
    while (team * 8 < dim) team *= 2;
    return launch<T, kVec, 8, false, false, 128, 3>(a, team, 128, num_sms, st);
  }
  if constexpr (kVec == 1 && sizeof(T) == 2)
    if (dim <= 2048) return launch<T, kVec, 4, true, false, 512, 1>(a, threads_of(4), threads_of(4), num_sms, st);
  constexpr bool kRing = kVec > 1 && sizeof(T) == 2;
  if (dim <= 4096) return launch<T, kVec, 8, true, kRing, 512, 1>(a, threads_of(8), threads_of(8), num_sms, st);
  if (dim <= 8192) return launch<T, kVec, 16, true, kRing, 512, 1>(a, threads_of(16), threads_of(16), num_sms, st);
  return launch<T, kVec, 32, true, false, 512, 1>(a, threads_of(32), threads_of(32), num_sms, st);
}

template <typename T>
int by_alignment(const BlockNormArgs& a, int num_sms, cudaStream_t st) {
  constexpr int kVec = 16 / sizeof(T);
  const cbr_block_norm_desc_t& d = a.d;
  const bool vec = d.dim % kVec == 0 && d.dx_stride % kVec == 0 && aligned16(a.dx) && aligned16(a.post_weight) &&
                   aligned16(a.pre_weight) && aligned16(a.gate) && aligned16(a.part) && aligned16(a.dgate) && aligned16(a.stats) &&
                   (!a.dx_out || (d.dx_out_stride % kVec == 0 && aligned16(a.dx_out))) &&
                   (!a.branch || (d.branch_stride % kVec == 0 && d.dbranch_stride % kVec == 0 && aligned16(a.branch) &&
                                  aligned16(a.dbranch))) &&
                   (!a.pre_weight || (d.x_out_stride % kVec == 0 && d.dh_stride % kVec == 0 && aligned16(a.x) && aligned16(a.dh)));
  return vec ? pick<T, kVec>(a, num_sms, st) : pick<T, 1>(a, num_sms, st);
}

}  // namespace

size_t block_norm_part_floats(const cbr_block_norm_desc_t& d) { return (size_t)kMaxCtas * blocks_per_sm(d.dim) * 4 * d.dim; }

int launch_block_norm_backward(const BlockNormArgs& a, int num_sms, cudaStream_t st) {
  if (a.d.dtype == CBR_F32) return by_alignment<float>(a, num_sms, st);
  if (a.d.dtype == CBR_BF16) return by_alignment<__nv_bfloat16>(a, num_sms, st);
  return by_alignment<__half>(a, num_sms, st);
}

}  // namespace cbr
