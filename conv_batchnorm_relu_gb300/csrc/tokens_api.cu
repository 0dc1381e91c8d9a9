// C ABI of the token operators (declared in include/cbr.h): argument checks and dispatch.
#include <algorithm>
#include <cmath>

#include "api_checks.h"
#include "cbr_internal.h"
#include "token_ops.h"

namespace cbr {
namespace {

constexpr int64_t kMaxVocab = 393216, kMaxTopk = 1024, kMaxDim = 16384;
constexpr int kMaxHeadDim = 1024, kMaxAxes = 8;

int check(const cbr_distill_desc_t* d) {
  if (!d) return CBR_ERR_INVALID_ARG;
  if (!extent(d->rows) || d->vocab < 1 || d->topk < 0 || !(d->temperature > 0.f) || !finite(d->temperature) ||
      !finite(1.4426951f / d->temperature) || (d->id_bytes != 4 && d->id_bytes != 8))
    return CBR_ERR_INVALID_ARG;
  if (!known_dtype(d->dtype) || !known_dtype(d->top_dtype) || d->vocab > kMaxVocab || d->topk > kMaxTopk)
    return CBR_ERR_UNSUPPORTED;
  return CBR_OK;
}

int run(DistillArgs a, bool need_stats, bool need_grad, bool backward, cudaStream_t st) {
  const cbr_distill_desc_t& d = a.d;
  if (!row_stride(d.logits_stride, d.vocab, d.rows) || (need_grad && !row_stride(d.dlogits_stride, d.vocab, d.rows)) ||
      !row_stride(d.ids_stride, d.topk, d.rows) || !row_stride(d.top_stride, d.topk, d.rows))
    return CBR_ERR_INVALID_ARG;
  if (d.rows == 0) return CBR_OK;
  if (!a.logits || (d.topk > 0 && (!a.top_ids || !a.top_logits)) || (!backward && !a.loss) ||
      (need_stats && !a.stats) || (need_grad && !a.dlogits))
    return CBR_ERR_INVALID_ARG;
  if (need_grad && !same_or_apart(a.dlogits, d.dlogits_stride, a.logits, d.logits_stride, d.rows))
    return CBR_ERR_INVALID_ARG;
  if (off(a.logits, elt(d.dtype)) || off(a.dlogits, elt(d.dtype)) || off(a.top_ids, d.id_bytes) ||
      off(a.top_logits, elt(d.top_dtype)) || off(a.teacher_lse, 4) || off(a.row_weight, 4) || off(a.loss, 4) ||
      off(a.stats, 4) || off(a.dloss, 4))
    return CBR_ERR_MISALIGNED;
  int sms = 0;
  if (const int e = device_for_call(&sms, &a.err)) return e;
  return backward ? launch_distill_backward(a, st) : launch_distill(a, st);
}

int check(const cbr_block_norm_desc_t* d) {
  if (!d) return CBR_ERR_INVALID_ARG;
  if (!extent(d->rows) || d->dim < 1 || !finite(d->residual_scale) || !finite(d->branch_scale))
    return CBR_ERR_INVALID_ARG;
  if (d->kind != CBR_NORM_RMS && d->kind != CBR_NORM_LAYER) return CBR_ERR_INVALID_ARG;
  if (!known_dtype(d->dtype) || d->dim > kMaxDim) return CBR_ERR_UNSUPPORTED;
  return CBR_OK;
}

bool gate_rows_ok(const cbr_block_norm_desc_t& d, const float* gate) {
  return !gate || (d.gate_rows >= 1 && d.rows % d.gate_rows == 0);
}

int check(const cbr_rotary_desc_t* d) {
  if (!d) return CBR_ERR_INVALID_ARG;
  if (!extent(d->batch) || !extent(d->tokens) || (d->tokens && d->batch > kMaxExtent / d->tokens) || d->heads_q < 0 ||
      d->heads_k < 0 || d->head_dim < 1 || d->rot_dim < 2 || d->rot_dim % 2 || d->rot_dim > d->head_dim ||
      d->axes < 1 || (d->layout != CBR_ROTARY_HALVES && d->layout != CBR_ROTARY_NEIGHBOURS))
    return CBR_ERR_INVALID_ARG;
  for (int i = 0; i < 3; ++i)
    if (!extent(d->q_stride[i]) || !extent(d->k_stride[i]) || !extent(d->q_out_stride[i]) ||
        !extent(d->k_out_stride[i]) || !extent(d->pos_stride[i]))
      return CBR_ERR_INVALID_ARG;
  const int64_t steps[3] = {d->batch, d->tokens, std::max(d->heads_q, d->heads_k)};
  for (int i = 0; i < 3; ++i)
    if (!in_reach(d->q_stride[i], steps[i]) || !in_reach(d->k_stride[i], steps[i]) || !in_reach(d->q_out_stride[i], steps[i]) ||
        !in_reach(d->k_out_stride[i], steps[i]) || !in_reach(d->pos_stride[i], i < 2 ? steps[i] : d->axes))
      return CBR_ERR_INVALID_ARG;
  if (!known_dtype(d->dtype) || d->head_dim > kMaxHeadDim || d->axes > kMaxAxes || d->heads_q > 65536 ||
      d->heads_k > 65536)
    return CBR_ERR_UNSUPPORTED;
  return CBR_OK;
}

int run(const cbr_rotary_desc_t* desc, const void* q, const void* k, const int32_t* positions, const int64_t* freq,
        const uint8_t* axis, void* q_out, void* k_out, bool backward, cudaStream_t st) {
  if (const int e = check(desc)) return e;
  const cbr_rotary_desc_t& d = *desc;
  if ((d.heads_q && !distinct(d.q_out_stride, d.batch, d.tokens, d.heads_q, d.head_dim)) || (d.heads_k && !distinct(d.k_out_stride, d.batch, d.tokens, d.heads_k, d.head_dim)))
    return CBR_ERR_INVALID_ARG;
  if (d.batch == 0 || d.tokens == 0 || d.heads_q + d.heads_k == 0) return CBR_OK;
  if ((d.heads_q && (!q || !q_out)) || (d.heads_k && (!k || !k_out)) || !positions || !freq || !axis)
    return CBR_ERR_INVALID_ARG;
  if ((d.heads_q && q == q_out && !same(d.q_stride, d.q_out_stride)) ||
      (d.heads_k && k == k_out && !same(d.k_stride, d.k_out_stride)))
    return CBR_ERR_INVALID_ARG;
  const size_t e = elt(d.dtype);
  if (off(q, e) || off(k, e) || off(q_out, e) || off(k_out, e) || off(positions, 4) || off(freq, 8))
    return CBR_ERR_MISALIGNED;
  int sms = 0;
  uint32_t* err = nullptr;
  if (const int s = device_for_call(&sms, &err)) return s;
  RotaryArgs a{d, q, k, positions, freq, axis, q_out, k_out, backward};
  return launch_rotary(a, sms, st);
}

}  // namespace
}  // namespace cbr

using namespace cbr;

extern "C" {

cbr_status_t cbr_distill_forward(const cbr_distill_desc_t* desc, const void* logits, const void* top_ids,
                                 const void* top_logits, const float* teacher_lse, const float* row_weight,
                                 float* loss, float* stats, cbr_stream_t stream) {
  return guarded([&]() -> int {
    if (const int e = check(desc)) return e;
    DistillArgs a{*desc, nullptr, logits, top_ids, top_logits, teacher_lse, row_weight, loss, stats, nullptr, nullptr};
    return run(a, true, false, false, reinterpret_cast<cudaStream_t>(stream));
  });
}

cbr_status_t cbr_distill_backward(const cbr_distill_desc_t* desc, const float* dloss, const void* logits,
                                  const void* top_ids, const void* top_logits, const float* teacher_lse,
                                  const float* row_weight, const float* stats, void* dlogits, cbr_stream_t stream) {
  return guarded([&]() -> int {
    if (const int e = check(desc)) return e;
    DistillArgs a{*desc, dloss, logits, top_ids, top_logits, teacher_lse, row_weight, nullptr,
                  const_cast<float*>(stats), dlogits, nullptr};
    return run(a, true, true, true, reinterpret_cast<cudaStream_t>(stream));
  });
}

cbr_status_t cbr_distill_forward_backward(const cbr_distill_desc_t* desc, const void* logits, const void* top_ids,
                                          const void* top_logits, const float* teacher_lse,
                                          const float* row_weight, float* loss, float* stats, void* dlogits,
                                          cbr_stream_t stream) {
  return guarded([&]() -> int {
    if (const int e = check(desc)) return e;
    DistillArgs a{*desc, nullptr, logits, top_ids, top_logits, teacher_lse, row_weight, loss, stats, dlogits, nullptr};
    return run(a, false, true, false, reinterpret_cast<cudaStream_t>(stream));
  });
}

cbr_status_t cbr_block_norm_forward(const cbr_block_norm_desc_t* desc, const void* x, const void* branch,
                                    const float* post_weight, const float* gate, const float* pre_weight,
                                    void* x_out, void* h, float* stats, cbr_stream_t stream) {
  return guarded([&]() -> int {
    if (const int e = check(desc)) return e;
    const cbr_block_norm_desc_t& d = *desc;
    // the join is there where its weight is: an empty branch may have no address
    const bool join = post_weight != nullptr;
    if (!join) gate = nullptr;
    if (!(d.eps > 0.f) || !finite(d.eps) || !gate_rows_ok(d, gate)) return CBR_ERR_INVALID_ARG;
    if ((!join && branch) || (!join && !pre_weight)) return CBR_ERR_INVALID_ARG;
    if (!row_stride(d.x_stride, d.dim, d.rows) || (join && !row_stride(d.branch_stride, d.dim, d.rows)) ||
        (join && !row_stride(d.x_out_stride, d.dim, d.rows)) || (pre_weight && !row_stride(d.h_stride, d.dim, d.rows)))
      return CBR_ERR_INVALID_ARG;
    if (d.rows == 0) return CBR_OK;
    if (!x || (join && (!branch || !x_out)) || (pre_weight && !h)) return CBR_ERR_INVALID_ARG;
    if (branch && (!same_or_apart(x_out, d.x_out_stride, x, d.x_stride, d.rows) ||
                   !same_or_apart(x_out, d.x_out_stride, branch, d.branch_stride, d.rows)))
      return CBR_ERR_INVALID_ARG;
    if (pre_weight && (!same_or_apart(h, d.h_stride, branch ? branch : x, branch ? d.branch_stride : d.x_stride, d.rows) ||
                       h == x_out || (branch && h == x)))
      return CBR_ERR_INVALID_ARG;
    const size_t e = elt(d.dtype);
    if (off(x, e) || off(branch, e) || off(x_out, e) || off(h, e) || off(post_weight, 4) || off(gate, 4) ||
        off(pre_weight, 4) || off(stats, 4))
      return CBR_ERR_MISALIGNED;
    BlockNormArgs a{};
    int sms = 0;
    uint32_t* err = nullptr;
    if (const int s = device_for_call(&sms, &err)) return s;
    a.d = d;
    a.x = x;
    a.branch = branch;
    a.post_weight = post_weight;
    a.gate = gate;
    a.pre_weight = pre_weight;
    a.x_out = x_out;
    a.h = h;
    a.stats = stats;
    return launch_block_norm(a, sms, reinterpret_cast<cudaStream_t>(stream));
  });
}

cbr_status_t cbr_block_norm_workspace_size(const cbr_block_norm_desc_t* desc, size_t* bytes) {
  return guarded([&]() -> int {
    if (const int e = check(desc)) return e;
    if (!bytes) return CBR_ERR_INVALID_ARG;
    *bytes = block_norm_part_floats(*desc) * sizeof(float);
    return CBR_OK;
  });
}

cbr_status_t cbr_block_norm_backward(const cbr_block_norm_desc_t* desc, const void* dx_out, const void* dh,
                                     const void* x_out, const void* branch, const float* post_weight,
                                     const float* gate, const float* pre_weight, const float* stats, void* dx,
                                     void* dbranch, float* dpost_weight, float* dgate, float* dpre_weight,
                                     void* ws, size_t ws_bytes, cbr_stream_t stream) {
  return guarded([&]() -> int {
    if (const int e = check(desc)) return e;
    const cbr_block_norm_desc_t& d = *desc;
    const bool join = post_weight != nullptr;
    if (!join) gate = nullptr;
    if (!gate_rows_ok(d, gate)) return CBR_ERR_INVALID_ARG;
    if ((!join && branch) || (!join && !pre_weight)) return CBR_ERR_INVALID_ARG;
    if ((dx_out && !row_stride(d.dx_out_stride, d.dim, d.rows)) || !row_stride(d.dx_stride, d.dim, d.rows) ||
        (join && (!row_stride(d.branch_stride, d.dim, d.rows) || !row_stride(d.dbranch_stride, d.dim, d.rows))) ||
        (pre_weight && (!row_stride(d.x_out_stride, d.dim, d.rows) || !row_stride(d.dh_stride, d.dim, d.rows))))
      return CBR_ERR_INVALID_ARG;
    if ((join && !dpost_weight) || (pre_weight && !dpre_weight)) return CBR_ERR_INVALID_ARG;
    if (d.rows > 0) {
      if (!dx || !stats || (!pre_weight && !dx_out) || (join && (!branch || !dbranch)) ||
          (pre_weight && (!dh || !x_out)) || (gate && !dgate) || !ws)
        return CBR_ERR_INVALID_ARG;
      if ((dx_out && !same_or_apart(dx, d.dx_stride, dx_out, d.dx_out_stride, d.rows)) || dx == x_out || dx == dh ||
          (branch && (!same_or_apart(dbranch, d.dbranch_stride, branch, d.branch_stride, d.rows) ||
                      !same_or_apart(dbranch, d.dbranch_stride, dh, d.dh_stride, d.rows) || dbranch == dx ||
                      dbranch == x_out || dbranch == dx_out || dx == branch)))
        return CBR_ERR_INVALID_ARG;
    }
    const size_t e = elt(d.dtype);
    if (off(dx_out, e) || off(dh, e) || off(x_out, e) || off(branch, e) || off(dx, e) || off(dbranch, e) ||
        off(post_weight, 4) || off(gate, 4) || off(pre_weight, 4) || off(stats, 4) || off(dpost_weight, 4) ||
        off(dgate, 4) || off(dpre_weight, 4) || off(ws, 16))
      return CBR_ERR_MISALIGNED;
    if (d.rows > 0 && ws_bytes < block_norm_part_floats(d) * sizeof(float)) return CBR_ERR_WORKSPACE;
    int sms = 0;
    uint32_t* err = nullptr;
    if (const int s = device_for_call(&sms, &err)) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (d.rows == 0) {   // sums over no rows
      if (join && cudaMemsetAsync(dpost_weight, 0, d.dim * 4, st) != cudaSuccess) return CBR_ERR_CUDA;
      if (pre_weight && cudaMemsetAsync(dpre_weight, 0, d.dim * 4, st) != cudaSuccess) return CBR_ERR_CUDA;
      return CBR_OK;
    }
    BlockNormArgs a{};
    a.d = d;
    a.x = x_out;
    a.branch = branch;
    a.post_weight = post_weight;
    a.gate = gate;
    a.pre_weight = pre_weight;
    a.stats = const_cast<float*>(stats);
    a.dx_out = dx_out;
    a.dh = dh;
    a.dx = dx;
    a.dbranch = dbranch;
    a.dpost_weight = dpost_weight;
    a.dgate = dgate;
    a.dpre_weight = dpre_weight;
    a.part = static_cast<float*>(ws);
    a.err = err;
    return launch_block_norm_backward(a, sms, st);
  });
}

cbr_status_t cbr_rotary_forward(const cbr_rotary_desc_t* desc, const void* q, const void* k,
                                const int32_t* positions, const int64_t* freq, const uint8_t* axis, void* q_out,
                                void* k_out, cbr_stream_t stream) {
  return guarded([&]() -> int {
    return run(desc, q, k, positions, freq, axis, q_out, k_out, false,
                             reinterpret_cast<cudaStream_t>(stream));
  });
}

cbr_status_t cbr_rotary_backward(const cbr_rotary_desc_t* desc, const void* dq_out, const void* dk_out,
                                 const int32_t* positions, const int64_t* freq, const uint8_t* axis, void* dq,
                                 void* dk, cbr_stream_t stream) {
  return guarded([&]() -> int {
    return run(desc, dq_out, dk_out, positions, freq, axis, dq, dk, true,
                             reinterpret_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
