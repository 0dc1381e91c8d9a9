// Host-side interface between the token operators' C ABI (tokens_api.cu) and their kernels.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/cbr.h"

namespace cbr {

// Runs the body of a C entry: a C++ exception (the caches of launch shapes take memory and a lock) ends in a
// status, not in the caller.
template <typename F>
cbr_status_t guarded(F&& body) noexcept {
  try {
    return static_cast<cbr_status_t>(body());
  } catch (...) {
    return CBR_ERR_CUDA;
  }
}

// The current device if this library runs on it (cbr_api.cu): its SM count and its error word.
int device_for_call(int* num_sms, uint32_t** err);

// Blocks of `threads` threads and `smem` bytes of dynamic shared memory that fit on an SM at once; 0 if the
// runtime refuses.  Asked once for each kernel, shape and device (block_norm.cu).
int blocks_that_fit(const void* kernel, int threads, int smem);

struct DistillArgs {
  cbr_distill_desc_t d;
  const float* dloss;        // null: ones
  const void* logits;
  const void* top_ids;
  const void* top_logits;
  const float* teacher_lse;  // null: the teacher is renormalised over its entries
  const float* row_weight;   // null: ones
  float* loss;
  float* stats;              // [rows][3]; written by the forward (may be null), read by the backward
  void* dlogits;             // null: loss only
  uint32_t* err;
};
// Loss (and gradient, where dlogits is set) / gradient from the forward's stats (distill.cu).
int launch_distill(const DistillArgs& a, cudaStream_t st);
int launch_distill_backward(const DistillArgs& a, cudaStream_t st);

struct BlockNormArgs {
  cbr_block_norm_desc_t d;
  const void* x;             // backward: x_out
  const void* branch;
  const float* post_weight;
  const float* gate;
  const float* pre_weight;
  void* x_out;
  void* h;
  float* stats;
  const void* dx_out;
  const void* dh;
  void* dx;
  void* dbranch;
  float* dpost_weight;
  float* dgate;
  float* dpre_weight;
  float* part;               // backward: per-block sums
  uint32_t* err;
};
int launch_block_norm(const BlockNormArgs& a, int num_sms, cudaStream_t st);
int launch_block_norm_backward(const BlockNormArgs& a, int num_sms, cudaStream_t st);
size_t block_norm_part_floats(const cbr_block_norm_desc_t& d);

struct RotaryArgs {
  cbr_rotary_desc_t d;
  const void* q;
  const void* k;
  const int32_t* positions;
  const int64_t* freq;
  const uint8_t* axis;
  void* q_out;
  void* k_out;
  bool backward;
};
int launch_rotary(const RotaryArgs& a, int num_sms, cudaStream_t st);

}  // namespace cbr
