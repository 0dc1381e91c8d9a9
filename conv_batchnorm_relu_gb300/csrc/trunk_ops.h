// Host-side interface between the trunk operators' C ABI (trunk_api.cu) and their kernels.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

#include "../../include/cbr.h"

namespace cbr {

struct AttentionArgs {
  cbr_attention_desc_t d;
  const void* q;
  const void* k;
  const void* v;
  const int32_t* key_lengths;  // null: k_tokens
  const int32_t* query_start;  // null: 0
  void* o;                     // forward: out, backward: in
  float* lse;                  // forward: out (may be null), backward: in
  const void* d_o;             // backward
  void* dq;
  void* dk;
  void* dv;
  void* ws;
  uint32_t* err;
};
size_t attention_forward_ws(const cbr_attention_desc_t& d);
size_t attention_backward_ws(const cbr_attention_desc_t& d);
int launch_attention(const AttentionArgs& a, cudaStream_t st);
int launch_attention_backward(const AttentionArgs& a, cudaStream_t st);

struct GroupNormArgs {
  cbr_group_norm_desc_t d;
  const void* x;
  const float* gamma;          // null: ones (and beta zeros)
  const float* beta;
  void* y;
  float* mean;                 // forward: out, backward: in
  float* rstd;
  const void* dy;              // backward
  void* dx;
  float* dgamma;
  float* dbeta;
  float* part;
  int num_sms;
  uint32_t* err;
};
size_t group_norm_forward_floats(const cbr_group_norm_desc_t& d);
size_t group_norm_backward_floats(const cbr_group_norm_desc_t& d, bool parameters);
int launch_group_norm(const GroupNormArgs& a, cudaStream_t st);
int launch_group_norm_backward(const GroupNormArgs& a, cudaStream_t st);

struct ClipArgs {
  int64_t count;
  const void* const* grads;
  const int64_t* sizes;
  const int32_t* dtypes;
  void* const* outs;           // null: norm and scale only
  float max_norm, unscale;
  float* norm;
  float* scale;
  double* part;
};
size_t clip_part_doubles(int64_t count);
int launch_clip(const ClipArgs& a, cudaStream_t st);

}  // namespace cbr
