// C ABI of the trunk operators (declared in include/cbr.h): argument checks and dispatch.
#include <algorithm>
#include <vector>

#include "api_checks.h"
#include "cbr_internal.h"
#include "token_ops.h"
#include "trunk_ops.h"

namespace cbr {
namespace {

constexpr int64_t kMaxTokens = int64_t(1) << 29, kMaxBlocks = (int64_t(1) << 31) - 1;
constexpr int64_t kMaxByteStride = int64_t(1) << 39;   // elements of 16 bits: what a tensor map can hold
constexpr int kMaxAttentionDim = 128, kMaxHeads = 65536, kMaxChannels = 16384, kMaxGroups = 4096;
constexpr int64_t kMaxTensors = int64_t(1) << 20;

int check(const cbr_attention_desc_t* d) {
  if (!d) return CBR_ERR_INVALID_ARG;
  if (!extent(d->batch) || d->q_tokens < 0 || d->k_tokens < 0 || d->heads_q < 1 || d->heads_k < 1 ||
      d->heads_q % d->heads_k || d->head_dim < 1 || !finite(d->scale) || d->scale < 0.f)
    return CBR_ERR_INVALID_ARG;
  if (d->scale > 0x1p127f) return CBR_ERR_UNSUPPORTED;   // times log2(e) it is to stay finite
  if ((d->dtype != CBR_F16 && d->dtype != CBR_BF16) || d->head_dim > kMaxAttentionDim || d->head_dim % 8 ||
      d->q_tokens > kMaxTokens || d->k_tokens > kMaxTokens || d->heads_q > kMaxHeads)
    return CBR_ERR_UNSUPPORTED;
  // the launches' blocks, one for each 128 queries and one for each 128 keys of a head (64 of either where D and the
  // bounds are taken) and one tile more at the most, stay far below 2^31
  const int64_t tiles = std::max(d->q_tokens, d->k_tokens) / 128 + 1;
  if (d->batch > (int64_t(1) << 28) / d->heads_q / tiles) return CBR_ERR_UNSUPPORTED;
  return CBR_OK;
}

// Strides of an attention operand [batch][tokens][heads]: multiples of 16 bytes; inputs may repeat over
// sequences and heads, not over tokens.
int check_strides(const cbr_attention_desc_t& d, const int64_t* s, int64_t tokens, int32_t heads, bool output) {
  const int64_t steps[3] = {d.batch, tokens, heads};
  for (int i = 0; i < 3; ++i) {
    if (steps[i] <= 1) continue;
    if (s[i] < 0 || s[i] >= kMaxByteStride || !in_reach(s[i], steps[i])) return CBR_ERR_INVALID_ARG;
    if (s[i] % 8) return CBR_ERR_MISALIGNED;
  }
  if (tokens > 1 && s[1] < d.head_dim) return CBR_ERR_INVALID_ARG;
  if (output && !distinct(s, d.batch, tokens, heads, d.head_dim)) return CBR_ERR_INVALID_ARG;
  return CBR_OK;
}

int check(const cbr_group_norm_desc_t* d) {
  if (!d) return CBR_ERR_INVALID_ARG;
  if (d->images < 0 || d->pixels < 0 || d->channels < 1 || d->groups < 1 || d->channels % d->groups)
    return CBR_ERR_INVALID_ARG;
  if (d->act != CBR_ACT_NONE && d->act != CBR_ACT_RELU && d->act != CBR_ACT_SILU) return CBR_ERR_INVALID_ARG;
  if (!known_dtype(d->dtype) || d->channels > kMaxChannels || d->groups > kMaxGroups || d->images > kMaxBlocks || d->pixels > kMaxBlocks)
    return CBR_ERR_UNSUPPORTED;
  return CBR_OK;
}

// Images and pixels of a feature map do not share memory.
bool map_strides(const cbr_group_norm_desc_t& d, const int64_t* s) {
  for (int i = 0; i < 2; ++i)
    if (!extent(s[i]) || !in_reach(s[i], i ? d.pixels : d.images)) return false;
  const int64_t axes[3] = {s[0], s[1], 0};
  return distinct(axes, d.images, d.pixels, 1, d.channels);
}

// Whether an out shares memory with another out or with a gradient that is not its own: which of the two a block would
// read or write last is chance.  (Gradients that are only read may share theirs.)
bool outs_overlap(int64_t count, const void* const* grads, const int64_t* sizes, const int32_t* dtypes, void* const* outs) {
  struct Range {
    uintptr_t begin, end;
    bool out;
  };
  std::vector<Range> r;
  r.reserve(2 * count);
  for (int64_t i = 0; i < count; ++i) {
    if (!sizes[i]) continue;
    const uintptr_t bytes = (uintptr_t)sizes[i] * elt(dtypes[i]), g = reinterpret_cast<uintptr_t>(grads[i]), o = reinterpret_cast<uintptr_t>(outs[i]);
    r.push_back({o, o + bytes, true});
    if (g != o) r.push_back({g, g + bytes, false});
  }
  std::sort(r.begin(), r.end(), [](const Range& a, const Range& b) { return a.begin < b.begin; });
  uintptr_t any = 0, out = 0;   // the furthest ends so far
  for (const Range& x : r) {
    if (x.begin < (x.out ? any : out)) return true;
    any = std::max(any, x.end);
    if (x.out) out = std::max(out, x.end);
  }
  return false;
}

bool same_map(const cbr_group_norm_desc_t& d, const int64_t* a, const int64_t* b) {
  return (d.images <= 1 || a[0] == b[0]) && (d.pixels <= 1 || a[1] == b[1]);
}

}  // namespace
}  // namespace cbr

using namespace cbr;

extern "C" {

cbr_status_t cbr_attention_workspace_size(const cbr_attention_desc_t* desc, size_t* fwd_bytes, size_t* bwd_bytes) {
  return guarded([&]() -> int {
    if (const int e = check(desc)) return e;
    if (fwd_bytes) *fwd_bytes = attention_forward_ws(*desc);
    if (bwd_bytes) *bwd_bytes = attention_backward_ws(*desc);
    return CBR_OK;
  });
}

cbr_status_t cbr_attention_forward(const cbr_attention_desc_t* desc, const void* q, const void* k, const void* v,
                                   const int32_t* key_lengths, const int32_t* query_start, void* o, float* lse,
                                   void* ws, size_t ws_bytes, cbr_stream_t stream) {
  return guarded([&]() -> int {
    if (const int e = check(desc)) return e;
    const cbr_attention_desc_t& d = *desc;
    if (const int e = check_strides(d, d.q_stride, d.q_tokens, d.heads_q, false)) return e;
    if (const int e = check_strides(d, d.k_stride, d.k_tokens, d.heads_k, false)) return e;
    if (const int e = check_strides(d, d.v_stride, d.k_tokens, d.heads_k, false)) return e;
    if (const int e = check_strides(d, d.o_stride, d.q_tokens, d.heads_q, true)) return e;
    if (d.batch == 0 || d.q_tokens == 0) return CBR_OK;
    if (!q || !o || (d.k_tokens && (!k || !v)) || o == q || o == k || o == v) return CBR_ERR_INVALID_ARG;
    if (off(q, 16) || off(k, 16) || off(v, 16) || off(o, 16) || off(lse, 4) || off(key_lengths, 4) ||
        off(query_start, 4) || off(ws, 16))
      return CBR_ERR_MISALIGNED;
    const size_t need = attention_forward_ws(d);
    if (need && !ws) return CBR_ERR_INVALID_ARG;
    if (need && ws_bytes < need) return CBR_ERR_WORKSPACE;
    AttentionArgs a{};
    int sms = 0;
    if (const int s = device_for_call(&sms, &a.err)) return s;
    a.d = d;
    a.q = q;
    a.k = k;
    a.v = v;
    a.key_lengths = key_lengths;
    a.query_start = query_start;
    a.o = o;
    a.lse = lse;
    a.ws = ws;
    return launch_attention(a, reinterpret_cast<cudaStream_t>(stream));
  });
}

cbr_status_t cbr_attention_backward(const cbr_attention_desc_t* desc, const void* d_o, const void* q, const void* k,
                                    const void* v, const void* o, const float* lse, const int32_t* key_lengths,
                                    const int32_t* query_start, void* dq, void* dk, void* dv, void* ws,
                                    size_t ws_bytes, cbr_stream_t stream) {
  return guarded([&]() -> int {
    if (const int e = check(desc)) return e;
    const cbr_attention_desc_t& d = *desc;
    if (const int e = check_strides(d, d.q_stride, d.q_tokens, d.heads_q, false)) return e;
    if (const int e = check_strides(d, d.k_stride, d.k_tokens, d.heads_k, false)) return e;
    if (const int e = check_strides(d, d.v_stride, d.k_tokens, d.heads_k, false)) return e;
    if (const int e = check_strides(d, d.o_stride, d.q_tokens, d.heads_q, false)) return e;
    if (const int e = check_strides(d, d.do_stride, d.q_tokens, d.heads_q, false)) return e;
    if (const int e = check_strides(d, d.dq_stride, d.q_tokens, d.heads_q, true)) return e;
    if (const int e = check_strides(d, d.dk_stride, d.k_tokens, d.heads_k, true)) return e;
    if (const int e = check_strides(d, d.dv_stride, d.k_tokens, d.heads_k, true)) return e;
    if (d.batch == 0 || (d.q_tokens == 0 && d.k_tokens == 0)) return CBR_OK;
    if ((d.q_tokens && (!d_o || !q || !o || !lse || !dq)) || (d.k_tokens && (!k || !v || !dk || !dv)))
      return CBR_ERR_INVALID_ARG;
    const void* in[5] = {d_o, q, k, v, o};
    const void* out[3] = {dq, dk, dv};
    for (int i = 0; i < 3; ++i) {
      for (const void* p : in)
        if (out[i] && out[i] == p) return CBR_ERR_INVALID_ARG;
      if (out[i] && out[i] == out[(i + 1) % 3]) return CBR_ERR_INVALID_ARG;
    }
    if (off(d_o, 16) || off(q, 16) || off(k, 16) || off(v, 16) || off(o, 16) || off(lse, 4) || off(key_lengths, 4) ||
        off(query_start, 4) || off(dq, 16) || off(dk, 16) || off(dv, 16) || off(ws, 16))
      return CBR_ERR_MISALIGNED;
    const size_t need = attention_backward_ws(d);
    if (need && !ws) return CBR_ERR_INVALID_ARG;
    if (need && ws_bytes < need) return CBR_ERR_WORKSPACE;
    AttentionArgs a{};
    int sms = 0;
    if (const int s = device_for_call(&sms, &a.err)) return s;
    a.d = d;
    a.q = q;
    a.k = k;
    a.v = v;
    a.key_lengths = key_lengths;
    a.query_start = query_start;
    a.o = const_cast<void*>(o);
    a.lse = const_cast<float*>(lse);
    a.d_o = d_o;
    a.dq = dq;
    a.dk = dk;
    a.dv = dv;
    a.ws = ws;
    return launch_attention_backward(a, reinterpret_cast<cudaStream_t>(stream));
  });
}

cbr_status_t cbr_group_norm_workspace_size(const cbr_group_norm_desc_t* desc, size_t* fwd_bytes, size_t* bwd_bytes) {
  return guarded([&]() -> int {
    if (const int e = check(desc)) return e;
    if (fwd_bytes) *fwd_bytes = group_norm_forward_floats(*desc) * sizeof(float);
    if (bwd_bytes) *bwd_bytes = group_norm_backward_floats(*desc, true) * sizeof(float);
    return CBR_OK;
  });
}

cbr_status_t cbr_group_norm_forward(const cbr_group_norm_desc_t* desc, const void* x, const float* gamma,
                                    const float* beta, void* y, float* mean, float* rstd, void* ws, size_t ws_bytes,
                                    cbr_stream_t stream) {
  return guarded([&]() -> int {
    if (const int e = check(desc)) return e;
    const cbr_group_norm_desc_t& d = *desc;
    if (!(d.eps > 0.f) || !finite(d.eps) || !map_strides(d, d.x_stride) || !map_strides(d, d.y_stride) || !gamma != !beta)
      return CBR_ERR_INVALID_ARG;
    if (d.images == 0 || d.pixels == 0) return CBR_OK;
    if (!x || !y || !mean || !rstd || (x == y && !same_map(d, d.x_stride, d.y_stride))) return CBR_ERR_INVALID_ARG;
    const size_t e = elt(d.dtype);
    if (off(x, e) || off(y, e) || off(gamma, 4) || off(beta, 4) || off(mean, 4) || off(rstd, 4) || off(ws, 16))
      return CBR_ERR_MISALIGNED;
    const size_t need = group_norm_forward_floats(d) * sizeof(float);
    if (need && !ws) return CBR_ERR_INVALID_ARG;
    if (need && ws_bytes < need) return CBR_ERR_WORKSPACE;
    GroupNormArgs a{};
    if (const int s = device_for_call(&a.num_sms, &a.err)) return s;
    a.d = d;
    a.x = x;
    a.gamma = gamma;
    a.beta = beta;
    a.y = y;
    a.mean = mean;
    a.rstd = rstd;
    a.part = static_cast<float*>(ws);
    return launch_group_norm(a, reinterpret_cast<cudaStream_t>(stream));
  });
}

cbr_status_t cbr_group_norm_backward(const cbr_group_norm_desc_t* desc, const void* dy, const void* x,
                                     const float* gamma, const float* beta, const float* mean, const float* rstd,
                                     void* dx, float* dgamma, float* dbeta, void* ws, size_t ws_bytes,
                                     cbr_stream_t stream) {
  return guarded([&]() -> int {
    if (const int e = check(desc)) return e;
    const cbr_group_norm_desc_t& d = *desc;
    if (!map_strides(d, d.x_stride) || !map_strides(d, d.dy_stride) || !map_strides(d, d.dx_stride) || !gamma != !beta ||
        !gamma != !dgamma || !gamma != !dbeta)
      return CBR_ERR_INVALID_ARG;
    const bool empty = d.images == 0 || d.pixels == 0;
    if (!empty && (!dy || !x || !mean || !rstd || !dx || dx == x ||
                   (dx == dy && !same_map(d, d.dx_stride, d.dy_stride))))
      return CBR_ERR_INVALID_ARG;
    const size_t e = elt(d.dtype);
    if (off(dy, e) || off(x, e) || off(dx, e) || off(gamma, 4) || off(beta, 4) || off(mean, 4) || off(rstd, 4) ||
        off(dgamma, 4) || off(dbeta, 4) || off(ws, 16))
      return CBR_ERR_MISALIGNED;
    const size_t need = empty ? 0 : group_norm_backward_floats(d, gamma != nullptr) * sizeof(float);
    if (need && !ws) return CBR_ERR_INVALID_ARG;
    if (need && ws_bytes < need) return CBR_ERR_WORKSPACE;
    GroupNormArgs a{};
    if (const int s = device_for_call(&a.num_sms, &a.err)) return s;
    cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
    if (empty) {   // sums over no pixels
      if (gamma && (cudaMemsetAsync(dgamma, 0, d.channels * 4, st) != cudaSuccess ||
                    cudaMemsetAsync(dbeta, 0, d.channels * 4, st) != cudaSuccess))
        return CBR_ERR_CUDA;
      return CBR_OK;
    }
    a.d = d;
    a.x = x;
    a.gamma = gamma;
    a.beta = beta;
    a.mean = const_cast<float*>(mean);
    a.rstd = const_cast<float*>(rstd);
    a.dy = dy;
    a.dx = dx;
    a.dgamma = dgamma;
    a.dbeta = dbeta;
    a.part = static_cast<float*>(ws);
    return launch_group_norm_backward(a, st);
  });
}

cbr_status_t cbr_clip_workspace_size(int64_t count, size_t* bytes) {
  return guarded([&]() -> int {
    if (count < 0 || !bytes) return CBR_ERR_INVALID_ARG;
    if (count > kMaxTensors) return CBR_ERR_UNSUPPORTED;
    *bytes = clip_part_doubles(count) * sizeof(double);
    return CBR_OK;
  });
}

cbr_status_t cbr_clip_gradients(int64_t count, const void* const* grads, const int64_t* sizes, const int32_t* dtypes,
                                void* const* outs, float max_norm, float unscale, float* norm, float* scale,
                                void* ws, size_t ws_bytes, cbr_stream_t stream) {
  return guarded([&]() -> int {
    if (count < 0 || (count && (!grads || !sizes || !dtypes)) || !(max_norm >= 0.f) || !(unscale > 0.f) ||
        !finite(unscale) || !norm || !scale || norm == scale || !ws)
      return CBR_ERR_INVALID_ARG;
    if (count > kMaxTensors) return CBR_ERR_UNSUPPORTED;
    for (int64_t i = 0; i < count; ++i) {
      if (!extent(sizes[i]) || (sizes[i] && (!grads[i] || (outs && !outs[i])))) return CBR_ERR_INVALID_ARG;
      if (!known_dtype(dtypes[i])) return CBR_ERR_UNSUPPORTED;
      if (off(grads[i], elt(dtypes[i])) || (outs && off(outs[i], elt(dtypes[i])))) return CBR_ERR_MISALIGNED;
    }
    if (off(norm, 4) || off(scale, 4) || off(ws, 16)) return CBR_ERR_MISALIGNED;
    if (outs && outs_overlap(count, grads, sizes, dtypes, outs)) return CBR_ERR_INVALID_ARG;
    if (ws_bytes < clip_part_doubles(count) * sizeof(double)) return CBR_ERR_WORKSPACE;
    const ClipArgs a{count, grads, sizes, dtypes, outs, max_norm, unscale, norm, scale, static_cast<double*>(ws)};
    int sms = 0;
    uint32_t* err = nullptr;
    if (const int s = device_for_call(&sms, &err)) return s;
    return launch_clip(a, reinterpret_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
