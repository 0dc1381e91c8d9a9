// Rotary positions over several axes (formulas: include/cbr.h).
//
// One block a token: the cosines and sines of its pairs once into shared memory, then all heads of
// q and k.  The angle is a product modulo 2^64 of the position and the frequency in turns, so it
// is reduced to one turn without rounding; its top 32 bits, as a signed fraction of half a turn,
// go to sincospif.
#include <algorithm>

#include "cbr_internal.h"
#include "token_ops.cuh"

namespace cbr {
namespace {

using namespace tok;

constexpr int kThreads = 256;

template <typename T>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const __grid_constant__ RotaryArgs a) {
  __shared__ float2 turn[512];
  const cbr_rotary_desc_t& d = a.d;
  const int pairs = d.rot_dim / 2, heads = d.heads_q + d.heads_k;
  const long long total = d.batch * d.tokens;
  for (long long i = blockIdx.x; i < total; i += gridDim.x) {
    const long long b = i / d.tokens, t = i % d.tokens;
    __syncthreads();
    for (int p = threadIdx.x; p < pairs; p += kThreads) {
      const int ax = min((int)a.axis[p], d.axes - 1);
      const long long pos = a.positions[b * d.pos_stride[0] + t * d.pos_stride[1] + ax * d.pos_stride[2]];
      const unsigned long long f = (unsigned long long)pos * (unsigned long long)a.freq[p];
      float sn, cs;
      sincospif((float)(int)(f >> 32) * 0x1p-31f, &sn, &cs);
      turn[p] = make_float2(cs, a.backward ? -sn : sn);
    }
    __syncthreads();
    for (int e = threadIdx.x; e < heads * d.head_dim; e += kThreads) {
      const int h = e / d.head_dim, c = e % d.head_dim;
      const bool q = h < d.heads_q;
      const int hh = q ? h : h - d.heads_q;
      const int64_t* si = q ? d.q_stride : d.k_stride;
      const int64_t* so = q ? d.q_out_stride : d.k_out_stride;
      const T* in = static_cast<const T*>(q ? a.q : a.k) + b * si[0] + t * si[1] + hh * si[2];
      T* out = static_cast<T*>(q ? a.q_out : a.k_out) + b * so[0] + t * so[1] + hh * so[2];
      if (c >= d.rot_dim) {
        out[c] = in[c];
        continue;
      }
      const bool halves = d.layout == CBR_ROTARY_HALVES;
      const int p = halves ? c : c / 2;
      if (halves ? c >= pairs : c % 2) continue;   // the pair's first element does both
      const int c2 = halves ? c + pairs : c + 1;
      const float x1 = to_f(in[c]), x2 = to_f(in[c2]);
      const float2 cs = turn[p];
      out[c] = from_f<T>(x1 * cs.x - x2 * cs.y);
      out[c2] = from_f<T>(x2 * cs.x + x1 * cs.y);
    }
  }
}

}  // namespace

int launch_rotary(const RotaryArgs& a, int num_sms, cudaStream_t st) {
  const int grid = (int)std::min<long long>(a.d.batch * a.d.tokens, (long long)num_sms * 8);
  if (a.d.dtype == CBR_F32) rotary_kernel<float><<<grid, kThreads, 0, st>>>(a);
  else if (a.d.dtype == CBR_BF16) rotary_kernel<__nv_bfloat16><<<grid, kThreads, 0, st>>>(a);
  else rotary_kernel<__half><<<grid, kThreads, 0, st>>>(a);
  return cudaGetLastError() == cudaSuccess ? CBR_OK : CBR_ERR_CUDA;
}

}  // namespace cbr
