// The order of the tasks in group norm's stream (group_norm.cu), on the host, too.
#pragma once
#include <cstdint>

#ifdef __CUDACC__
#define CBR_ANYWHERE __host__ __device__ __forceinline__
#else
#define CBR_ANYWHERE inline
#endif

namespace cbr {
namespace gn {

// Step s of the tasks has the moments (sums) of image s, run by run; the merge of image s - half's moments; and the results
// of image s - lag, run by run.  1 <= half <= lag <= images.
struct Order {
  uint32_t images, runs, half, lag;
};
enum Kind { kMoments, kMerge, kResult };
struct Task {
  Kind kind;
  uint32_t image, run;

  // The i-th task.
  static CBR_ANYWHERE Task of(const Order& f, uint32_t i) {
    // steps of the same size: before the first merge, before the first result, with all three, without moments, with
    // results alone
    uint32_t step = 0, size = f.runs, n = f.half * f.runs;
    bool first = true, merge = false;
    if (i >= n) {
      i -= n, step = f.half, size = f.runs + 1, n = (f.lag - f.half) * size, merge = true;
      if (i >= n) {
        i -= n, step = f.lag, size = 2 * f.runs + 1, n = (f.images - f.lag) * size;
        if (i >= n) {
          i -= n, step = f.images, size = f.runs + 1, n = f.half * size, first = false;
          if (i >= n) i -= n, step = f.images + f.half, size = f.runs, merge = false;
        }
      }
    }
    const uint32_t past = i / size;
    i -= past * size;
    step += past;
    if (first) {
      if (i < f.runs) return Task{kMoments, step, i};
      i -= f.runs;
    }
    if (merge) {
      if (i == 0) return Task{kMerge, step - f.half, 0};
      --i;
    }
    return Task{kResult, step - f.lag, i};
  }
  static CBR_ANYWHERE uint32_t total(uint32_t images, uint32_t runs) { return images * (2 * runs + 1); }
};

}  // namespace gn
}  // namespace cbr
