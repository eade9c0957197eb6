// rope_axes.h — the split of a head's pairs over the axes of its position.
#pragma once

#include <cuda_runtime.h>

namespace lrkv {

constexpr int kMaxAxes = 4;

// Pairs [end[a - 1], end[a]) turn by the position on axis a.
struct RopeAxes {
  int n;
  int end[kMaxAxes];
  __host__ __device__ __forceinline__ int axis(int k) const {
    int a = 0;
#pragma unroll
    for (int i = 0; i < kMaxAxes - 1; ++i) a += (i < n - 1 && k >= end[i]) ? 1 : 0;
    return a;
  }
};

// False unless 1 <= axes <= 4 and the sections (pairs per axis, none negative)
// add up to head_dim / 2.
inline bool rope_axes_make(int axes, const int* sections, int head_dim, RopeAxes& out) {
  if (axes < 1 || axes > kMaxAxes || !sections || head_dim < 2 || head_dim % 2 != 0) return false;
  long long sum = 0;
  out.n = axes;
  for (int a = 0; a < kMaxAxes; ++a) {
    if (a < axes) {
      if (sections[a] < 0) return false;
      sum += sections[a];
    }
    if (sum > head_dim / 2) return false;
    out.end[a] = static_cast<int>(sum);
  }
  return sum == head_dim / 2;
}

}  // namespace lrkv
