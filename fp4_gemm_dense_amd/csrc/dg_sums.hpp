// Sums of partial rows in a fixed order (norm.hip, activation.hip).
#pragma once

#include "dg_device.hpp"

namespace dg {

// Sums of `rows` partial rows, `stride` floats apart: a workgroup of 256 sums 32 columns,
// 8 threads (4 columns each) across and 32 down, each every 32nd row; their sums meet in
// LDS in order.  first: where row 0 lies apart, its distance from its place.
__device__ __forceinline__ void sum_rows(const float* part, int stride, int rows, float* out, int first = 0) {
  __shared__ v4f sums[32][8];
  const int cx = threadIdx.x & 7, ry = threadIdx.x >> 3;
  const float* src = part + (size_t)blockIdx.x * 32 + cx * 4;
  v4f s = {0.f, 0.f, 0.f, 0.f};
  for (int i = ry; i < rows; i += 8 * 32) {
    v4f t[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      t[u] = i + u * 32 < rows ? *reinterpret_cast<const v4f*>(src + (size_t)(i + u * 32) * stride + (i + u * 32 ? 0 : first))
                               : v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < 8; ++u) s += t[u];
  }
  sums[ry][cx] = s;
  __syncthreads();
  if (threadIdx.x < 8) {
    v4f t = sums[0][threadIdx.x];
#pragma unroll
    for (int y = 1; y < 32; ++y) t += sums[y][threadIdx.x];
    *reinterpret_cast<v4f*>(out + (size_t)blockIdx.x * 32 + threadIdx.x * 4) = t;
  }
}

}  // namespace dg
