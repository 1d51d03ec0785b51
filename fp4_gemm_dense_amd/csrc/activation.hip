// The backward pass through a linear layer's activation for gfx950: dz = dy * act'(z), or of a
// gated one dz = [dy * up * act'(gate), dy * act(gate)], quantised to MXFP4 for the products of
// the layer's gradients (along the rows for the input's, along the columns of the transposed
// operand for the weight's), with the bias gradient's column sums from the same read.
//
// dz is rounded to bf16 and quantised from there, so that the codes are those of the values
// that dz stores; the sums take the unrounded ones.
//
// Bound: HBM.  An element of dz costs 2 bytes of z and 2 of dy (gated: 1) of reading and
// 17/32 of writing per direction.
#include <algorithm>

#include "../../include/dg.h"
#include "dg_activation.hpp"
#include "dg_internal.hpp"
#include "dg_quant.hpp"
#include "dg_sums.hpp"
#include "quant_tile.hpp"

namespace dg {

struct ActBackParams {
  const uint16_t* dy;
  const uint16_t* z;   // null: the identity's
  uint16_t* dz;
  uint8_t* q;
  int32_t* sf;
  uint8_t* qt;
  int32_t* sft;
  float* part;         // [ceil(m / 128)][n] of dbias, or null
  int m, n;
  Activation act;
};

// One workgroup takes 128 rows x 128 columns (gated: of both halves, one after the other),
// quantises the rows from registers on the way into LDS and the columns from there.
template <bool GATED>
__global__ void __launch_bounds__(256) activation_backward_kernel(ActBackParams p) {
  __shared__ QuantTile<uint16_t> lds;
  __shared__ float sums[16][128];
  const int tid = threadIdx.x;
  const int w = GATED ? p.n >> 1 : p.n;                         // columns of dy
  const uint32_t kb_n = (uint32_t)w >> 7, mb_n = ((uint32_t)p.m + 127) >> 7;
  const long long total = (long long)mb_n * kb_n;
  const int rr = tid >> 4, c = (tid & 15) * 8;
  for (long long t = blockIdx.x; t < total; t += gridDim.x) {
    const uint32_t mb = (uint32_t)(t / kb_n), kb = (uint32_t)(t - (long long)mb * kb_n);
    const int rows = min(128, p.m - (int)(mb * 128u));
    Vec8<uint16_t> g[8], up[GATED ? 8 : 1];
    float sum[8], sum_up[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = sum_up[e] = 0.f;
    const size_t at_dy = (size_t)mb * 128u * w + kb * 128u + c, at_z = (size_t)mb * 128u * p.n + kb * 128u + c;
    v4i vy[8], vz[8], vu[GATED ? 8 : 1];
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int r = s * 16 + rr;
      const v4i none = {0, 0, 0, 0};
      vy[s] = r < rows ? *reinterpret_cast<const v4i*>(p.dy + at_dy + (size_t)r * w) : none;
      vz[s] = r < rows && p.z ? *reinterpret_cast<const v4i*>(p.z + at_z + (size_t)r * p.n) : none;
      if constexpr (GATED) vu[s] = r < rows ? *reinterpret_cast<const v4i*>(p.z + at_z + (size_t)r * p.n + w) : none;
    }
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      float y[8], z[8], a[8], d[8];
      unpack_bf16x8(vy[s], y);
      unpack_bf16x8(vz[s], z);
      activate_both<8>(z, a, d, p.act);
      if constexpr (GATED) {
        float u[8];
        unpack_bf16x8(vu[s], u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          d[e] *= y[e] * u[e];
          a[e] *= y[e];
          sum_up[e] += a[e];
        }
        up[s].p = pack_bf16x8(a);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] *= y[e];
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[e] += d[e];
      g[s].p = pack_bf16x8(d);
    }
    auto put = [&](const Vec8<uint16_t>(&v)[8], uint32_t col0) {
      if (p.dz) {
#pragma unroll
        for (int s = 0; s < 8; ++s)
          if (s * 16 + rr < rows)
            *reinterpret_cast<v4i*>(p.dz + ((size_t)mb * 128u + s * 16 + rr) * p.n + col0 + c) = v[s].p;
      }
      if (!p.q && !p.qt) return;   // (uniform)
      const size_t half_mp = (size_t)mb_n * 64;
      quantize_tile(lds, v, rows,
                    QuantOut{p.q ? reinterpret_cast<uint32_t*>(p.q) + (((size_t)mb * 128u * p.n + col0) >> 3) : nullptr, nullptr,
                             p.sf ? p.sf + (size_t)(col0 >> 7) * p.m + mb * 128u : nullptr,
                             p.qt ? p.qt + (size_t)col0 * half_mp + (size_t)mb * 64 : nullptr,
                             p.sft ? p.sft + (size_t)mb * p.n + col0 : nullptr, (size_t)p.n >> 3, half_mp});
    };
    auto put_sums = [&](const float(&v)[8], uint32_t col0) {
      // 16 threads down a column, added in order
#pragma unroll
      for (int e = 0; e < 8; ++e) sums[rr][c + e] = v[e];
      __syncthreads();
      if (tid < 128) {
        float t = sums[0][tid];
#pragma unroll
        for (int y = 1; y < 16; ++y) t += sums[y][tid];
        p.part[(size_t)mb * p.n + col0 + tid] = t;
      }
      __syncthreads();
    };
    put(g, kb * 128u);
    if constexpr (GATED) put(up, (uint32_t)w + kb * 128u);
    if (p.part) {
      put_sums(sum, kb * 128u);
      if constexpr (GATED) put_sums(sum_up, (uint32_t)w + kb * 128u);
    }
  }
}

// dbias: the partial rows' sums, 32 columns a workgroup.
__global__ void __launch_bounds__(256) activation_dbias_kernel(const float* part, float* dbias, int parts, int n) {
  sum_rows(part, n, parts, dbias);
}

static bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

// (a place of z is a size_t; rows and blocks are ints)
static bool activation_backward_fits(int m, int n, bool gated) {
  return n % (gated ? 256 : 128) == 0 && m <= 0x7fffffff - 127;
}

}  // namespace dg

using namespace dg;

extern "C" {

size_t dg_activation_backward_workspace_bytes(int m, int n) {
  if (m <= 0 || n <= 0 || !activation_backward_fits(m, n, false)) return 0;
  return m <= 128 ? 0 : (size_t)((m + 127) / 128) * n * sizeof(float);
}

int dg_activation_backward(const uint16_t* dy, const uint16_t* z, int activation, uint16_t* dz, uint8_t* q, int32_t* sf,
                           uint8_t* qt, int32_t* sft, float* dbias, int m, int n, void* workspace, size_t workspace_bytes,
                           void* stream) {
  try {
    Activation act;
    if (!dy || (!dz && !q && !qt && !dbias) || !q != !sf || !qt != !sft || !activation_of(activation, &act))
      return DG_ERR_INVALID_ARG;
    if (!z && activation != DG_ACT_NONE) return DG_ERR_INVALID_ARG;
    if (m <= 0 || n <= 0) return DG_ERR_INVALID_ARG;
    if (misaligned(dy, 16) || misaligned(z, 16) || misaligned(dz, 16) || misaligned(q, 16) || misaligned(qt, 16) ||
        misaligned(sf, 4) || misaligned(sft, 4) || misaligned(dbias, 16))
      return DG_ERR_INVALID_ARG;
    const bool gated = activation & DG_ACT_GATED;
    if (!activation_backward_fits(m, n, gated)) return DG_ERR_UNSUPPORTED;
    const size_t need = dbias ? dg_activation_backward_workspace_bytes(m, n) : 0;
    if (need && (!workspace || workspace_bytes < need || misaligned(workspace, 16))) return DG_ERR_INVALID_ARG;
    DeviceInfo di = current_device_info();
    if (!di.ok) return DG_ERR_NO_DEVICE;
    const int mb = (int)(((long long)m + 127) / 128), cols = gated ? n / 2 : n;
    // (up to 128 rows the one partial row is dbias)
    float* const part = !dbias ? nullptr : need ? static_cast<float*>(workspace) : dbias;
    const ActBackParams p{dy, z, dz, q, sf, qt, sft, part, m, n, act};
    const int grid = (int)std::min<long long>((long long)mb * (cols / 128), (long long)dg_get_num_cus() * 8);
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    if (gated) hipLaunchKernelGGL(activation_backward_kernel<true>, dim3(grid), dim3(256), 0, hs, p);
    else hipLaunchKernelGGL(activation_backward_kernel<false>, dim3(grid), dim3(256), 0, hs, p);
    if (hipGetLastError() != hipSuccess) return DG_ERR_HIP;
    if (!need) return DG_OK;
    hipLaunchKernelGGL(activation_dbias_kernel, dim3(n / 32), dim3(256), 0, hs, part, dbias, mb, n);
    return hipGetLastError() == hipSuccess ? DG_OK : DG_ERR_HIP;
  } catch (...) {
    return DG_ERR_HIP;
  }
}

}  // extern "C"
