// RMS norm with the residual's addition and a quantised output, and its backward
// pass, for gfx950.
//
// Forward, per row: h = bf16(x + residual), r = 1 / sqrt(mean(h^2) + eps), and
// y = h * r * weight quantised per block (e4m3 with fp32 or UE8M0 scales per 1x128,
// or MXFP4) straight from registers.  The residual stream is stored in bf16, and the
// norm reads the stored value, so that the backward pass sees the same n = h * r.
// Backward, with n = h * r and g = dy * weight: dx = dh + r (g - n mean(g n)),
// dweight = sum over rows of dy * n.
//
// Bound: HBM (forward 7 bytes per element with a residual, backward 8).
#include <algorithm>
#include <cmath>

#include "../../include/dg.h"
#include "dg_internal.hpp"
#include "dg_quant.hpp"

namespace dg {

struct NormParams {
  const uint16_t* x;
  const uint16_t* residual;
  const uint16_t* weight;
  uint16_t* h;
  void* q;
  void* sf;
  float* rstd;
  int m, k;
  float eps;
};

constexpr int NORM_THREADS = 256;

// Sum of v over the workgroup, in a fixed order; every thread gets it.
template <int WAVES>
__device__ __forceinline__ float block_sum(float v, float* red) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) v += __shfl_xor(v, o, 64);
  const int wave = threadIdx.x >> 6;
  __syncthreads();
  if ((threadIdx.x & 63) == 0) red[wave] = v;
  __syncthreads();
  float s = 0.f;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) s += red[w];
  return s;
}

// One workgroup per row; a thread holds V vectors of 8 values, vector i at
// (i * threads + tid): 16 lanes side by side hold one 1x128 block.
template <int FMT, int V>
__global__ void __launch_bounds__(NORM_THREADS) add_rms_norm_kernel(NormParams p) {
  __shared__ float red[NORM_THREADS / 64];
  const int tid = threadIdx.x;
  const int nv = p.k / 8, kb_n = p.k / 128;
  for (int row = blockIdx.x; row < p.m; row += gridDim.x) {
    const size_t base = (size_t)row * nv;
    v4i hv[V];
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = i * NORM_THREADS + tid;
      hv[i] = v4i{0, 0, 0, 0};
      if (j >= nv) continue;
      hv[i] = reinterpret_cast<const v4i*>(p.x)[base + j];
      float a[8];
      unpack_bf16x8(hv[i], a);
      if (p.residual) {
        float b[8];
        unpack_bf16x8(reinterpret_cast<const v4i*>(p.residual)[base + j], b);
#pragma unroll
        for (int e = 0; e < 8; ++e) a[e] += b[e];
        hv[i] = pack_bf16x8(a);
        unpack_bf16x8(hv[i], a);
      }
      if (p.h) reinterpret_cast<v4i*>(p.h)[base + j] = hv[i];
#pragma unroll
      for (int e = 0; e < 8; ++e) ss = fmaf(a[e], a[e], ss);
    }
    const float r = 1.0f / sqrtf(block_sum<NORM_THREADS / 64>(ss, red) / (float)p.k + p.eps);
    if (p.rstd && tid == 0) p.rstd[row] = r;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = i * NORM_THREADS + tid;
      if (j >= nv) continue;
      float y[8], w[8];
      unpack_bf16x8(hv[i], y);
      unpack_bf16x8(reinterpret_cast<const v4i*>(p.weight)[j], w);
      uint32_t amax = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        y[e] = y[e] * r * w[e];
        amax = umax(amax, abs_bits(y[e]));
      }
      const int kb = j >> 4;
      if constexpr (FMT == DG_QUANT_MXFP4) {
        const uint32_t byte = ue8m0_byte<false>(group_max<4>(amax));
        static_cast<uint32_t*>(p.q)[base + j] = byte == 255u ? 0u : e2m1x8(y, ue8m0_value(byte));
        const uint32_t word = scale_word(byte);
        if ((tid & 15) == 0) static_cast<uint32_t*>(p.sf)[(size_t)kb * p.m + row] = word;
      } else {
        amax = group_max<16>(amax);
        float inv;
        if constexpr (FMT == DG_QUANT_E4M3_F32) {
          float s = __uint_as_float(amax) / 448.0f;
          s = amax == 0 ? 1.0f : (amax >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : fmaxf(s, 0x1p-126f));
          inv = 1.0f / s;
          if ((tid & 15) == 0) static_cast<float*>(p.sf)[(size_t)kb * p.m + row] = s;
        } else {
          const uint32_t byte = ue8m0_byte<true>(amax);
          inv = ue8m0_value(byte == 255u ? 255u : 254u - byte);   // 2^(127 - byte)
          if ((tid & 15) == 0) static_cast<uint8_t*>(p.sf)[(size_t)row * ((kb_n + 3) / 4 * 4) + kb] = (uint8_t)byte;
        }
        const v2i c = {(int)e4m3x4(y[0] * inv, y[1] * inv, y[2] * inv, y[3] * inv),
                       (int)e4m3x4(y[4] * inv, y[5] * inv, y[6] * inv, y[7] * inv)};
        static_cast<v2i*>(p.q)[base + j] = c;
      }
    }
    if constexpr (FMT == DG_QUANT_E4M3_UE8M0) {
      const int full = (kb_n + 3) / 4 * 4;   // the last word's unused bytes
      if (tid < full - kb_n) static_cast<uint8_t*>(p.sf)[(size_t)row * full + kb_n + tid] = 127;
    }
  }
}

struct NormBackParams {
  const uint16_t* dy;
  const uint16_t* dh;
  const uint16_t* h;
  const uint16_t* weight;
  const float* rstd;
  uint16_t* dx;
  float* part;   // [workgroups][k]
  int m, k;
};

// A workgroup takes rows blockIdx.x, + gridDim.x, ...; a thread keeps its columns'
// share of dweight in registers over them and writes one partial row at the end.
template <int V>
__global__ void __launch_bounds__(NORM_THREADS) rms_norm_backward_kernel(NormBackParams p) {
  __shared__ float red[NORM_THREADS / 64];
  const int tid = threadIdx.x;
  const int nv = p.k / 8;
  float dw[V][8];
#pragma unroll
  for (int i = 0; i < V; ++i)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
  for (int row = blockIdx.x; row < p.m; row += gridDim.x) {
    const size_t base = (size_t)row * nv;
    const float r = p.rstd[row];
    v4i dyv[V], hv[V];
    float dot = 0.f;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = i * NORM_THREADS + tid;
      dyv[i] = hv[i] = v4i{0, 0, 0, 0};
      if (j >= nv) continue;
      dyv[i] = reinterpret_cast<const v4i*>(p.dy)[base + j];
      hv[i] = reinterpret_cast<const v4i*>(p.h)[base + j];
      float a[8], n[8], w[8];
      unpack_bf16x8(dyv[i], a);
      unpack_bf16x8(hv[i], n);
      unpack_bf16x8(reinterpret_cast<const v4i*>(p.weight)[j], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[e] *= r;
        dw[i][e] = fmaf(a[e], n[e], dw[i][e]);
        dot = fmaf(a[e] * w[e], n[e], dot);
      }
    }
    const float mean = block_sum<NORM_THREADS / 64>(dot, red) / (float)p.k;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = i * NORM_THREADS + tid;
      if (j >= nv) continue;
      float a[8], n[8], w[8], d[8];
      unpack_bf16x8(dyv[i], a);
      unpack_bf16x8(hv[i], n);
      unpack_bf16x8(reinterpret_cast<const v4i*>(p.weight)[j], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = 0.f;
      if (p.dh) unpack_bf16x8(reinterpret_cast<const v4i*>(p.dh)[base + j], d);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] += r * (a[e] * w[e] - n[e] * r * mean);
      reinterpret_cast<v4i*>(p.dx)[base + j] = pack_bf16x8(d);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = i * NORM_THREADS + tid;
    if (j >= nv) continue;
    v4f* o = reinterpret_cast<v4f*>(p.part + (size_t)blockIdx.x * p.k + (size_t)j * 8);
    o[0] = v4f{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
    o[1] = v4f{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
  }
}

__global__ void __launch_bounds__(256) norm_dweight_kernel(const float* part, float* dweight, int parts, int k) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= k) return;
  float s = 0.f;
  for (int i = 0; i < parts; ++i) s += part[(size_t)i * k + c];
  dweight[c] = s;
}

// Rows of partial sums of dweight (workgroups of the backward kernel): a function of
// the sizes alone, so that the sum's order is, too.
static int norm_parts(int m) { return std::min(m, 512); }

constexpr int NORM_MAX_K = 32768;

template <int FMT>
static hipError_t launch_norm(const NormParams& p, int grid, hipStream_t hs) {
  const int v = (p.k / 8 + NORM_THREADS - 1) / NORM_THREADS;
  if (v <= 1) hipLaunchKernelGGL((add_rms_norm_kernel<FMT, 1>), dim3(grid), dim3(NORM_THREADS), 0, hs, p);
  else if (v <= 2) hipLaunchKernelGGL((add_rms_norm_kernel<FMT, 2>), dim3(grid), dim3(NORM_THREADS), 0, hs, p);
  else if (v <= 4) hipLaunchKernelGGL((add_rms_norm_kernel<FMT, 4>), dim3(grid), dim3(NORM_THREADS), 0, hs, p);
  else if (v <= 8) hipLaunchKernelGGL((add_rms_norm_kernel<FMT, 8>), dim3(grid), dim3(NORM_THREADS), 0, hs, p);
  else hipLaunchKernelGGL((add_rms_norm_kernel<FMT, 16>), dim3(grid), dim3(NORM_THREADS), 0, hs, p);
  return hipGetLastError();
}

static hipError_t launch_norm_backward(const NormBackParams& p, int grid, hipStream_t hs) {
  const int v = (p.k / 8 + NORM_THREADS - 1) / NORM_THREADS;
  if (v <= 1) hipLaunchKernelGGL(rms_norm_backward_kernel<1>, dim3(grid), dim3(NORM_THREADS), 0, hs, p);
  else if (v <= 2) hipLaunchKernelGGL(rms_norm_backward_kernel<2>, dim3(grid), dim3(NORM_THREADS), 0, hs, p);
  else if (v <= 4) hipLaunchKernelGGL(rms_norm_backward_kernel<4>, dim3(grid), dim3(NORM_THREADS), 0, hs, p);
  else if (v <= 8) hipLaunchKernelGGL(rms_norm_backward_kernel<8>, dim3(grid), dim3(NORM_THREADS), 0, hs, p);
  else hipLaunchKernelGGL(rms_norm_backward_kernel<16>, dim3(grid), dim3(NORM_THREADS), 0, hs, p);
  return hipGetLastError();
}

}  // namespace dg

using namespace dg;

static bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

extern "C" {

int dg_add_rms_norm(const uint16_t* x, const uint16_t* residual, const uint16_t* weight, uint16_t* h, void* q,
                    void* sf, int format, float* rstd, int m, int k, float eps, void* stream) {
  try {
    if (!x || !weight || !q || !sf) return DG_ERR_INVALID_ARG;
    if (format != DG_QUANT_E4M3_F32 && format != DG_QUANT_E4M3_UE8M0 && format != DG_QUANT_MXFP4)
      return DG_ERR_INVALID_ARG;
    if (m <= 0 || k <= 0 || !(eps > 0.f) || !std::isfinite(eps)) return DG_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(residual, 16) || misaligned(weight, 16) || misaligned(h, 16) ||
        misaligned(q, 16) || misaligned(sf, 4) || misaligned(rstd, 4))
      return DG_ERR_INVALID_ARG;
    if (k % 128 != 0 || k > NORM_MAX_K) return DG_ERR_UNSUPPORTED;
    DeviceInfo di = current_device_info();
    if (!di.ok) return DG_ERR_NO_DEVICE;
    int cus = dg_get_num_cus();
    if (cus <= 0) cus = di.num_cus;
    NormParams p{x, residual, weight, h, q, sf, rstd, m, k, eps};
    const int grid = std::min(m, cus * 8);
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    const hipError_t e = format == DG_QUANT_E4M3_F32     ? launch_norm<DG_QUANT_E4M3_F32>(p, grid, hs)
                         : format == DG_QUANT_E4M3_UE8M0 ? launch_norm<DG_QUANT_E4M3_UE8M0>(p, grid, hs)
                                                         : launch_norm<DG_QUANT_MXFP4>(p, grid, hs);
    return e == hipSuccess ? DG_OK : DG_ERR_HIP;
  } catch (...) {
    return DG_ERR_HIP;
  }
}

size_t dg_add_rms_norm_backward_workspace_bytes(int m, int k) {
  if (m <= 0 || k <= 0 || k % 128 != 0 || k > NORM_MAX_K) return 0;
  return (size_t)norm_parts(m) * k * sizeof(float);
}

int dg_add_rms_norm_backward(const uint16_t* dy, const uint16_t* dh, const uint16_t* h, const uint16_t* weight,
                             const float* rstd, uint16_t* dx, float* dweight, int m, int k, void* workspace,
                             size_t workspace_bytes, void* stream) {
  try {
    if (!dy || !h || !weight || !rstd || !dx || !dweight || !workspace) return DG_ERR_INVALID_ARG;
    if (m <= 0 || k <= 0) return DG_ERR_INVALID_ARG;
    if (misaligned(dy, 16) || misaligned(dh, 16) || misaligned(h, 16) || misaligned(weight, 16) ||
        misaligned(dx, 16) || misaligned(dweight, 16) || misaligned(rstd, 4) || misaligned(workspace, 16))
      return DG_ERR_INVALID_ARG;
    if (k % 128 != 0 || k > NORM_MAX_K) return DG_ERR_UNSUPPORTED;
    if (workspace_bytes < dg_add_rms_norm_backward_workspace_bytes(m, k)) return DG_ERR_INVALID_ARG;
    DeviceInfo di = current_device_info();
    if (!di.ok) return DG_ERR_NO_DEVICE;
    const int parts = norm_parts(m);
    NormBackParams p{dy, dh, h, weight, rstd, dx, static_cast<float*>(workspace), m, k};
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    hipError_t e = launch_norm_backward(p, parts, hs);
    if (e != hipSuccess) return DG_ERR_HIP;
    hipLaunchKernelGGL(norm_dweight_kernel, dim3((k + 255) / 256), dim3(256), 0, hs, p.part, dweight, parts, k);
    return hipGetLastError() == hipSuccess ? DG_OK : DG_ERR_HIP;
  } catch (...) {
    return DG_ERR_HIP;
  }
}

}  // extern "C"
