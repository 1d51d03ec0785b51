// Quantisation to MXFP4 for gfx950: E2M1 codes with a power-of-two scale per block
// of 32 values, along the rows, along the columns (of the transposed operand), or
// both from one read.
//
// Mathematics: e = the least integer with 6 * 2^e >= max |x| of the block, from the
// maximum's bit pattern (no logarithm); code = E2M1(x * 2^-e), nearest, ties to the
// even code, by gfx950's scaled conversion.  Nothing saturates.
//
// Bound: HBM.  A bf16 element costs 2 bytes of reading and 17/32 of writing per
// direction.
#include <algorithm>

#include "../../include/dg.h"
#include "dg_internal.hpp"
#include "dg_quant.hpp"

namespace dg {

struct QuantParams {
  const void* x;
  uint8_t* q;
  int32_t* sf;
  uint8_t* qt;
  int32_t* sft;
  uint16_t* values;
  int groups, m, k;
};

// Eight consecutive values of x from element i, and the largest magnitude's bits.
struct Vec8 {
  float v[8];
  uint32_t amax;
};
template <typename T>
__device__ __forceinline__ void load8(const T* x, size_t i, Vec8& o) {
  if constexpr (sizeof(T) == 2) {
    unpack_bf16x8(*reinterpret_cast<const v4i*>(x + i), o.v);
  } else {
    const v4f a = *reinterpret_cast<const v4f*>(x + i), b = *reinterpret_cast<const v4f*>(x + i + 4);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      o.v[j] = a[j];
      o.v[4 + j] = b[j];
    }
  }
  o.amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) o.amax = umax(o.amax, abs_bits(o.v[j]));
}

// Blocks along k: a lane holds 8 values, 4 lanes a block, 16 lanes a 128-wide K block.
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantParams p) {
  const T* x = static_cast<const T*>(p.x);
  const size_t total = (size_t)p.groups * p.m * (p.k / 8);   // a multiple of 16
  const uint32_t per_row = (uint32_t)p.k / 8;
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (size_t)gridDim.x * 256) {
    Vec8 t;
    load8(x, i * 8, t);
    const uint32_t byte = ue8m0_byte<false>(group_max<4>(t.amax));
    const float scale = ue8m0_value(byte);
    const uint32_t w = byte == 255u ? 0u : e2m1x8(t.v, scale);
    if (p.q) {
      reinterpret_cast<uint32_t*>(p.q)[i] = w;
      const uint32_t word = scale_word(byte);
      if ((threadIdx.x & 15) == 0) {
        const size_t row = i / per_row;
        const uint32_t kb = (uint32_t)(i - row * per_row) >> 4;
        const size_t g = row / p.m, r = row - g * p.m;
        p.sf[(g * (p.k / 128) + kb) * p.m + r] = (int32_t)word;
      }
    }
    if (p.values) reinterpret_cast<v4i*>(p.values)[i] = e2m1x8_to_bf16(w, scale);
  }
}

// Blocks along m (and along k, when asked): one workgroup takes 128 rows x 128
// columns, quantises the rows from registers on the way into LDS, and the columns
// from there: a thread holds two columns of one block of 32 rows.
template <typename T>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(QuantParams p) {
  __shared__ T tile[128][128];
  __shared__ uint32_t bytes[128];
  const T* x = static_cast<const T*>(p.x);
  const int tid = threadIdx.x;
  const int kb_n = p.k / 128, mb_n = (p.m + 127) / 128;
  const size_t mp = (size_t)mb_n * 128;
  const long long total = (long long)p.groups * mb_n * kb_n;
  for (long long t = blockIdx.x; t < total; t += gridDim.x) {
    const int kb = (int)(t % kb_n);
    const long long gm = t / kb_n;
    const int mb = (int)(gm % mb_n);
    const size_t g = (size_t)(gm / mb_n);
    if (tid < 128) bytes[tid] = 0;
    for (int s = 0; s < 8; ++s) {
      const int r = s * 16 + (tid >> 4), c = (tid & 15) * 8;
      const int row = mb * 128 + r;
      Vec8 v;
#pragma unroll
      for (int j = 0; j < 8; ++j) v.v[j] = 0.f;
      v.amax = 0;
      const size_t at = (g * p.m + row) * (size_t)p.k + (size_t)kb * 128 + c;
      const bool in = row < p.m;
      if (in) load8(x, at, v);
      T* dst = &tile[r][c];
      if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<v4i*>(dst) = in ? *reinterpret_cast<const v4i*>(x + at) : v4i{0, 0, 0, 0};
      } else {
        *reinterpret_cast<v4f*>(dst) = v4f{v.v[0], v.v[1], v.v[2], v.v[3]};
        *reinterpret_cast<v4f*>(dst + 4) = v4f{v.v[4], v.v[5], v.v[6], v.v[7]};
      }
      const uint32_t byte = ue8m0_byte<false>(group_max<4>(v.amax));
      const float scale = ue8m0_value(byte);
      const uint32_t w = byte == 255u ? 0u : e2m1x8(v.v, scale);
      const uint32_t word = scale_word(byte);
      if (in && p.q) {
        reinterpret_cast<uint32_t*>(p.q)[at / 8] = w;
        if ((tid & 15) == 0) p.sf[(g * kb_n + kb) * p.m + row] = (int32_t)word;
      }
      if (in && p.values) reinterpret_cast<v4i*>(p.values)[at / 8] = e2m1x8_to_bf16(w, scale);
    }
    __syncthreads();
    const int c = (tid & 63) * 2, b = tid >> 6;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      float v[32];
      uint32_t amax = 0;
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        if constexpr (sizeof(T) == 2) v[r] = bf16_to_f32((uint16_t)tile[b * 32 + r][c + h]);
        else v[r] = tile[b * 32 + r][c + h];
        amax = umax(amax, abs_bits(v[r]));
      }
      const uint32_t byte = ue8m0_byte<false>(amax);
      const float scale = ue8m0_value(byte);
      v4i w;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float e[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) e[j] = v[8 * q + j];
        w[q] = byte == 255u ? 0 : (int)e2m1x8(e, scale);
      }
      const size_t col = g * p.k + (size_t)kb * 128 + c + h;
      *reinterpret_cast<v4i*>(p.qt + col * (mp / 2) + (size_t)mb * 64 + b * 16) = w;
      atomicOr(&bytes[c + h], byte << (8 * b));
    }
    __syncthreads();
    if (tid < 128) p.sft[(g * mb_n + mb) * p.k + (size_t)kb * 128 + tid] = (int32_t)bytes[tid];
    __syncthreads();
  }
}

}  // namespace dg

using namespace dg;

static bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

extern "C" int dg_quantize_mxfp4(const void* x, int x_type, uint8_t* q, int32_t* sf, uint8_t* qt, int32_t* sft,
                                 uint16_t* values, int num_groups, int m, int k, void* stream) {
  try {
    if (!x || (!q && !qt && !values) || !q != !sf || !qt != !sft) return DG_ERR_INVALID_ARG;
    if (x_type != DG_BF16 && x_type != DG_F32) return DG_ERR_INVALID_ARG;
    if (num_groups <= 0 || m <= 0 || k <= 0) return DG_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(q, 16) || misaligned(qt, 16) || misaligned(values, 16) || misaligned(sf, 4) ||
        misaligned(sft, 4))
      return DG_ERR_INVALID_ARG;
    if (k % 128 != 0 || (long long)num_groups * m > 0x7fffffffLL || m > 0x7fffffff - 127) return DG_ERR_UNSUPPORTED;
    DeviceInfo di = current_device_info();
    if (!di.ok) return DG_ERR_NO_DEVICE;
    int cus = dg_get_num_cus();
    if (cus <= 0) cus = di.num_cus;
    QuantParams p{x, q, sf, qt, sft, values, num_groups, m, k};
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    if (qt) {
      const long long tiles = (long long)num_groups * ((m + 127) / 128) * (k / 128);
      const int grid = (int)std::min<long long>(tiles, (long long)cus * 8);
      if (x_type == DG_BF16)
        hipLaunchKernelGGL(quantize_tiles_kernel<uint16_t>, dim3(grid), dim3(256), 0, hs, p);
      else
        hipLaunchKernelGGL(quantize_tiles_kernel<float>, dim3(grid), dim3(256), 0, hs, p);
    } else {
      const long long blocks = ((long long)num_groups * m * (k / 8) + 255) / 256;
      const int grid = (int)std::min<long long>(blocks, (long long)cus * 8);
      if (x_type == DG_BF16)
        hipLaunchKernelGGL(quantize_rows_kernel<uint16_t>, dim3(grid), dim3(256), 0, hs, p);
      else
        hipLaunchKernelGGL(quantize_rows_kernel<float>, dim3(grid), dim3(256), 0, hs, p);
    }
    return hipGetLastError() == hipSuccess ? DG_OK : DG_ERR_HIP;
  } catch (...) {
    return DG_ERR_HIP;
  }
}
