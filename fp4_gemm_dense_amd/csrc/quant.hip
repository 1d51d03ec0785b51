// Quantisation to MXFP4 for gfx950: E2M1 codes with a power-of-two scale per block
// of 32 values, along the rows, along the columns (of the transposed operand), or
// both from one read.
//
// Mathematics: e = the least integer with 6 * 2^e >= max |x| of the block, from the
// maximum's bit pattern (no logarithm); code = E2M1(x * 2^-e), nearest, ties to the
// even code, by gfx950's scaled conversion.  Nothing saturates.
//
// Bound: HBM.  A bf16 element costs 2 bytes of reading and 17/32 of writing per
// direction.  Measured (one MI355X, inputs not in the caches; a 1 GiB copy runs at 5.1
// TB/s): 4096 x 7168 bf16 along the rows 16.0 us (4.7 TB/s), transposed 17.1 (4.3), both
// 22.5 (4.0); 16384 x 7168 both 82 (4.4); 2 x 4096 x 7168 fp32 rows and values 71 (5.4);
// 5 x 7168 with values 3.4, of which the launch is 2.7.
#include <algorithm>

#include "../../include/dg.h"
#include "dg_internal.hpp"
#include "dg_quant.hpp"
#include "quant_tile.hpp"

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

// Blocks along k.  A workgroup takes 16 rows x 512 columns: a wave reads 512 values of
// each of its four rows (all four loads in flight), 16 lanes a K block, and the 16
// rows' scale words leave through LDS as 64-byte runs (K-block-major).
constexpr int QR_ROWS = 16, QR_COLS = 512;
template <typename T>
__global__ void __launch_bounds__(256) quantize_rows_kernel(QuantParams p) {
  __shared__ uint32_t words[QR_COLS / 128][QR_ROWS];
  const T* x = static_cast<const T*>(p.x);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int kb_n = p.k >> 7;
  const uint32_t cb = ((uint32_t)p.k + QR_COLS - 1) / QR_COLS, rb = ((uint32_t)p.m + QR_ROWS - 1) / QR_ROWS;
  const long long total = (long long)cb * rb * p.groups;
  for (long long t = blockIdx.x; t < total; t += gridDim.x) {
    const uint32_t row_block = (uint32_t)(t / cb), c0 = (uint32_t)(t - (long long)row_block * cb) * QR_COLS;
    const uint32_t g = row_block / rb, r0 = (row_block - g * rb) * QR_ROWS;
    const uint32_t col = c0 + lane * 8;
    const bool in = col < (uint32_t)p.k;
    Vec8<T> v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = r0 + i * 4 + wave;
      if (in && r < (uint32_t)p.m) v[i].load(x + ((size_t)g * p.m + r) * p.k + col);
      else v[i].zero();
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t r = r0 + i * 4 + wave;
      const RowCodes o = quantize_row8(v[i]);
      if (in && r < (uint32_t)p.m) {
        const size_t at = (((size_t)g * p.m + r) * p.k + col) >> 3;
        if (p.q) reinterpret_cast<uint32_t*>(p.q)[at] = o.w;
        if (p.values) reinterpret_cast<v4i*>(p.values)[at] = e2m1x8_to_bf16(o.w, o.scale);
      }
      if ((lane & 15) == 0) words[lane >> 4][i * 4 + wave] = o.word;
    }
    if (p.sf) {   // (uniform)
      __syncthreads();
      if (tid < 64) {
        const uint32_t kb = (c0 >> 7) + (tid >> 4), r = r0 + (tid & 15);
        if (kb < (uint32_t)kb_n && r < (uint32_t)p.m)
          p.sf[((size_t)g * kb_n + kb) * p.m + r] = (int32_t)words[tid >> 4][tid & 15];
      }
      __syncthreads();
    }
  }
}

// Blocks along m (and along k, when asked): one workgroup takes 128 rows x 128
// columns (quant_tile.hpp).  (With the tiles in
// 2 x 2 squares on one XCD, so that its L2 could join the 64-byte runs of codes, 0-4 %
// slower; with 512 threads a tile, half a block each, the same at 4096 x 7168 and 2-6 %
// slower at 4096 x 4096 and 16384 x 7168: it is not the loads in flight.)
template <typename T>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(QuantParams p) {
  __shared__ QuantTile<T> lds;
  const T* x = static_cast<const T*>(p.x);
  const int tid = threadIdx.x;
  const uint32_t kb_n = (uint32_t)p.k >> 7, mb_n = ((uint32_t)p.m + 127) >> 7;
  const size_t mp = (size_t)mb_n * 128;
  const long long total = (long long)p.groups * mb_n * kb_n;
  for (long long t = blockIdx.x; t < total; t += gridDim.x) {
    const uint32_t gm = (uint32_t)(t / kb_n), kb = (uint32_t)(t - (long long)gm * kb_n);
    const uint32_t g = gm / mb_n, mb = gm - g * mb_n;
    const int rr = tid >> 4, c = (tid & 15) * 8;
    const size_t first = ((size_t)g * p.m + mb * 128u) * p.k + kb * 128u;
    const int rows = min(128, p.m - (int)(mb * 128u));
    Vec8<T> v[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int r = s * 16 + rr;
      if (r < rows) v[s].load(x + first + c + (size_t)r * p.k);
      else v[s].zero();
    }
    quantize_tile(lds, v, rows,
                  QuantOut{p.q ? reinterpret_cast<uint32_t*>(p.q) + (first >> 3) : nullptr,
                           p.values ? reinterpret_cast<v4i*>(p.values) + (first >> 3) : nullptr,
                           p.sf ? p.sf + ((size_t)g * kb_n + kb) * p.m + mb * 128u : nullptr,
                           p.qt + ((size_t)g * p.k + kb * 128u) * (mp / 2) + (size_t)mb * 64,
                           p.sft + ((size_t)g * mb_n + mb) * p.k + kb * 128u, (size_t)p.k >> 3, mp / 2});
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
    const int cus = dg_get_num_cus();
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
      const long long tiles = (long long)num_groups * ((m + QR_ROWS - 1) / QR_ROWS) * (((long long)k + QR_COLS - 1) / QR_COLS);
      const int grid = (int)std::min<long long>(tiles, (long long)cus * 64);
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
