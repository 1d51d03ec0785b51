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

// Eight consecutive values of a row as they are in memory.
template <typename T>
struct Vec8;
template <>
struct Vec8<uint16_t> {
  v4i p;
  __device__ __forceinline__ void zero() { p = v4i{0, 0, 0, 0}; }
  __device__ __forceinline__ void load(const uint16_t* x) { p = *reinterpret_cast<const v4i*>(x); }
  __device__ __forceinline__ void to_lds(uint16_t* l) const { *reinterpret_cast<v4i*>(l) = p; }
  // bit pattern of the largest magnitude, as fp32
  __device__ __forceinline__ uint32_t amax() const {
    const us2 a = us2max(us2max(us2abs(p.x), us2abs(p.y)), us2max(us2abs(p.z), us2abs(p.w)));
    return umax(a.x, a.y) << 16;
  }
  __device__ __forceinline__ uint32_t codes(float scale) const { return e2m1x8(p, scale); }
};
template <>
struct Vec8<float> {
  v4f a, b;
  __device__ __forceinline__ void zero() { a = b = v4f{0.f, 0.f, 0.f, 0.f}; }
  __device__ __forceinline__ void load(const float* x) {
    a = *reinterpret_cast<const v4f*>(x);
    b = *reinterpret_cast<const v4f*>(x + 4);
  }
  __device__ __forceinline__ void to_lds(float* l) const {
    *reinterpret_cast<v4f*>(l) = a;
    *reinterpret_cast<v4f*>(l + 4) = b;
  }
  __device__ __forceinline__ uint32_t amax() const {
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) m = umax(m, umax(abs_bits(a[j]), abs_bits(b[j])));
    return m;
  }
  __device__ __forceinline__ uint32_t codes(float scale) const {
    const float v[8] = {a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]};
    return e2m1x8(v, scale);
  }
};

// The row direction of one vector: its 4-lane block's codes, and the scale word of its
// 16-lane K block (all lanes of the 16 take part).
struct RowCodes {
  uint32_t w, word;
  float scale;
};
template <typename T>
__device__ __forceinline__ RowCodes quantize_row8(const Vec8<T>& v) {
  const uint32_t byte = ue8m0_byte<false>(group_max<4>(v.amax()));
  RowCodes r;
  r.scale = ue8m0_value(byte);
  r.w = byte == 255u ? 0u : v.codes(r.scale);
  r.word = scale_word(byte);
  return r;
}

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
// columns, quantises the rows from registers on the way into LDS, and the columns
// from there: a thread holds two columns of one block of 32 rows.  (With the tiles in
// 2 x 2 squares on one XCD, so that its L2 could join the 64-byte runs of codes, 0-4 %
// slower; with 512 threads a tile, half a block each, the same at 4096 x 7168 and 2-6 %
// slower at 4096 x 4096 and 16384 x 7168: it is not the loads in flight.)
template <typename T>
__global__ void __launch_bounds__(256) quantize_tiles_kernel(QuantParams p) {
  __shared__ __attribute__((aligned(16))) T tile[128][128];
  __shared__ uint32_t words[128];
  __shared__ __attribute__((aligned(4))) uint8_t bytes[128][4];
  const T* x = static_cast<const T*>(p.x);
  const int tid = threadIdx.x;
  const uint32_t kb_n = (uint32_t)p.k >> 7, mb_n = ((uint32_t)p.m + 127) >> 7;
  const size_t mp = (size_t)mb_n * 128;
  const long long total = (long long)p.groups * mb_n * kb_n;
  for (long long t = blockIdx.x; t < total; t += gridDim.x) {
    const uint32_t gm = (uint32_t)(t / kb_n), kb = (uint32_t)(t - (long long)gm * kb_n);
    const uint32_t g = gm / mb_n, mb = gm - g * mb_n;
    const int rr = tid >> 4, c = (tid & 15) * 8;
    const T* src = x + ((size_t)g * p.m + mb * 128u) * p.k + kb * 128u + c;
    const int rows = min(128, p.m - (int)(mb * 128u));
    Vec8<T> v[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int r = s * 16 + rr;
      if (r < rows) v[s].load(src + (size_t)r * p.k);
      else v[s].zero();
    }
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int r = s * 16 + rr;
      v[s].to_lds(&tile[r][c]);
      if (p.q || p.values) {   // (uniform)
        const RowCodes o = quantize_row8(v[s]);
        if (r < rows) {
          const size_t at = (((size_t)g * p.m + mb * 128u + r) * p.k + kb * 128u + c) >> 3;
          if (p.q) reinterpret_cast<uint32_t*>(p.q)[at] = o.w;
          if (p.values) reinterpret_cast<v4i*>(p.values)[at] = e2m1x8_to_bf16(o.w, o.scale);
        }
        if ((tid & 15) == 0) words[r] = o.word;
      }
    }
    __syncthreads();
    if (p.sf && tid < rows) p.sf[((size_t)g * kb_n + kb) * p.m + mb * 128u + tid] = (int32_t)words[tid];
    const int c2 = (tid & 63) * 2, b = tid >> 6;
    v4i w[2];
    uint32_t byte[2];
    if constexpr (sizeof(T) == 2) {
      uint32_t e[32];   // rows b*32 .. of columns c2 (low half) and c2 + 1
      us2 am = us2{0, 0};
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        e[r] = *reinterpret_cast<const uint32_t*>(&tile[b * 32 + r][c2]);
        am = us2max(am, us2abs((int)e[r]));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        byte[h] = ue8m0_byte<false>((uint32_t)(h ? am.y : am.x) << 16);
        const float scale = ue8m0_value(byte[h]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          v4i pr;   // eight rows of the column
#pragma unroll
          for (int j = 0; j < 4; ++j)
            pr[j] = (int)__builtin_amdgcn_perm(e[8 * q + 2 * j + 1], e[8 * q + 2 * j], h ? 0x07060302u : 0x05040100u);
          w[h][q] = byte[h] == 255u ? 0 : (int)e2m1x8(pr, scale);
        }
      }
    } else {
      float e[2][32];
      uint32_t am[2] = {0, 0};
#pragma unroll
      for (int r = 0; r < 32; ++r) {
        const float2 f = *reinterpret_cast<const float2*>(&tile[b * 32 + r][c2]);
        e[0][r] = f.x;
        e[1][r] = f.y;
        am[0] = umax(am[0], abs_bits(f.x));
        am[1] = umax(am[1], abs_bits(f.y));
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        byte[h] = ue8m0_byte<false>(am[h]);
        const float scale = ue8m0_value(byte[h]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          float o[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) o[j] = e[h][8 * q + j];
          w[h][q] = byte[h] == 255u ? 0 : (int)e2m1x8(o, scale);
        }
      }
    }
    // the codes leave through LDS (the tile is read): four lanes write the 64 bytes of a
    // column, where each lane writing its own would send 16-byte pieces of 64 lines
    __syncthreads();
    uint8_t* stage = reinterpret_cast<uint8_t*>(tile);   // [128 columns][64 bytes, + 16 against bank conflicts]
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      *reinterpret_cast<v4i*>(stage + (c2 + h) * 80 + b * 16) = w[h];
      bytes[c2 + h][b] = (uint8_t)byte[h];
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int col = i * 64 + (tid >> 2);
      *reinterpret_cast<v4i*>(p.qt + ((size_t)g * p.k + kb * 128u + col) * (mp / 2) + (size_t)mb * 64 + (tid & 3) * 16) =
          *reinterpret_cast<const v4i*>(stage + col * 80 + (tid & 3) * 16);
    }
    if (tid < 128) p.sft[((size_t)g * mb_n + mb) * p.k + kb * 128u + tid] = *reinterpret_cast<const int32_t*>(bytes[tid]);
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
