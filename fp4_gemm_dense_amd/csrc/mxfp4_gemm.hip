// MXFP4 x MXFP4 dense GEMM for gfx950: D = C + A.B^T (NT), bf16 out.
//
// Mathematics: every 16x16x128 instruction (v_mfma_scale_f32_16x16x128_f8f6f4, both
// operands E2M1) multiplies one 128-wide K block and applies both UE8M0 scales per 32
// values itself, so the fp32 accumulators chain through it and nothing is promoted on
// the vector ALUs.  A lane (row = lane % 16, g = lane / 16) holds K [32g, 32g + 32) of
// its row: 16 bytes, and byte g of the row's scale word.  Blocks are computed
// transposed (B's rows as the instruction's first operand), so a lane's four results
// are four consecutive columns of one row of D.
#include <algorithm>

#include "../../include/dg.h"
#include "dg_device.hpp"
#include "dg_internal.hpp"

namespace dg {

struct Mxfp4Params {
  const uint8_t* a;
  const int32_t* a_sf;
  const uint8_t* b;
  const int32_t* b_sf;
  const uint16_t* c;
  uint16_t* d;
  int m, n, k;
};

__device__ __forceinline__ v4f mfma_mxfp4(const v4i& a, uint32_t sa, const v4i& b, uint32_t sb, const v4f& c) {
  const v8i a8 = {a.x, a.y, a.z, a.w, 0, 0, 0, 0}, b8 = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, FMT_E2M1, FMT_E2M1, 0, (int)sa, 0, (int)sb);
}

// One wave per workgroup computes 64 x 64 of D with fragments read from memory.
// Rows past the end of A or B are read from the last row; their results are not stored.
__global__ void __launch_bounds__(64) mxfp4_gemm_kernel(Mxfp4Params p) {
  constexpr int T = 4;
  const int lane = threadIdx.x, lrow = lane & 15, lgrp = lane >> 4;
  const int m0 = blockIdx.y * 64, n0 = blockIdx.x * 64;
  const int kb_n = p.k >> 7;
  const uint8_t* ap[T];
  const uint8_t* bp[T];
  int ar[T], br[T];
#pragma unroll
  for (int i = 0; i < T; ++i) {
    ar[i] = min(m0 + i * 16 + lrow, p.m - 1);
    br[i] = min(n0 + i * 16 + lrow, p.n - 1);
    ap[i] = p.a + (size_t)ar[i] * (p.k / 2) + lgrp * 16;
    bp[i] = p.b + (size_t)br[i] * (p.k / 2) + lgrp * 16;
  }
  v4f acc[T][T];
#pragma unroll
  for (int i = 0; i < T; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j) acc[i][j] = v4f{0.f, 0.f, 0.f, 0.f};
  for (int kb = 0; kb < kb_n; ++kb) {
    v4i af[T], bf[T];
    uint32_t sa[T], sb[T];
#pragma unroll
    for (int i = 0; i < T; ++i) {
      af[i] = *reinterpret_cast<const v4i*>(ap[i] + (size_t)kb * 64);
      bf[i] = *reinterpret_cast<const v4i*>(bp[i] + (size_t)kb * 64);
      sa[i] = (uint32_t)p.a_sf[(size_t)kb * p.m + ar[i]] >> (8 * lgrp) & 255u;
      sb[i] = (uint32_t)p.b_sf[(size_t)kb * p.n + br[i]] >> (8 * lgrp) & 255u;
    }
#pragma unroll
    for (int i = 0; i < T; ++i)
#pragma unroll
      for (int j = 0; j < T; ++j) acc[i][j] = mfma_mxfp4(bf[j], sb[j], af[i], sa[i], acc[i][j]);
  }
#pragma unroll
  for (int i = 0; i < T; ++i) {
    const int row = m0 + i * 16 + lrow;
#pragma unroll
    for (int j = 0; j < T; ++j) {
      const int col = n0 + j * 16 + 4 * lgrp;
      if (row >= p.m || col >= p.n) continue;
      const size_t at = (size_t)row * p.n + col;
      v4f v = acc[i][j];
      if (p.c) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] += bf16_to_f32(p.c[at + e]);
      }
      *reinterpret_cast<uint2*>(p.d + at) = uint2{pack_bf16x2_rne(v[0], v[1]), pack_bf16x2_rne(v[2], v[3])};
    }
  }
}

}  // namespace dg

using namespace dg;

static bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

extern "C" {

size_t dg_mxfp4_gemm_workspace_bytes(int m, int n, int k, int num_cus) {
  (void)m; (void)n; (void)k; (void)num_cus;
  return 0;
}

int dg_mxfp4_gemm_nt(const uint8_t* a, const int32_t* a_sf, const uint8_t* b, const int32_t* b_sf,
                     const uint16_t* c, uint16_t* d, int m, int n, int k, void* workspace, size_t workspace_bytes,
                     void* stream) {
  try {
    (void)workspace; (void)workspace_bytes;
    if (!a || !a_sf || !b || !b_sf || !d) return DG_ERR_INVALID_ARG;
    if (m <= 0 || n <= 0 || k <= 0) return DG_ERR_INVALID_ARG;
    if (misaligned(a, 16) || misaligned(b, 16) || misaligned(c, 16) || misaligned(d, 16) || misaligned(a_sf, 4) ||
        misaligned(b_sf, 4))
      return DG_ERR_INVALID_ARG;
    const long long lim = 1LL << 31;
    if (k % 128 != 0 || n % 16 != 0 || (long long)m * (k / 2) > lim || (long long)n * (k / 2) > lim ||
        (long long)m * n * 2 > lim || (long long)m * (k / 32) > lim || (long long)n * (k / 32) > lim)
      return DG_ERR_UNSUPPORTED;
    if ((m + 63) / 64 > 65535) return DG_ERR_UNSUPPORTED;
    DeviceInfo di = current_device_info();
    if (!di.ok) return DG_ERR_NO_DEVICE;
    Mxfp4Params p{a, a_sf, b, b_sf, c, d, m, n, k};
    hipLaunchKernelGGL(mxfp4_gemm_kernel, dim3((n + 63) / 64, (m + 63) / 64), dim3(64), 0,
                       reinterpret_cast<hipStream_t>(stream), p);
    return hipGetLastError() == hipSuccess ? DG_OK : DG_ERR_HIP;
  } catch (...) {
    return DG_ERR_HIP;
  }
}

}  // extern "C"
