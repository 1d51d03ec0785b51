// MXFP4 linear layer for gfx950: d = residual + act(A.B^T + bias), or with a gated activation
// d = residual + act(gate) * up, gate and up the two halves of A.B^T + bias; optionally the
// pre-activation A.B^T + bias itself, for the backward pass.
//
// The products are the kernels of mxfp4_tile.hpp on the dense GEMM's plans; the epilogue works
// on the fp32 accumulators where they are (after the K groups' sums have met, or in the reduce
// of a plan split along K), so neither u nor act(u) goes to memory between the two.  act reads
// the unrounded u, whether or not z is stored: the same d either way.
//
// Bound: as the dense GEMM, and the epilogue behind a unit's last product, which nothing
// overlaps but the next unit's copies.  Measured (one MI355X; in brackets the dense GEMM, whose D
// is [m, n]): 4096 x 16384 x 7168 gated with SiLU 229 us (225), with z, 134 MB more, 241, and in
// passes one upon another, at the clock that power then leaves, 248-258 and 261-272 (230-257); 4096 x
// 7168 x 16384 with residual 247 (235); 4096 x 24576 x 1536 without 107 (98), SiLU 119-126, gated
// SiLU with z 128, GELU 150-160 (its polynomial for 128 values of a lane in a unit); 2001 x 4096 x
// 7168 GELU with residual and z 41 (35); 1 x 4096 x 7168 6.6 (6.1).
#include <algorithm>

#include "../../include/dg.h"
#include "mxfp4_tile.hpp"

namespace dg {

// The split tiles' partial sums in slice order, and the epilogue: a thread takes W outputs of one
// row (for one launch over the slices of all split tiles).
template <bool GATED, int W>
__global__ void __launch_bounds__(256) linear_reduce_kernel(Mxfp4LinearParams<GATED> p, int bm, int bn, int split_tiles) {
  const int per_row = bn / (GATED ? 2 * W : W);
  const long long per_tile = (long long)bm * per_row, total = per_tile * split_tiles;
  const size_t tile = (size_t)bm * bn;
  const int cols = GATED ? p.n >> 1 : p.n;
  const LinearOut<GATED, W> out(p);
  for (long long i = (long long)blockIdx.x * 256 + threadIdx.x; i < total; i += (long long)gridDim.x * 256) {
    const int st = (int)(i / per_tile), q = (int)(i - (long long)st * per_tile);
    const int r = q / per_row, at = (q - r * per_row) * W;   // the first output, of the tile's
    int tm, tn;
    raster_tile(p.full_tiles + st, p.tiles_m, p.tiles_n, p.group_m, &tm, &tn);
    // the tile's column of the first result, and of the other half's
    const int c = !GATED ? at : W == 8 ? (at >> 5) * 64 + (at & 31) : at * 2;
    const int row = tm * bm + r, col = GATED ? gated_output<W>(tn * bn + c) : tn * bn + c;
    const bool ok = row < p.m && col < cols;
    const auto cv = out.load_c(out.place(row, col, ok));
    auto sum = [&](int c, int bias_col, float (&v)[W]) {
      const float* w = p.ws + (size_t)st * p.splits * tile + (size_t)r * bn + c;
#pragma unroll
      for (int e = 0; e < W; e += 4) {
        v4f t = *reinterpret_cast<const v4f*>(w + e);
        for (int s = 1; s < p.splits; ++s) t += *reinterpret_cast<const v4f*>(w + s * tile + e);
#pragma unroll
        for (int j = 0; j < 4; ++j) v[e + j] = t[j];
      }
      if (p.bias && ok) add_bf16(v, reinterpret_cast<const int*>(p.bias + bias_col));
    };
    float u[W], up[W];
    sum(c, col, u);
    if constexpr (GATED) {
      sum(c + (W == 8 ? 32 : 4), cols + col, up);
    } else {
#pragma unroll
      for (int e = 0; e < W; ++e) up[e] = 0.f;
    }
    out(row, col, ok, u, up, cv);
  }
}

bool activation_of(int activation, Activation* a) {
  // 2 sqrt(2 / pi) and 0.044715 times it
  constexpr float c1 = 1.5957691216057308f, c3 = 0.07135481627260025f;
  switch (activation & ~DG_ACT_GATED) {
    case DG_ACT_NONE: *a = {ACT_KIND_CLAMP, -__builtin_inff(), 0.f, 0.f}; return true;
    case DG_ACT_RELU: *a = {ACT_KIND_CLAMP, 0.f, 0.f, 0.f}; return true;
    case DG_ACT_SILU: *a = {ACT_KIND_SIGMOID, 0.f, 1.f, 0.f}; return true;
    case DG_ACT_GELU: *a = {ACT_KIND_ERF, 0.f, 0.f, 0.f}; return true;
    case DG_ACT_GELU_TANH: *a = {ACT_KIND_SIGMOID, 0.f, c1, c3}; return true;
  }
  return false;
}

template <bool GATED>
static hipError_t launch_linear(const Mxfp4LinearParams<GATED>& p, const Mxfp4Plan& pl, int cus, hipStream_t hs) {
  if (pl.skinny >= 0) return launch_mxfp4_skinny(p, pl.skinny, hs);
  hipError_t e = launch_mxfp4_tile(p, pl.tile, pl.grid, hs);
  if (e != hipSuccess || !pl.ws_bytes) return e;
  const Mxfp4TileInfo t = mxfp4_tile_info(pl.tile);
  const int split_tiles = pl.tiles_m * pl.tiles_n - pl.full_tiles;
  const int grid = (int)std::min<long long>(((long long)split_tiles * t.bm * (t.bn / 8) + 255) / 256, (long long)cus * 8);
  if constexpr (GATED) {
    if (t.narrow) {
      hipLaunchKernelGGL((linear_reduce_kernel<GATED, 4>), dim3(grid), dim3(256), 0, hs, p, t.bm, t.bn, split_tiles);
      return hipGetLastError();
    }
  }
  hipLaunchKernelGGL((linear_reduce_kernel<GATED, 8>), dim3(grid), dim3(256), 0, hs, p, t.bm, t.bn, split_tiles);
  return hipGetLastError();
}

static bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

}  // namespace dg

using namespace dg;

extern "C" int dg_mxfp4_linear(const uint8_t* a, const int32_t* a_sf, const uint8_t* b, const int32_t* b_sf,
                               const uint16_t* bias, int activation, const uint16_t* residual, uint16_t* z, uint16_t* d,
                               int m, int n, int k, void* workspace, size_t workspace_bytes, void* stream) {
  try {
    Activation act;
    if (!a || !a_sf || !b || !b_sf || !d || !activation_of(activation, &act)) return DG_ERR_INVALID_ARG;
    if (m <= 0 || n <= 0 || k <= 0) return DG_ERR_INVALID_ARG;
    if (misaligned(a, 16) || misaligned(b, 16) || misaligned(bias, 16) || misaligned(residual, 16) || misaligned(z, 16) ||
        misaligned(d, 16) || misaligned(a_sf, 4) || misaligned(b_sf, 4))
      return DG_ERR_INVALID_ARG;
    const bool gated = activation & DG_ACT_GATED;
    if (!mxfp4_sizes_fit(m, n, k) || (gated && n % 32 != 0)) return DG_ERR_UNSUPPORTED;
    DeviceInfo di = current_device_info();
    if (!di.ok) return DG_ERR_NO_DEVICE;
    const int cus = dg_get_num_cus();
    const Mxfp4Plan pl = plan_mxfp4(m, n, k, cus);
    if (pl.ws_bytes && (!workspace || workspace_bytes < pl.ws_bytes || misaligned(workspace, 16))) return DG_ERR_INVALID_ARG;
    log_mxfp4_plan("mxfp4_linear", m, n, k, pl);
    const Mxfp4Params p{a, a_sf, b, b_sf, residual, d, static_cast<float*>(workspace), m, n, k,
                        pl.tiles_m, pl.tiles_n, 8, pl.splits, pl.kb_per_split, pl.full_tiles, pl.units};
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    const hipError_t e = gated ? launch_linear(Mxfp4LinearParams<true>{p, bias, z, act}, pl, cus, hs)
                               : launch_linear(Mxfp4LinearParams<false>{p, bias, z, act}, pl, cus, hs);
    return e == hipSuccess ? DG_OK : DG_ERR_HIP;
  } catch (...) {
    return DG_ERR_HIP;
  }
}
