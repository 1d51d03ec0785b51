// MXFP4 products grouped by expert with ragged sizes (gfx950): the rows of the groups lie one
// behind another without padding, ms[g] of them on the device.
//   along M   d[r] = A[r] . B_g^T for the rows r of group g: a layer's output, and with the
//             transposed weights the gradient of its input
//   along K   d[g] = A_g . B_g^T over the K blocks of group g: the gradient of each weight, from
//             operands that the quantiser below makes, blocks along the rows of each group
//
// The tile kernel of mxfp4_tile.hpp walks the groups' tiles as one list: every workgroup adds up
// the tiles of the groups before each (two scans by one wave, into LDS) and finds a tile's group
// by comparing its index with 64 ends at a time.  A tile's rows past its group's end belong to
// the next one: they are read and multiplied, and not stored.  The copies run on from tile to
// tile over the groups' borders.  Few rows a group: the streaming kernel, one workgroup per 16
// columns of each group, which reads the weights of the groups that have rows once.
#include <algorithm>

#include "../../include/dg.h"
#include "mxfp4_tile.hpp"
#include "quant_tile.hpp"

namespace dg {

using RaggedParams = Mxfp4GroupedParams<MX_RAGGED>;
using KGroupParams = Mxfp4GroupedParams<MX_KGROUP>;

// (a launch has fewer than 2^32 threads: 256 and 512 a workgroup)
constexpr long long kMaxSkinnyGrid = 1LL << 24, kMaxKgGrid = 1LL << 22;

static bool tile_serves(const Mxfp4TileInfo& t, int groups, long long units) {
  return t.lds + group_table_bytes(groups) <= kLdsBytes && (t.kg == 1 || units <= kMaxKgGrid);
}

struct GroupedPlan {
  int skinny, tile, grid;
};

// Tiles of the whole call as the host can guess them: groups of equal size, and half a tile
// more for each where a group has several.
static long long ragged_units(int m, int groups, int bm, int tiles_n, long long* most) {
  const int with_rows = std::min(m, groups);
  const double rows = (double)m / with_rows;
  *most = ((long long)m / bm + with_rows) * tiles_n;
  const double tiles = rows <= bm ? 1.0 : rows / bm + 0.5;
  return std::min(*most, (long long)(with_rows * tiles * tiles_n + 0.5));
}

static GroupedPlan plan_ragged(int m, int n, int k, int groups, int cus) {
  const int force = mxfp4_forced();
  GroupedPlan best{-1, 0, 0};
  if (force >= kMxSkinnyIdBase && (long long)(n / 16) * groups < kMaxSkinnyGrid) {
    best.skinny = std::min(force - kMxSkinnyIdBase, 1);
    return best;
  }
  const int rows = (m + groups - 1) / groups;
  if (force < 0 && rows <= 16 && (long long)(n / 16) * groups < kMaxSkinnyGrid) {
    best.skinny = rows <= 8 ? 0 : 1;
    return best;
  }
  double best_t = 1e30;
  for (int id = 0; id < kMxTileCount; ++id) {
    const Mxfp4TileInfo t = mxfp4_tile_info(id);
    long long most;
    const long long units = ragged_units(m, groups, t.bm, (n + t.bn - 1) / t.bn, &most);
    if (!tile_serves(t, groups, most)) continue;
    double us = mxfp4_tile_time(id, units, k / 128, cus);
    if (id == force) us = 0.0;
    if (us < best_t - 1e-9) {
      best_t = us;
      best.tile = id;
      // (a tile with K groups takes one unit per workgroup)
      best.grid = (int)(t.kg > 1 ? most : std::min<long long>(most, cus));
    }
  }
  return best;
}

// Tiles of every group alike, of which those without K blocks have none.
static GroupedPlan plan_kgroup(int m, int n, int kb, int groups, int cus) {
  const int force = mxfp4_forced();
  const int kb_each = std::max(1, kb / groups);
  GroupedPlan best{-1, 0, 0};
  double best_t = 1e30;
  for (int id = 0; id < kMxTileCount; ++id) {
    const Mxfp4TileInfo t = mxfp4_tile_info(id);
    const long long units = (long long)((m + t.bm - 1) / t.bm) * ((n + t.bn - 1) / t.bn) * groups;
    if (!tile_serves(t, groups, units)) continue;
    double us = mxfp4_tile_time(id, units, kb_each, cus);
    if (id == force) us = 0.0;
    if (us < best_t - 1e-9) {
      best_t = us;
      best.tile = id;
      best.grid = (int)(t.kg > 1 ? units : std::min<long long>(units, cus));
    }
  }
  return best;
}

template <typename P>
static P grouped_params(const uint8_t* a, const int32_t* a_sf, const uint8_t* b, const int32_t* b_sf, uint16_t* d, int m, int n,
                        int k, const Mxfp4TileInfo& t, const int32_t* ms, int groups) {
  return P{{a, a_sf, b, b_sf, nullptr, d, nullptr, m, n, k, (m + t.bm - 1) / t.bm, (n + t.bn - 1) / t.bn, 8, 1, k / 128, 0, 0}, ms, groups};
}

struct RaggedQuantParams {
  const void* x;
  const int32_t* ms;
  uint8_t* q;
  int32_t* sf;
  uint8_t* qt;
  int32_t* sft;
  int m, k, groups, blocks;
};

// One workgroup takes 128 rows of a group x 128 columns (quant_tile.hpp).  LDS: the tile, and
// the groups' first blocks and first rows.
template <typename T>
__global__ void __launch_bounds__(256) quantize_ragged_kernel(RaggedQuantParams p) {
  __shared__ QuantTile<T> lds;
  extern __shared__ int table[];
  int* const block_end = table;                  // [groups]
  int* const row_start = table + p.groups;       // [groups + 1]
  const T* x = static_cast<const T*>(p.x);
  const int tid = threadIdx.x, lane = tid & 63;
  // (blocks are the tiles of 128 rows and one column)
  if (tid < 64) build_groups<MX_RAGGED>(p.ms, p.groups, p.m, 128, 0, 1, block_end, row_start, lane);
  __syncthreads();
  const int blocks = block_end[p.groups - 1];
  const uint32_t kb_n = (uint32_t)p.k >> 7;
  const long long total = (long long)blocks * kb_n;
  const int rr = tid >> 4, c = (tid & 15) * 8;
  for (long long t = blockIdx.x; t < total; t += gridDim.x) {
    const uint32_t mb = (uint32_t)(t / kb_n), kb = (uint32_t)(t - (long long)mb * kb_n);
    int g = 0;
    for (int i = 0; i < p.groups; i += 64) g += __popcll(__ballot(i + lane < p.groups && block_end[i + lane] <= (int)mb));
    const int r0 = row_start[g] + ((int)mb - (g ? block_end[g - 1] : 0)) * 128;
    const int rows = min(128, row_start[g + 1] - r0);
    const size_t first = (size_t)r0 * p.k + kb * 128u;
    Vec8<T> v[8];
#pragma unroll
    for (int s = 0; s < 8; ++s) {
      const int r = s * 16 + rr;
      if (r < rows) v[s].load(x + first + c + (size_t)r * p.k);
      else v[s].zero();
    }
    quantize_tile(lds, v, rows,
                  QuantOut{p.q ? reinterpret_cast<uint32_t*>(p.q) + (first >> 3) : nullptr, nullptr,
                           p.sf ? p.sf + (size_t)kb * p.m + r0 : nullptr,
                           p.qt + (size_t)kb * 128u * ((size_t)p.blocks * 64) + (size_t)mb * 64, p.sft + (size_t)mb * p.k + kb * 128u,
                           (size_t)p.k >> 3, (size_t)p.blocks * 64});
  }
}

static bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

}  // namespace dg

using namespace dg;

extern "C" {

int dg_mxfp4_ragged_blocks(int m, int num_groups) {
  if (m <= 0 || num_groups <= 0 || num_groups > kMaxGroups) return 0;
  return (int)(((long long)m + 127LL * num_groups) / 128);
}

int dg_quantize_mxfp4_ragged(const void* x, int x_type, const int32_t* ms, uint8_t* q, int32_t* sf, uint8_t* qt, int32_t* sft,
                             int m, int k, int num_groups, void* stream) {
  try {
    if (!x || !ms || !qt || !sft || !q != !sf) return DG_ERR_INVALID_ARG;
    if (x_type != DG_BF16 && x_type != DG_F32) return DG_ERR_INVALID_ARG;
    if (m <= 0 || k <= 0 || num_groups <= 0) return DG_ERR_INVALID_ARG;
    if (misaligned(x, 16) || misaligned(q, 16) || misaligned(qt, 16) || misaligned(sf, 4) || misaligned(sft, 4) ||
        misaligned(ms, 4))
      return DG_ERR_INVALID_ARG;
    if (k % 128 != 0 || num_groups > kMaxGroups || m > 0x7fffffff - 127) return DG_ERR_UNSUPPORTED;
    DeviceInfo di = current_device_info();
    if (!di.ok) return DG_ERR_NO_DEVICE;
    const RaggedQuantParams p{x, ms, q, sf, qt, sft, m, k, num_groups, dg_mxfp4_ragged_blocks(m, num_groups)};
    const int grid = (int)std::min<long long>((long long)p.blocks * (k / 128), (long long)dg_get_num_cus() * 8);
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    if (x_type == DG_BF16)
      hipLaunchKernelGGL(quantize_ragged_kernel<uint16_t>, dim3(grid), dim3(256), group_table_bytes(num_groups), hs, p);
    else
      hipLaunchKernelGGL(quantize_ragged_kernel<float>, dim3(grid), dim3(256), group_table_bytes(num_groups), hs, p);
    return hipGetLastError() == hipSuccess ? DG_OK : DG_ERR_HIP;
  } catch (...) {
    return DG_ERR_HIP;
  }
}

int dg_m_grouped_mxfp4_gemm_nt_ragged(const uint8_t* a, const int32_t* a_sf, const uint8_t* b, const int32_t* b_sf,
                                      const int32_t* ms, uint16_t* d, int m, int n, int k, int num_groups, void* stream) {
  try {
    if (!a || !a_sf || !b || !b_sf || !ms || !d) return DG_ERR_INVALID_ARG;
    if (m <= 0 || n <= 0 || k <= 0 || num_groups <= 0) return DG_ERR_INVALID_ARG;
    if (misaligned(a, 16) || misaligned(b, 16) || misaligned(d, 16) || misaligned(a_sf, 4) || misaligned(b_sf, 4) ||
        misaligned(ms, 4))
      return DG_ERR_INVALID_ARG;
    if (!mxfp4_sizes_fit(m, n, k) || num_groups > kMaxGroups) return DG_ERR_UNSUPPORTED;
    DeviceInfo di = current_device_info();
    if (!di.ok) return DG_ERR_NO_DEVICE;
    const GroupedPlan pl = plan_ragged(m, n, k, num_groups, dg_get_num_cus());
    const RaggedParams p = grouped_params<RaggedParams>(a, a_sf, b, b_sf, d, m, n, k, mxfp4_tile_info(pl.tile), ms, num_groups);
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    const hipError_t e = pl.skinny >= 0 ? launch_mxfp4_skinny(p, pl.skinny, hs, num_groups)
                                        : launch_mxfp4_tile(p, pl.tile, pl.grid, hs, group_table_bytes(num_groups));
    return e == hipSuccess ? DG_OK : DG_ERR_HIP;
  } catch (...) {
    return DG_ERR_HIP;
  }
}

int dg_k_grouped_mxfp4_gemm_nt_ragged(const uint8_t* a, const int32_t* a_sf, const uint8_t* b, const int32_t* b_sf,
                                      const int32_t* ms, uint16_t* d, int m, int n, int k, int num_groups, void* stream) {
  try {
    if (!a || !a_sf || !b || !b_sf || !ms || !d) return DG_ERR_INVALID_ARG;
    if (m <= 0 || n <= 0 || k <= 0 || num_groups <= 0) return DG_ERR_INVALID_ARG;
    if (misaligned(a, 16) || misaligned(b, 16) || misaligned(d, 16) || misaligned(a_sf, 4) || misaligned(b_sf, 4) ||
        misaligned(ms, 4))
      return DG_ERR_INVALID_ARG;
    if (!mxfp4_sizes_fit(m, n, k) || num_groups > kMaxGroups) return DG_ERR_UNSUPPORTED;
    DeviceInfo di = current_device_info();
    if (!di.ok) return DG_ERR_NO_DEVICE;
    const GroupedPlan pl = plan_kgroup(m, n, k / 128, num_groups, dg_get_num_cus());
    const KGroupParams p = grouped_params<KGroupParams>(a, a_sf, b, b_sf, d, m, n, k, mxfp4_tile_info(pl.tile), ms, num_groups);
    const hipError_t e = launch_mxfp4_tile(p, pl.tile, pl.grid, reinterpret_cast<hipStream_t>(stream), group_table_bytes(num_groups));
    return e == hipSuccess ? DG_OK : DG_ERR_HIP;
  } catch (...) {
    return DG_ERR_HIP;
  }
}

}  // extern "C"
