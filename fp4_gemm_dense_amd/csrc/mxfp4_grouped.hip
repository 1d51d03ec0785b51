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
// tile over the groups' borders.
//
// Bound: with few rows the stream of the weights (64 rows over 32 experts of 4096 x 7168 80 us: 403 MB
// at 5.0 TB/s); with many the schedule, as the dense GEMM, and the groups' last tiles (8192 rows over 8
// 144-150 us, 3.2-3.3 PFLOP/s; 4000 rows over 8 of 4096 x 2048 34, 1.6 rounds of units); along K with few
// rows a group the end of a unit, 4.5 us that nothing overlaps beside two or three stages (4000 rows in 8
// groups of 4096 x 2048 46-51: 134 MB of D at half of a copy's rate).  The quantiser: HBM, and its second
// round of tiles (three inputs in turn: 4000 x 2048 bf16 10.2 us, fp32 14.6; 4000 x 4096 15.2 and 21.9,
// 1248 tiles at most on 1024 places; 16384 x 7168 85 and 133; the plain one 8.4, 11.0, 12.0, 17.6, 80, 130).
#include <algorithm>
#include <cstdio>
#include <cstdlib>

#include "../../include/dg.h"
#include "mxfp4_tile.hpp"
#include "quant_tile.hpp"

namespace dg {

using RaggedParams = Mxfp4GroupedParams<MX_RAGGED>;
using KGroupParams = Mxfp4GroupedParams<MX_KGROUP>;

struct GroupedPlan {
  int tile, grid;
  long long most;   // tiles that the call can have
};

// The tile with the least estimated time.  units(tile): how many of it the call has by the host's
// guess, and the most it can have; slow: how far the 256x256 tile runs behind its estimate.  A
// ring has to leave room for the table; tiles with K groups take one unit per workgroup.
template <typename F>
static GroupedPlan plan_grouped(int groups, int kb, int cus, double slow, F units) {
  const int force = mxfp4_forced();
  GroupedPlan best{2, 0, 0};
  double best_t = 1e30;
  for (int id = 0; id < kMxGroupedTileCount; ++id) {
    const Mxfp4TileInfo t = mxfp4_tile_info(id);
    long long most;
    const long long guess = units(t, &most);
    if (t.lds + group_table_bytes(groups) > kLdsBytes || (t.kg > 1 && most > cus)) continue;
    const double us = id == force ? 0.0 : mxfp4_tile_time(id, guess, kb, cus) * (t.bm == 256 ? slow : 1.0);
    if (us < best_t - 1e-9) {
      best_t = us;
      best = {id, (int)std::min<long long>(most, cus), most};
    }
  }
  return best;
}

// Along M: groups of equal size, and half a tile more for each.  (8192 x 4096 x 7168 in 8 groups
// 144 us on 192x256, 161 on 128x256, 176 on 256x256, 187 on 128x128: 3 rounds of units, 5, 3 and 9; 3901
// x 2048 x 4096 in 16 31 on 192x256, 38 on the best other.  The tile taken is on average 2 % behind the
// best of 80 shapes with 4 to 64 groups of like and unlike sizes, at worst 26 %; 64 x
// 4096 x 7168 in 32, the weights' stream, 80 on 128x256, 86 on 128x128, 80 on 64x128, and 111 by a
// streaming kernel of 16 columns a workgroup, as the dense GEMM has for few rows; 8 rows in 8
// groups 26 on 64x128 with two K groups, 34 streaming.)
static GroupedPlan plan_ragged(int m, int n, int k, int groups, int cus) {
  return plan_grouped(groups, k / 128, cus, 1.05, [=](const Mxfp4TileInfo& t, long long* most) {
    const long long tiles_n = (n + t.bn - 1) / t.bn;
    const int with_rows = std::min(m, groups);
    *most = ((long long)m / t.bm + with_rows) * tiles_n;
    const double tiles = std::max(1.0, (double)m / with_rows / t.bm + 0.5);
    return std::min(*most, (long long)(with_rows * tiles * tiles_n + 0.5));
  });
}

// Along K: every group that has rows has the same tiles.  (16384 rows in 8 groups, 4096 x 7168, 335
// us on 256x256, 362 on 128x256, 429 on 128x128; 4000 rows, 4096 x 2048, 46, 49 and 57; 1000 rows
// in 32, 4096 x 7168, which writes D alone, 455, 506 and 597.)
static GroupedPlan plan_kgroup(int m, int n, int kb, int groups, int cus) {
  return plan_grouped(groups, std::max(1, kb / groups), cus, 0.95, [=](const Mxfp4TileInfo& t, long long* most) {
    return *most = (long long)((m + t.bm - 1) / t.bm) * ((n + t.bn - 1) / t.bn) * groups;
  });
}

// (with DG_LOG=1)
static void log_grouped_plan(const char* call, int m, int n, int k, int groups, const GroupedPlan& pl) {
  const char* log = std::getenv("DG_LOG");
  if (!log || log[0] != '1') return;
  const Mxfp4TileInfo t = mxfp4_tile_info(pl.tile);
  std::fprintf(stderr, "[dg] %s m=%d n=%d k=%d groups=%d -> tile %dx%d, %d K group%s, at most %lld tiles, %d workgroups\n", call, m, n, k,
               groups, t.bm, t.bn, t.kg, t.kg > 1 ? "s" : "", pl.most, pl.grid);
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
    log_grouped_plan("m_grouped_mxfp4_gemm_nt_ragged", m, n, k, num_groups, pl);
    const RaggedParams p = grouped_params<RaggedParams>(a, a_sf, b, b_sf, d, m, n, k, mxfp4_tile_info(pl.tile), ms, num_groups);
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    const hipError_t e = launch_mxfp4_tile(p, pl.tile, pl.grid, hs, group_table_bytes(num_groups));
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
    log_grouped_plan("k_grouped_mxfp4_gemm_nt_ragged", m, n, k, num_groups, pl);
    const KGroupParams p = grouped_params<KGroupParams>(a, a_sf, b, b_sf, d, m, n, k, mxfp4_tile_info(pl.tile), ms, num_groups);
    const hipError_t e = launch_mxfp4_tile(p, pl.tile, pl.grid, reinterpret_cast<hipStream_t>(stream), group_table_bytes(num_groups));
    return e == hipSuccess ? DG_OK : DG_ERR_HIP;
  } catch (...) {
    return DG_ERR_HIP;
  }
}

}  // extern "C"
