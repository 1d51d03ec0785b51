// MXFP4 x MXFP4 dense GEMM for gfx950: D = C + A.B^T (NT), bf16 out.
//
// Mathematics: every 16x16x128 instruction (v_mfma_scale_f32_16x16x128_f8f6f4, both
// operands E2M1) multiplies one 128-wide K block and applies both UE8M0 scales per 32
// values itself, so the fp32 accumulators chain through it and nothing is promoted on
// the vector ALUs.  A lane (row = lane % 16, g = lane / 16) holds K [32g, 32g + 32) of
// its row: 16 bytes, and byte g of the row's scale word.  Blocks are computed
// transposed (B's rows as the instruction's first operand), so a lane's four results
// are four consecutive columns of one row of D.
//
// Tile kernel (persistent, eight waves, two per SIMD):
//   * a stage is 256 values of K, so a tile row is one 128-byte line; A, B and their
//     scale words come through a ring of R LDS slots by LDS-DMA loads;
//   * a wave multiplies K block kb while it reads the fragments of kb + 1: A's into a
//     second register set, B's into the registers of the column block that has just
//     had its last use;
//   * one barrier per stage, inside its second K block, after the first column blocks:
//     by then the wave's reads of the slot are back without a wait.  It frees the slot
//     for stage s + R and certifies stage s + 1;
//   * the stage copies run on into the next tile, so its first stage is there when
//     the tile ends; D goes from the registers to memory, 16 bytes a lane: the columns
//     of B's fragments are permuted so that a lane's two neighbouring column blocks
//     are eight adjacent columns;
//   * K may be split (few tiles, or a small last round): slices write fp32 partial
//     tiles to the workspace, which the split-K reduce adds in slice order.  Where one
//     tile per workgroup covers the problem, tiles of 64x64 to 128x128 instead run two
//     groups of four waves that take a tile's stages in turn, each with a ring of its own
//     (a stage's chain of barrier, reads and products is 0.5-0.6 us however small; 200 x
//     4096 x 7168 18.4 us on 64x128 with one group, 12.6 with two, 10.7 on 64x64).
//
// Measured (one MI355X, a kernel trace on quantised normal values, operands not in L2; such
// times differ by 5 % from card to card): 8192 x 8192 x 8192 247-260 us (4.2-4.5 PFLOP/s),
// 4096 x 7168 x 16384 235-265, 4096 x 4096 x 7168 58-62, all on 256x256; 1111 x 2112 x 7168
// 19.5-20.5 on 96x128; 200 x 4096 x 7168 11.5-12 on 64x64.  What bounds the large ones is
// the schedule first and power second: the matrix cores are busy in half of the cycles
// whatever the codes, at 1.8-2.0 GHz on normal values and at 2.3 GHz on zeros (4096 x 7168
// x 16384 200 us there), while matrix instructions alone reach 6.8 PFLOP/s on random codes
// at the clock that power leaves them and 9.6 on zeros (100 us).  A short K pays the end of
// a unit besides: 4.5 us of a 256x256 one, its stores waited for one stage after their
// issue by all CUs at once (4096 x 24576 x 1536 105 us, its products alone 45).
// Timing copies without the stage copies ran 20 % faster, without the barrier 6 %,
// without the scales 6 %, without the fragment reads 11 %, without any of them 6.4
// PFLOP/s; waiting for fewer copies, or copying from L2 only, changed 1 and 3-8 %.  The
// middle sizes (one 96x128 tile per workgroup) wait for copies: from L2 only they ran 12
// % faster; and where tiles fill just over half of the CUs the others have nothing to do
// (4096 x 2112 x 7168, 144 tiles, 51 us; split_rule takes no K slices there).
// Tried without gain: four waves of 128x128 each (fewer LDS reads per matrix
// instruction, but the accumulators take half of the registers and the rest spills: 3-8
// % slower), only half of the waves copying, more of a stage's copies put off into the
// next one, loads that pull the next stage into L2, a later barrier, raised wave
// priority, other raster bands, a 256x224 tile.  Not tried: non-temporal stores of D,
// stages of one K block in more slots, tiles of 128x192 and 192x192.
#include <algorithm>
#include <cstdio>
#include <cstdlib>

#include "../../include/dg.h"
#include "mxfp4_tile.hpp"

namespace dg {

static const Mxfp4TileInfo kMxTiles[] = {
#define X(id, MT, NT, WM, WN, R, KG) {MxTile<MT, NT, WM, WN, R, KG>::BM, MxTile<MT, NT, WM, WN, R, KG>::BN, KG, MxTile<MT, NT, WM, WN, R, KG>::LDS, NT < 4},
    DG_MXFP4_TILES(X) DG_MXFP4_GROUPED_TILES(X)
#undef X
};

Mxfp4TileInfo mxfp4_tile_info(int id) { return kMxTiles[id]; }

static int skinny_rows(int id) {
  switch (id) {
#define X(i, MT, P) case i: return MT * 16;
    DG_MXFP4_SKINNY(X)
#undef X
  }
  return 0;
}

static Mxfp4Plan plan_mxfp4_tile(int m, int n, int k, int cus, int id) {
  Mxfp4Plan pl{};
  const Mxfp4TileInfo t = kMxTiles[id];
  pl.skinny = -1;
  pl.tile = id;
  pl.tiles_m = (m + t.bm - 1) / t.bm;
  pl.tiles_n = (n + t.bn - 1) / t.bn;
  const long long tiles = (long long)pl.tiles_m * pl.tiles_n;
  const int kb = k / 128;
  long long full = tiles;
  pl.splits = t.kg > 1 ? 1 : split_rule(tiles, cus, kb, &full);
  pl.kb_per_split = kb;
  if (pl.splits > 1) {
    pl.kb_per_split = ((kb + pl.splits - 1) / pl.splits + 1) & ~1;   // whole stages
    pl.splits = (kb + pl.kb_per_split - 1) / pl.kb_per_split;
    if (pl.splits < 2) {
      pl.splits = 1;
      pl.kb_per_split = kb;
      full = tiles;
    }
  }
  pl.full_tiles = (int)full;
  pl.units = (int)(full + (tiles - full) * pl.splits);
  pl.ws_bytes = (size_t)(tiles - full) * (pl.splits > 1 ? pl.splits : 0) * t.bm * t.bn * 4;
  pl.grid = std::min(pl.units, cus);
  return pl;
}

int mxfp4_forced() {
  const char* f = std::getenv("DG_FORCE_MXFP4");   // (for tuning)
  return f ? std::atoi(f) : -1;
}

// Of each tile: a stage of 256 values of K, and a unit's fixed share, in microseconds.
static constexpr double kStage[] = {1.85, 1.12, 0.76, 0.69, 0.57, 0.81, 0.52, 1.05, 1.45};
static constexpr double kUnit[] = {4.5, 2.0, 1.0, 1.0, 1.8, 1.9, 1.6, 2.5, 3.3};
static_assert(sizeof(kStage) / sizeof(kStage[0]) == kMxGroupedTileCount && sizeof(kMxTiles) / sizeof(kMxTiles[0]) == kMxGroupedTileCount,
              "tiles");

double mxfp4_tile_time(int id, long long units, int kb, int cus) {
  const int kg = kMxTiles[id].kg, whole = ((kb + 1) / 2 + kg - 1) / kg;
  return (double)((units + cus - 1) / cus) * (whole * kStage[id] + kUnit[id]);
}

// Up to 32 rows: the streaming kernel reads all of A once per 16 columns, so it is taken
// while row blocks x columns stay small (measured against the best tile: 1 x 4096 x 7168
// 6.0 against 9.7 us, 16 x 7168 x 2048 5.9 / 5.7, 32 x 4096 x 7168 8.5 / 9.9; past the
// limit 1 x 24576 x 1536 10.7 / 7.5, 32 x 7168 x 16384 28.8 / 19.7).  Otherwise the tile
// with the least estimated time in microseconds: rounds of units, each its stages at the
// tile's pace and a fixed share (pipeline fill, D); a split plan's partials' round trip
// and second launch; and the rate at which the units' CUs stream B.  The constants fit
// 247 shapes, M 1 to 8192, 512 x 2048 to 32768 x 512 and 7168 x 16384 (geometric mean
// 0.2 % over the best tile of each; worst 64 x 7168 x 16384, 18 %).
Mxfp4Plan plan_mxfp4(int m, int n, int k, int cus) {
  constexpr double kSplit = 5.7, kPartialRate = 3.6e6, kStreamRate = 40.0e3;   // us, bytes per us
  const int force = mxfp4_forced();
  int skinny = -1;
  const int mt = m <= 16 ? 1 : m <= 32 ? 2 : 0;
  if (mt && (long long)mt * n <= 8192) skinny = mt >> 1;
  if (force >= 0) skinny = force >= kMxSkinnyIdBase && skinny_rows(force - kMxSkinnyIdBase) >= m ? force - kMxSkinnyIdBase : -1;
  Mxfp4Plan best{};
  if (skinny >= 0) {
    best.skinny = skinny;
    return best;
  }
  double best_t = 1e30;
  for (int id = 0; id < kMxTileCount; ++id) {
    const int kg = kMxTiles[id].kg;
    const Mxfp4Plan pl = plan_mxfp4_tile(m, n, k, cus, id);
    if (kg > 1 && pl.units > cus) continue;   // one unit per workgroup (a pinned one is passed over, too)
    double t = mxfp4_tile_time(id, pl.full_tiles, k / 128, cus);
    if (pl.splits > 1)
      t += (pl.kb_per_split + 1) / 2 * kStage[id] + kUnit[id] + kSplit + 2.0 * (double)pl.ws_bytes / kPartialRate;
    t = std::max(t, 0.5 * n * k / (kStreamRate * std::min(pl.units, cus)));
    if (t < best_t - 1e-9 || id == force) {
      best_t = id == force ? 0.0 : t;
      best = pl;
    }
  }
  return best;
}

void log_mxfp4_plan(const char* call, int m, int n, int k, const Mxfp4Plan& pl) {
  const char* log = std::getenv("DG_LOG");
  if (!log || log[0] != '1') return;
  if (pl.skinny >= 0)
    std::fprintf(stderr, "[dg] %s m=%d n=%d k=%d -> streaming kernel, %d rows\n", call, m, n, k, skinny_rows(pl.skinny));
  else
    std::fprintf(stderr, "[dg] %s m=%d n=%d k=%d -> tile %dx%d, %d K group%s, %d tiles (%d whole, the rest x %d K slices), "
                 "%d workgroups, workspace %zu bytes\n", call, m, n, k, kMxTiles[pl.tile].bm, kMxTiles[pl.tile].bn,
                 kMxTiles[pl.tile].kg, kMxTiles[pl.tile].kg > 1 ? "s" : "", pl.tiles_m * pl.tiles_n, pl.full_tiles, pl.splits,
                 pl.grid, pl.ws_bytes);
}

bool mxfp4_sizes_fit(int m, int n, int k) {
  const long long lim = 1LL << 31;
  return k % 128 == 0 && n % 16 == 0 && (long long)m * (k / 2) <= lim && (long long)n * (k / 2) <= lim &&
         (long long)m * n * 2 <= lim && (long long)m * (k / 32) <= lim && (long long)n * (k / 32) <= lim;
}

static bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

}  // namespace dg

using namespace dg;

extern "C" {

size_t dg_mxfp4_gemm_workspace_bytes(int m, int n, int k, int num_cus) {
  try {
    if (m <= 0 || n <= 0 || k <= 0 || !mxfp4_sizes_fit(m, n, k)) return 0;
    if (num_cus <= 0) num_cus = dg_get_num_cus();
    if (num_cus <= 0) return 0;
    return plan_mxfp4(m, n, k, num_cus).ws_bytes;
  } catch (...) {
    return 0;
  }
}

int dg_mxfp4_gemm_nt(const uint8_t* a, const int32_t* a_sf, const uint8_t* b, const int32_t* b_sf,
                     const uint16_t* c, uint16_t* d, int m, int n, int k, void* workspace, size_t workspace_bytes,
                     void* stream) {
  try {
    if (!a || !a_sf || !b || !b_sf || !d) return DG_ERR_INVALID_ARG;
    if (m <= 0 || n <= 0 || k <= 0) return DG_ERR_INVALID_ARG;
    if (misaligned(a, 16) || misaligned(b, 16) || misaligned(c, 16) || misaligned(d, 16) || misaligned(a_sf, 4) ||
        misaligned(b_sf, 4))
      return DG_ERR_INVALID_ARG;
    if (!mxfp4_sizes_fit(m, n, k)) return DG_ERR_UNSUPPORTED;
    DeviceInfo di = current_device_info();
    if (!di.ok) return DG_ERR_NO_DEVICE;
    const int cus = dg_get_num_cus();
    const Mxfp4Plan pl = plan_mxfp4(m, n, k, cus);
    if (pl.ws_bytes && (!workspace || workspace_bytes < pl.ws_bytes || misaligned(workspace, 16)))
      return DG_ERR_INVALID_ARG;
    Mxfp4Params p{a, a_sf, b, b_sf, c, d, static_cast<float*>(workspace), m, n, k,
                  pl.tiles_m, pl.tiles_n, 8, pl.splits, pl.kb_per_split, pl.full_tiles, pl.units};
    log_mxfp4_plan("mxfp4_gemm_nt", m, n, k, pl);
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    hipError_t e = pl.skinny >= 0 ? launch_mxfp4_skinny(p, pl.skinny, hs) : launch_mxfp4_tile(p, pl.tile, pl.grid, hs);
    if (e == hipSuccess && pl.ws_bytes) {
      const Mxfp4TileInfo t = kMxTiles[pl.tile];
      Fp8GemmParams rp{};
      rp.ws = p.ws; rp.c = c; rp.d = d; rp.m = m; rp.n = n; rp.k = k; rp.num_groups = 1;
      rp.tiles_m = pl.tiles_m; rp.tiles_n = pl.tiles_n; rp.group_m = p.group_m;
      GemmPlan rpl{};
      rpl.block_m = t.bm; rpl.block_n = t.bn; rpl.num_tiles = pl.tiles_m * pl.tiles_n;
      rpl.full_tiles = pl.full_tiles; rpl.splits = pl.splits;
      e = launch_splitk_reduce(rp, rpl, cus, hs);
    }
    return e == hipSuccess ? DG_OK : DG_ERR_HIP;
  } catch (...) {
    return DG_ERR_HIP;
  }
}

}  // extern "C"
