// The backward pass through a linear layer's activation for gfx950: dz = dy * act'(z), or of a
// gated one dz = [dy * up * act'(gate), dy * act(gate)], quantised to MXFP4 for the products of
// the layer's gradients (along the rows for the input's, along the columns of the transposed
// operand for the weight's), with the bias gradient's column sums from the same read.
//
// dz is rounded to bf16 and quantised from there, so that the codes are those of the values
// that dz stores; the sums take the unrounded ones.
//
// Bound: HBM.  An element of dz costs 2 bytes of z and 2 of dy (gated: 1) of reading and
// 17/32 of writing per direction.  Measured (one MI355X, both directions and dbias): 4096 x 16384
// gated with SiLU 78-82 us (floor at a copy's 5.1 TB/s 53), SiLU alone 87-91 (66), the identity 83; 2001 x
// 4096 GELU 15.4 and 4.6 of the sums (8.1: 512 tiles on 256 CUs, whose reads, arithmetic and writes follow
// one another); 130 x 4096 gated 6.8 + 2.7.  Of the first, 9 us are dbias and 15 the columns.  (The 128-row
// gated kernel has 164 registers: one workgroup on a CU.  The ungated one has 115, the 32-row ones up to 99: two.)
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
  float* part;         // [chunks of row tiles][n] of dbias, or null
  int m, n, per;       // per: row tiles of a chunk
  Activation act;
};

// A workgroup of 512 takes `per` tiles of ROWS rows x 128 columns one below another (gated: of
// both halves): a thread has ROWS / 32 vectors of eight values, whose dz is quantised along the row
// as it goes to LDS; the columns are quantised from there (quant_tile.hpp), while the next
// tile's values are on their way.  The other half's dz waits in registers.  ROWS is 128, or 32 where
// that leaves most CUs without a tile, since a tile's arithmetic is one CU's.
constexpr int ACT_THREADS = 512;
template <bool GATED, int KIND, int ROWS>
__global__ void __launch_bounds__(ACT_THREADS) activation_backward_kernel(ActBackParams p) {
  constexpr int VECS = ROWS / 32;
  __shared__ QuantTile<uint16_t> lds;
  __shared__ float sums[ACT_THREADS / 64][128];
  const int tid = threadIdx.x;
  const int w = GATED ? p.n >> 1 : p.n;                         // columns of dy
  const uint32_t kb_n = (uint32_t)w >> 7, mb_n = ((uint32_t)p.m + 127) >> 7;
  const size_t half_mp = (size_t)mb_n * 64;
  const uint32_t chunk = blockIdx.x / kb_n, kb = blockIdx.x - chunk * kb_n;
  const uint32_t tiles = mb_n * (128 / ROWS), tile0 = chunk * (uint32_t)p.per, tile1 = min(tiles, tile0 + (uint32_t)p.per);
  const int rr = tid >> 4, c = (tid & 15) * 8;
  // (rows past the end lie past the buffers and read zeros; so does all of a z that is not there)
  v4i vy[VECS], vz[VECS], vu[GATED ? VECS : 1];
  auto rows_of = [&](uint32_t tile) { return max(0, min(ROWS, p.m - (int)(tile * ROWS))); };
  auto bytes_of = [&](uint32_t tile, int stride) -> uint32_t {
    const int rows = rows_of(tile);
    return rows == 0 ? 0u : ((uint32_t)(rows - 1) * (uint32_t)stride + 128u) * 2u;
  };
  auto place = [&](int s, int stride) { return (int)(((uint32_t)(s * 32 + rr) * (uint32_t)stride + (uint32_t)c) * 2u); };
  auto load = [&](uint32_t tile) {
    const size_t row0 = (size_t)tile * ROWS;
    const v4i rs_y = make_buffer_rsrc(p.dy + row0 * w + kb * 128u, bytes_of(tile, w));
    const v4i rs_z = make_buffer_rsrc(p.z + row0 * p.n + kb * 128u, p.z ? bytes_of(tile, p.n) : 0u);
#pragma unroll
    for (int s = 0; s < VECS; ++s) {
      vy[s] = dg_raw_buffer_load_v4i32(rs_y, place(s, w), 0, 0);
      vz[s] = dg_raw_buffer_load_v4i32(rs_z, place(s, p.n), 0, 0);
    }
  };
  auto load_up = [&](uint32_t tile) {
    if constexpr (GATED) {
      const v4i rs_u = make_buffer_rsrc(p.z + (size_t)tile * ROWS * p.n + kb * 128u + w, bytes_of(tile, p.n));
#pragma unroll
      for (int s = 0; s < VECS; ++s) vu[s] = dg_raw_buffer_load_v4i32(rs_u, place(s, p.n), 0, 0);
    }
  };
  float sum[8], sum_up[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) sum[e] = sum_up[e] = 0.f;
  load(tile0);
  load_up(tile0);
  for (uint32_t tile = tile0; tile < tile1; ++tile) {
    const int rows = rows_of(tile);
    const size_t row0 = (size_t)tile * ROWS;
    const uint32_t mb = tile * ROWS / 128, sub = tile % (128 / ROWS);
    auto out_of = [&](uint32_t col0) -> QuantOut {
      return {p.q ? reinterpret_cast<uint32_t*>(p.q) + ((row0 * p.n + col0) >> 3) : nullptr, nullptr,
              p.sf ? p.sf + (size_t)(col0 >> 7) * p.m + row0 : nullptr,
              p.qt ? p.qt + (size_t)col0 * half_mp + (size_t)mb * 64 + sub * 16 : nullptr,
              p.sft ? reinterpret_cast<int32_t*>(reinterpret_cast<uint8_t*>(p.sft + (size_t)mb * p.n + col0) + sub) : nullptr,
              (size_t)p.n >> 3, half_mp};
    };
    // a vector's dz on its way: to memory, to its codes, to LDS
    auto put = [&](const Vec8<uint16_t>& v, int r, uint32_t col0, const QuantOut& o) {
      if (p.dz && r < rows) *reinterpret_cast<v4i*>(p.dz + row0 * p.n + col0 + ((uint32_t)r * (uint32_t)p.n + (uint32_t)c)) = v.p;
      if (p.q || p.qt) quantize_tile_row<uint32_t>(lds, v, r, c, rows, o);   // (uniform)
    };
    const QuantOut o = out_of(kb * 128u);
#pragma unroll
    for (int s = 0; s < VECS; ++s) {
      float y[8], z[8], a[8], d[8];
      unpack_bf16x8(vy[s], y);
      unpack_bf16x8(vz[s], z);
      activate_both<KIND>(z, a, d, p.act);
      if constexpr (GATED) {
        float u[8];
        unpack_bf16x8(vu[s], u);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          d[e] *= y[e] * u[e];
          a[e] *= y[e];
          sum_up[e] += a[e];
        }
        vu[s] = pack_bf16x8(a);
        asm volatile("" : "+v"(vu[s]));   // (packed here, as the sums below)
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] *= y[e];
      }
      // (added here, not where the sums are used: until then the addends would take the registers
      // of two thirds of the waves)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum[e] += d[e];
        asm volatile("" : "+v"(sum[e]));
        if constexpr (GATED) asm volatile("" : "+v"(sum_up[e]));
      }
      put(Vec8<uint16_t>{pack_bf16x8(d)}, s * 32 + rr, kb * 128u, o);
      __builtin_amdgcn_sched_barrier(0);   // (one vector after another: side by side they take twice the registers)
    }
    if (tile + 1 < tile1) load(tile + 1);
    if (p.q || p.qt) quantize_tile_columns<ACT_THREADS, ROWS>(lds, rows, o);
    if constexpr (GATED) {
      const uint32_t col0 = (uint32_t)w + kb * 128u;
      const QuantOut o2 = out_of(col0);
#pragma unroll
      for (int s = 0; s < VECS; ++s) put(Vec8<uint16_t>{vu[s]}, s * 32 + rr, col0, o2);
      if (tile + 1 < tile1) load_up(tile + 1);
      if (p.q || p.qt) quantize_tile_columns<ACT_THREADS, ROWS>(lds, rows, o2);
    }
  }
  // the columns' sums: 32 threads down a column, in order
  auto put_sums = [&](float(&v)[8], uint32_t col0) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[e] += __shfl_xor(v[e], 16, 64);
      v[e] += __shfl_xor(v[e], 32, 64);
    }
    __syncthreads();   // (the sums before are read)
    if ((tid & 63) < 16) {
#pragma unroll
      for (int e = 0; e < 8; ++e) sums[tid >> 6][c + e] = v[e];
    }
    __syncthreads();
    if (tid < 128) {
      float s = sums[0][tid];
#pragma unroll
      for (int y = 1; y < ACT_THREADS / 64; ++y) s += sums[y][tid];
      p.part[(size_t)chunk * p.n + col0 + tid] = s;
    }
  };
  if (p.part && rows_of(tile0) > 0) {   // (uniform)
    put_sums(sum, kb * 128u);
    if constexpr (GATED) put_sums(sum_up, (uint32_t)w + kb * 128u);
  }
}

// dbias: the partial rows' sums, 32 columns a workgroup.
__global__ void __launch_bounds__(256) activation_dbias_kernel(const float* part, float* dbias, int parts, int n) {
  sum_rows(part, n, parts, dbias);
}

// Row tiles of 128, or of 32 where those serve a quarter of the chip's 256 CUs or fewer (130 x 4096
// gated 14.0 -> 11.6 us, 500 x 2048 13.1 -> 12.2), except where the partial rows would then need a
// launch that they do not need now (128 x 8192 9.2, 11.8 with 32), in chunks of as many tiles as give
// at most two workgroups to each of 256 CUs (one chunk where a row of tiles alone has more).  A chunk is
// a whole number of tiles, so that sizes just past an even share have far fewer workgroups (GELU 2048 x
// 4096 512, 18.3 us, 2049 x 4096 288, 21.5; SiLU 4096 x 32768 512, 173 us, 4096 x 32896 257, 256).
// (Functions of the sizes alone, so that the order of the sums is, too.)
struct ActPlan {
  int rows, per, chunks, sums;   // sums: the chunks that hold rows (the last block of 128 is filled up)
};
static ActPlan act_plan(int m, int columns) {
  const long long kb = columns / 128, mb = ((long long)m + 127) / 128;
  const int rows = mb * kb <= 64 && (mb > 1 || m <= 32) ? 32 : 128;
  const long long tiles = mb * (128 / rows), wanted = std::max<long long>(1, 512 / kb);
  const long long per = (tiles + wanted - 1) / wanted;
  return {rows, (int)per, (int)((tiles + per - 1) / per), (int)((((long long)m + rows - 1) / rows + per - 1) / per)};
}

template <bool GATED, int ROWS>
static hipError_t launch_activation_backward(const ActBackParams& p, int grid, hipStream_t hs) {
#define DG_ACT(K) hipLaunchKernelGGL((activation_backward_kernel<GATED, K, ROWS>), dim3(grid), dim3(ACT_THREADS), 0, hs, p)
  if (p.act.kind == ACT_KIND_CLAMP) DG_ACT(ACT_KIND_CLAMP);
  else if (p.act.kind == ACT_KIND_SIGMOID) DG_ACT(ACT_KIND_SIGMOID);
  else DG_ACT(ACT_KIND_ERF);
#undef DG_ACT
  return hipGetLastError();
}

static bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) % a) != 0; }

// (rows and blocks are ints; a tile's bytes are counted in 31 bits)
static bool activation_backward_fits(int m, int n, bool gated) {
  return n % (gated ? 256 : 128) == 0 && m <= 0x7fffffff - 127 && n < 1 << 23;
}

}  // namespace dg

using namespace dg;

extern "C" {

size_t dg_activation_backward_workspace_bytes(int m, int n) {
  if (m <= 0 || n <= 0 || !activation_backward_fits(m, n, false)) return 0;
  const int sums = std::max(act_plan(m, n).sums, n % 256 == 0 ? act_plan(m, n / 2).sums : 0);
  return sums <= 1 ? 0 : (size_t)sums * n * sizeof(float);
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
    const int cols = gated ? n / 2 : n;
    const ActPlan pl = act_plan(m, cols);
    // (a single partial row is dbias)
    float* const part = !dbias ? nullptr : pl.sums > 1 ? static_cast<float*>(workspace) : dbias;
    const ActBackParams p{dy, z, dz, q, sf, qt, sft, part, m, n, pl.per, act};
    const int grid = pl.chunks * (cols / 128);
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    hipError_t e;
    if (gated) e = pl.rows == 32 ? launch_activation_backward<true, 32>(p, grid, hs) : launch_activation_backward<true, 128>(p, grid, hs);
    else e = pl.rows == 32 ? launch_activation_backward<false, 32>(p, grid, hs) : launch_activation_backward<false, 128>(p, grid, hs);
    if (e != hipSuccess) return DG_ERR_HIP;
    if (!dbias || pl.sums == 1) return DG_OK;
    hipLaunchKernelGGL(activation_dbias_kernel, dim3(n / 32), dim3(256), 0, hs, part, dbias, pl.sums, n);
    return hipGetLastError() == hipSuccess ? DG_OK : DG_ERR_HIP;
  } catch (...) {
    return DG_ERR_HIP;
  }
}

}  // extern "C"
