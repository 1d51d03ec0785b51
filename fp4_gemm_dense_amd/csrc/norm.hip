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
// Bound: HBM (forward 7 bytes per element with a residual, backward 8); rows of up to some
// 512 by the waves they take, one or two of them a row.  Measured (one MI355X, inputs not
// in the caches; a 1 GiB copy runs at 5.1 TB/s): forward 8192 x 7168 70 us MXFP4, 74 UE8M0,
// 76 fp32 scales (5.4-5.6 TB/s), 8192 x 512 7.8-8.3 (floor 5.5), 65536 x 128 26-27 (floor
// 11: 16 of a wave's 64 lanes have values), 3 x 7168 3.9, of which the launch is 2.7;
// backward 4096 x 7168 46.5 us in both kernels (5.1 TB/s), 8192 x 512 15, 65536 x 128 51
// (floors 6.5 and 13: at most 1024 workgroups walk the rows), 130 x 2048 3.9.
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
  double inv_k;
};

// A row is spread over a workgroup of 64 .. 1024 threads (whole waves), V vectors of 8
// values per thread: vector i of thread t is i * threads + t, so 16 lanes side by side
// hold a 1x128 block and a wave's 64 vectors one UE8M0 word's four blocks.
struct NormShape {
  int v, threads;
};
static NormShape norm_shape(int k) {
  const int nv = k / 8;
  const int v = nv <= 256 ? 1 : nv <= 1024 ? 2 : 4;
  return {v, ((nv + v - 1) / v + 63) / 64 * 64};
}
constexpr int NORM_MAX_K = 32768, NORM_MAX_WAVES = 16;

template <int O>
__device__ __forceinline__ float lane_swap(float v) {
  return __uint_as_float(lane_swap<O>(__float_as_uint(v)));
}
template <int O>
__device__ __forceinline__ double lane_swap(double v) {
  const uint64_t b = (uint64_t)__double_as_longlong(v);
  return __longlong_as_double((long long)((uint64_t)lane_swap<O>((uint32_t)(b >> 32)) << 32 | lane_swap<O>((uint32_t)b)));
}

// Sum of v over the workgroup, in a fixed order; every thread gets it.  One barrier: a
// caller that sums again passes another buffer.
template <typename F>
__device__ __forceinline__ F block_sum(F v, F* red) {
  v += lane_swap<1>(v);
  v += lane_swap<2>(v);
  v += lane_swap<4>(v);
  v += lane_swap<8>(v);
  v += __shfl_xor(v, 16, 64);
  v += __shfl_xor(v, 32, 64);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) red[threadIdx.x >> 6] = v;
  __syncthreads();
  F s = 0;
  for (int w = 0; w < waves; ++w) s += red[w];
  return s;
}

// Bounds of max |h * weight|, 2^-100 .. 2^100.  From the lower one on the products of a
// block are exact (one that is subnormal beside the largest has code 0); within both no
// step of a quotient by them leaves fp32's normal range.  And of max |y|: for a scale of
// 2^-126 or more (448 * 2^-126), and 2^-126 .. 2^127, where truncating it leaves neither 0
// nor the largest number for what is past them.
constexpr uint32_t kExactLo = 27u << 23, kExactHi = 227u << 23, kNormalScale = 0x04e00000u;
constexpr uint32_t kNormalLo = 1u << 23, kNormalHi = 254u << 23;

// y is rounded twice, to fp32 and to its code.  So that the second rounding goes to the
// nearer side, the first one goes to odd: toward zero, with the last bit set where anything
// was cut off (midpoints of codes and borders between scales have five significant bits
// at most, so that an odd y is never one of them).  r is the sum of two fp32 numbers, which
// leaves 2^-48 of y; lo is not 0, so that no product is exact but 0, which becomes 2^-149
// of its sign and has code 0 all the same.  (With fp32 roundings of r and y one code in
// four million differed from y's in 64 bits.  It costs some 1 % of a long row and 5 % of a
// short one, a third of it for the squares in fp64: 8192 x 7168 with UE8M0 scales 72.3 ->
// 73.0 us, 8192 x 512 7.5 -> 7.9, 65536 x 128, which the vector ALUs bound, 22.6 -> 25.4.)
struct TwoFloats {
  float hi, lo;
};
__device__ __forceinline__ void times_odd(const float (&product)[8], TwoFloats r, float (&y)[8]) {
  float t[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) t[e] = product[e] * r.lo;
  // (the rounding mode of fp32 is set within the block, which the compiler cannot enter)
  asm("s_setreg_imm32_b32 hwreg(HW_REG_MODE, 0, 2), 3\n\t"
      "v_fma_f32 %0, %8, %16, %17\n\t"
      "v_fma_f32 %1, %9, %16, %18\n\t"
      "v_fma_f32 %2, %10, %16, %19\n\t"
      "v_fma_f32 %3, %11, %16, %20\n\t"
      "v_fma_f32 %4, %12, %16, %21\n\t"
      "v_fma_f32 %5, %13, %16, %22\n\t"
      "v_fma_f32 %6, %14, %16, %23\n\t"
      "v_fma_f32 %7, %15, %16, %24\n\t"
      "s_setreg_imm32_b32 hwreg(HW_REG_MODE, 0, 2), 0"
      : "=&v"(y[0]), "=&v"(y[1]), "=&v"(y[2]), "=&v"(y[3]), "=&v"(y[4]), "=&v"(y[5]), "=&v"(y[6]), "=&v"(y[7])
      : "v"(product[0]), "v"(product[1]), "v"(product[2]), "v"(product[3]), "v"(product[4]), "v"(product[5]), "v"(product[6]),
        "v"(product[7]), "v"(r.hi), "v"(t[0]), "v"(t[1]), "v"(t[2]), "v"(t[3]), "v"(t[4]), "v"(t[5]), "v"(t[6]), "v"(t[7]));
#pragma unroll
  for (int e = 0; e < 8; ++e) y[e] = __uint_as_float(__float_as_uint(y[e]) | 1u);
}
// The pattern of one positive product's y to odd, from its rounding to nearest.
__device__ __forceinline__ uint32_t times_odd(float product, TwoFloats r) {
  const float t = product * r.lo, y = fmaf(product, r.hi, t);
  const float err = fmaf(product, r.hi, -y) + t;
  return (__float_as_uint(y) - (__float_as_uint(err) >> 31)) | 1u;
}
__device__ __forceinline__ float fp64_to_odd(double v) {
  const float f = (float)v;
  const uint32_t u = __float_as_uint(f);
  if ((double)f == v || f == 0.f || !(fabsf(f) < INFINITY)) return f;   // (below fp32's least: 0)
  return __uint_as_float((fabs((double)f) > fabs(v) ? u - 1 : u) | 1u);
}

// y = h * weight * r of one vector where the product may have left fp32's range (or the
// block is zeros or not finite), in fp64, rounded to odd (ODD) or to nearest.  Returns the
// pattern of max |y| over the block's LANES lanes, which all take part.
template <int LANES, bool ODD>
__device__ __forceinline__ uint32_t y_by_fp64(const v4i& h, const v4i& weight, double r, float (&y)[8]) {
  float a[8], w[8];
  unpack_bf16x8(h, a);
  unpack_bf16x8(weight, w);
  uint32_t amax = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double v = (double)a[e] * (double)w[e] * r;
    y[e] = ODD ? fp64_to_odd(v) : (float)v;
    amax = umax(amax, abs_bits(y[e]));
  }
  return group_max<LANES>(amax);
}

// One row per workgroup.  (Measured against 2, 4 and 8 rows per workgroup, with the
// next row loaded ahead and the K-block-major scales leaving in longer runs, and
// against 2 to 8 persistent workgroups per CU: one row was the fastest at 8192 x 7168
// in every format, 70-75 us against 73-84.)
template <int FMT, int V>
__global__ void __launch_bounds__(V == 4 ? 1024 : 512) add_rms_norm_kernel(NormParams p) {
  __shared__ double red[NORM_MAX_WAVES];
  const int tid = threadIdx.x, nt = blockDim.x;
  const int nv = p.k >> 3, kb_n = p.k >> 7;
  const int row = blockIdx.x;
  const size_t base = (size_t)row * nv;
  v4i hv[V], rv[V], wv[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = i * nt + tid;
    hv[i] = rv[i] = wv[i] = v4i{0, 0, 0, 0};
    if (j < nv) {
      hv[i] = reinterpret_cast<const v4i*>(p.x)[base + j];
      if (p.residual) rv[i] = reinterpret_cast<const v4i*>(p.residual)[base + j];
      wv[i] = reinterpret_cast<const v4i*>(p.weight)[j];
    }
  }
  double ss = 0;   // (the squares of bf16 numbers are exact in fp64, and its range holds them)
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = i * nt + tid;
    float a[8];
    unpack_bf16x8(hv[i], a);
    if (p.residual) {
      float b[8];
      unpack_bf16x8(rv[i], b);
#pragma unroll
      for (int e = 0; e < 8; ++e) a[e] += b[e];
      hv[i] = pack_bf16x8(a);
      unpack_bf16x8(hv[i], a);
    }
    if (p.h && j < nv) reinterpret_cast<v4i*>(p.h)[base + j] = hv[i];
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = fma((double)a[e], (double)a[e], ss);
  }
  // the sum and r in 64 bits: a code near a border follows y = (h * weight) * r, whose first
  // product is exact (two bf16 values)
  const double r64 = 1.0 / sqrt(block_sum(ss, red) * p.inv_k + (double)p.eps);
  const float r = (float)r64;
  const TwoFloats r2 = {r, (float)(r64 - (double)r)};
  // the products that the two numbers serve (none where r is one number, or subnormal)
  const uint32_t span = r >= 0x1p-100f && r2.lo != 0.f ? kExactHi - kExactLo : 0u;
  if (p.rstd && tid == 0) p.rstd[row] = r;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = i * nt + tid;   // (j >= nv: whole groups of 16 lanes; their vectors are zeros)
    const bool in = j < nv;
    float y[8], w[8], prod[8];
    unpack_bf16x8(hv[i], y);
    unpack_bf16x8(wv[i], w);
    uint32_t pmax = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      prod[e] = y[e] * w[e];
      pmax = umax(pmax, abs_bits(prod[e]));
    }
    const int kb = j >> 4;
    constexpr int LANES = FMT == DG_QUANT_MXFP4 ? 4 : 16;
    pmax = group_max<LANES>(pmax);
    const float ptop = __uint_as_float(pmax);
    // amax: of max |y| (rounding keeps the order)
    if constexpr (FMT == DG_QUANT_E4M3_F32) {
      uint32_t amax = abs_bits(ptop * r);
      const bool exact = pmax - kExactLo < kExactHi - kExactLo && amax - kNormalScale < 0x7f800000u - kNormalScale;
      if (__builtin_expect(!exact & in, 0)) amax = y_by_fp64<LANES, false>(hv[i], wv[i], r64, y);
      const float top = __uint_as_float(amax);
      const float s = amax == 0 ? 1.0f : (amax >= 0x7f800000u ? __uint_as_float(0x7fc00000u) : fmaxf(top / 448.0f, 0x1p-126f));
      if (in && (tid & 15) == 0) static_cast<float*>(p.sf)[(size_t)kb * p.m + row] = s;
      // y / s is 448 (h w) / max |h w| wherever s is not at its least: r cancels, both
      // products have 16 bits, and ties between two codes are common (1 in 2600 on normal
      // data).  The quotient by a reciprocal is corrected by its remainder, which is exact:
      // a tie comes out as itself and goes to the even code.  (y / s in fp32 decides one
      // tie in six by the roundings of y and s.)
      if (__builtin_expect(exact, 1)) {
        const float it = __builtin_amdgcn_rcpf(ptop);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float n = prod[e] * 448.0f, q0 = n * it;
          y[e] = fmaf(fmaf(-q0, ptop, n), it, q0);
        }
      } else {
        const float inv = amax == 0 || amax >= 0x7f800000u ? s : fminf(448.0f / top, 0x1p126f);   // (NaN: so are the codes)
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= inv;
      }
    } else {
      uint32_t amax = times_odd(ptop, r2), byte;
      const bool two = ((pmax - kExactLo < span) & (amax - kNormalLo < kNormalHi - kNormalLo)) | !in;
      if constexpr (FMT == DG_QUANT_MXFP4) {
        if (__builtin_expect(two, 1)) times_odd(prod, r2, y);
        else amax = y_by_fp64<LANES, true>(hv[i], wv[i], r64, y);
        byte = ue8m0_byte<false>(amax);
        const uint32_t word = scale_word(byte);
        if (in) {
          static_cast<uint32_t*>(p.q)[base + j] = byte == 255u ? 0u : e2m1x8(y, ue8m0_value(byte));
          if ((tid & 15) == 0) static_cast<uint32_t*>(p.sf)[(size_t)kb * p.m + row] = word;
        }
        continue;
      }
      if (__builtin_expect(two, 1)) {
        byte = in ? ue8m0_byte<true>(amax) : 127u;
        const float inv = __uint_as_float((254u - byte) << 23);             // 2^(127 - byte)
        times_odd(prod, TwoFloats{r2.hi * inv, r2.lo * inv}, y);            // (both products are exact)
      } else {
        byte = ue8m0_byte<true>(y_by_fp64<LANES, true>(hv[i], wv[i], r64, y));
        const float inv = ue8m0_value(byte == 255u ? 255u : 254u - byte);
#pragma unroll
        for (int e = 0; e < 8; ++e) y[e] *= inv;
      }
      // the wave's four blocks make one word (past the end: 2^0)
      uint32_t word = byte << (8 * ((tid >> 4) & 3));
      word |= (uint32_t)__shfl_xor((int)word, 16, 64);
      word |= (uint32_t)__shfl_xor((int)word, 32, 64);
      if (in && (tid & 63) == 0) static_cast<uint32_t*>(p.sf)[(size_t)row * ((kb_n + 3) >> 2) + (kb >> 2)] = word;
    }
    if constexpr (FMT != DG_QUANT_MXFP4)
      if (in)
        static_cast<v2i*>(p.q)[base + j] = v2i{(int)e4m3x4(y[0], y[1], y[2], y[3]), (int)e4m3x4(y[4], y[5], y[6], y[7])};
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
// share of dweight in registers over them and writes one partial row at the end.  The
// next row's dy and h are loaded before this row's sum is waited for.  With more than
// 512 threads a thread has 128 registers, too few for two rows (or even one): dy and h
// are then read again for dx.
template <int V, int THREADS>
__global__ void __launch_bounds__(THREADS) rms_norm_backward_kernel(NormBackParams p) {
  __shared__ float red[2][NORM_MAX_WAVES];
  constexpr bool AHEAD = THREADS <= 512;
  const int tid = threadIdx.x, nt = blockDim.x;
  const int nv = p.k >> 3;
  const float inv_k = 1.0f / (float)p.k;
  const v4i none = {0, 0, 0, 0};
  auto at = [&](const uint16_t* t, int row, int i) -> v4i {
    const int j = i * nt + tid;
    return j < nv ? reinterpret_cast<const v4i*>(t)[(size_t)row * nv + j] : none;
  };
  float dw[V][8];
  v4i wv[V], dyn[V], hn[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    wv[i] = at(p.weight, 0, i);
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[i][e] = 0.f;
  }
  int row = blockIdx.x, turn = 0;
  float rn = 0.f;
  auto load_next = [&](int r) {
    rn = p.rstd[r];
#pragma unroll
    for (int i = 0; i < V; ++i) {
      dyn[i] = at(p.dy, r, i);
      hn[i] = at(p.h, r, i);
    }
  };
  if (AHEAD && row < p.m) load_next(row);
  for (; row < p.m; row += gridDim.x) {
    v4i dyc[V], hc[V], dhc[V];
    float dot = 0.f;
    const float r = AHEAD ? rn : p.rstd[row];
    if (AHEAD && p.dh) {
#pragma unroll
      for (int i = 0; i < V; ++i) dhc[i] = at(p.dh, row, i);
    }
#pragma unroll
    for (int i = 0; i < V; ++i) {
      dyc[i] = AHEAD ? dyn[i] : at(p.dy, row, i);
      hc[i] = AHEAD ? hn[i] : at(p.h, row, i);
      float a[8], n[8], w[8];
      unpack_bf16x8(dyc[i], a);
      unpack_bf16x8(hc[i], n);
      unpack_bf16x8(wv[i], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        n[e] *= r;
        dw[i][e] = fmaf(a[e], n[e], dw[i][e]);
        dot = fmaf(a[e] * w[e], n[e], dot);
      }
    }
    if (AHEAD && row + (int)gridDim.x < p.m) load_next(row + gridDim.x);
    const float mean = block_sum(dot, red[turn]) * inv_k;
    turn ^= 1;
#pragma unroll
    for (int i = 0; i < V; ++i) {
      const int j = i * nt + tid;
      float a[8], n[8], w[8], d[8];
      unpack_bf16x8(AHEAD ? dyc[i] : at(p.dy, row, i), a);
      unpack_bf16x8(AHEAD ? hc[i] : at(p.h, row, i), n);
      unpack_bf16x8(wv[i], w);
      unpack_bf16x8(p.dh ? (AHEAD ? dhc[i] : at(p.dh, row, i)) : none, d);
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] += r * (a[e] * w[e] - n[e] * r * mean);
      if (j < nv) reinterpret_cast<v4i*>(p.dx)[(size_t)row * nv + j] = pack_bf16x8(d);
    }
  }
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = i * nt + tid;
    if (j >= nv) continue;
    v4f* o = reinterpret_cast<v4f*>(p.part + (size_t)blockIdx.x * p.k + (size_t)j * 8);
    o[0] = v4f{dw[i][0], dw[i][1], dw[i][2], dw[i][3]};
    o[1] = v4f{dw[i][4], dw[i][5], dw[i][6], dw[i][7]};
  }
}

// dweight from the partial rows: a workgroup sums 32 columns, 8 threads (4 columns
// each) across and 32 down, each every 32nd row; their sums meet in LDS in order.
__global__ void __launch_bounds__(256) norm_dweight_kernel(const float* part, float* dweight, int parts, int k) {
  __shared__ v4f sums[32][8];
  const int cx = threadIdx.x & 7, ry = threadIdx.x >> 3;
  const float* src = part + (size_t)blockIdx.x * 32 + cx * 4;
  v4f s = {0.f, 0.f, 0.f, 0.f};
  for (int i = ry; i < parts; i += 8 * 32) {
    v4f t[8];
#pragma unroll
    for (int u = 0; u < 8; ++u)
      t[u] = i + u * 32 < parts ? *reinterpret_cast<const v4f*>(src + (size_t)(i + u * 32) * k) : v4f{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int u = 0; u < 8; ++u) s += t[u];
  }
  sums[ry][cx] = s;
  __syncthreads();
  if (threadIdx.x < 8) {
    v4f t = sums[0][threadIdx.x];
#pragma unroll
    for (int y = 1; y < 32; ++y) t += sums[y][threadIdx.x];
    *reinterpret_cast<v4f*>(dweight + (size_t)blockIdx.x * 32 + threadIdx.x * 4) = t;
  }
}

// Few rows: one launch and no workspace.  dweight needs no row's sum (n = h * rstd), so
// the first k / 64 workgroups read 64 columns of dy and h once more and add them up, 8
// threads (8 columns each) across and the others down the rows; one workgroup more for
// each row forms dx.  first: the workgroup to start at (dx written over dy or h: two
// launches, dweight's and then the rows').
template <int V, int THREADS>
__global__ void __launch_bounds__(THREADS) rms_norm_backward_few_kernel(NormBackParams p, float* dweight, int first) {
  __shared__ float sums[NORM_MAX_WAVES][64];
  __shared__ float red[NORM_MAX_WAVES];
  const int tid = threadIdx.x, nt = blockDim.x;
  const int block = first + (int)blockIdx.x, dw_blocks = p.k >> 6;
  const int nv = p.k >> 3;
  if (block < dw_blocks) {
    const int cx = tid & 7, wave = tid >> 6, step = nt >> 3;
    const size_t col = (size_t)block * 8 + cx;
    float dw[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int r0 = tid >> 3; r0 < p.m; r0 += 4 * step) {
      v4i dy[4], h[4];
      float r[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int row = min(r0 + u * step, p.m - 1);
        dy[u] = reinterpret_cast<const v4i*>(p.dy)[(size_t)row * nv + col];
        h[u] = reinterpret_cast<const v4i*>(p.h)[(size_t)row * nv + col];
        r[u] = p.rstd[row];
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (r0 + u * step >= p.m) break;
        float a[8], n[8];
        unpack_bf16x8(dy[u], a);
        unpack_bf16x8(h[u], n);
#pragma unroll
        for (int e = 0; e < 8; ++e) dw[e] = fmaf(a[e], n[e] * r[u], dw[e]);
      }
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) {
#pragma unroll
      for (int o = 8; o < 64; o <<= 1) dw[e] += __shfl_xor(dw[e], o, 64);
      if ((tid & 63) < 8) sums[wave][cx * 8 + e] = dw[e];
    }
    __syncthreads();
    if (tid < 64) {
      float t = sums[0][tid];
      for (int w = 1; w < nt >> 6; ++w) t += sums[w][tid];
      dweight[block * 64 + tid] = t;
    }
    return;
  }
  const int row = block - dw_blocks;
  const v4i none = {0, 0, 0, 0};
  v4i dy[V], h[V], w[V], dh[V];
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = i * nt + tid;
    const size_t at = (size_t)row * nv + j;
    const bool in = j < nv;
    dy[i] = in ? reinterpret_cast<const v4i*>(p.dy)[at] : none;
    h[i] = in ? reinterpret_cast<const v4i*>(p.h)[at] : none;
    w[i] = in ? reinterpret_cast<const v4i*>(p.weight)[j] : none;
    dh[i] = in && p.dh ? reinterpret_cast<const v4i*>(p.dh)[at] : none;
  }
  const float r = p.rstd[row];
  float dot = 0.f;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    float a[8], n[8], wf[8];
    unpack_bf16x8(dy[i], a);
    unpack_bf16x8(h[i], n);
    unpack_bf16x8(w[i], wf);
#pragma unroll
    for (int e = 0; e < 8; ++e) dot = fmaf(a[e] * wf[e], n[e] * r, dot);
  }
  const float mean = block_sum(dot, red) * (1.0f / (float)p.k);
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int j = i * nt + tid;
    float a[8], n[8], wf[8], d[8];
    unpack_bf16x8(dy[i], a);
    unpack_bf16x8(h[i], n);
    unpack_bf16x8(w[i], wf);
    unpack_bf16x8(dh[i], d);
#pragma unroll
    for (int e = 0; e < 8; ++e) d[e] += r * (a[e] * wf[e] - n[e] * r * mean);
    if (j < nv) reinterpret_cast<v4i*>(p.dx)[(size_t)row * nv + j] = pack_bf16x8(d);
  }
}

// One launch pays up to some 1200 rows (130 x 2048 3.6 us, 5.9 with partial rows and a
// second launch; 600 x 7168 9.9 / 13.5; 1200 x 7168 18.2 / 21.5; 1200 x 2048 9.9 / 10.2;
// 2400 x 7168 41 / 34): each column is read by one workgroup.
static bool norm_few(int m) { return m <= 1024; }

// (a workgroup's next row, up to 1024 further, is an int)
static bool norm_backward_fits(int m, int k) { return k % 128 == 0 && k <= NORM_MAX_K && m <= 0x7fffffff - 1024; }

// Workgroups of the backward kernel, each with one partial row of dweight: one of up to
// eight waves per CU of the whole chip, or up to four smaller ones (more would write and
// read more partial rows than they overlap: 4096 x 7168 takes 49 us with 256, 54 with
// 512, 60 with 1024; 8192 x 512 takes 25, 17 and 14).  A function of the sizes alone, so
// that the order of the sums is, too.
static int norm_parts(int m, int k) {
  const int waves = norm_shape(k).threads / 64;
  return std::min(m, 256 * std::max(1, std::min(4, 8 / waves)));
}

template <int FMT>
static hipError_t launch_norm(const NormParams& p, hipStream_t hs) {
  const NormShape s = norm_shape(p.k);
  if (s.v == 1) hipLaunchKernelGGL((add_rms_norm_kernel<FMT, 1>), dim3(p.m), dim3(s.threads), 0, hs, p);
  else if (s.v == 2) hipLaunchKernelGGL((add_rms_norm_kernel<FMT, 2>), dim3(p.m), dim3(s.threads), 0, hs, p);
  else hipLaunchKernelGGL((add_rms_norm_kernel<FMT, 4>), dim3(p.m), dim3(s.threads), 0, hs, p);
  return hipGetLastError();
}

static hipError_t launch_norm_backward(const NormBackParams& p, int grid, hipStream_t hs) {
  const NormShape s = norm_shape(p.k);
  if (s.v == 1) hipLaunchKernelGGL((rms_norm_backward_kernel<1, 512>), dim3(grid), dim3(s.threads), 0, hs, p);
  else if (s.v == 2) hipLaunchKernelGGL((rms_norm_backward_kernel<2, 512>), dim3(grid), dim3(s.threads), 0, hs, p);
  else if (s.threads <= 512) hipLaunchKernelGGL((rms_norm_backward_kernel<4, 512>), dim3(grid), dim3(s.threads), 0, hs, p);
  else hipLaunchKernelGGL((rms_norm_backward_kernel<4, 1024>), dim3(grid), dim3(s.threads), 0, hs, p);
  return hipGetLastError();
}

// 512 threads up to 256 rows, 1024 for more (300 x 2048 5.3 us with 512, 4.9 with 1024;
// 130 x 2048 3.6 / 3.8), whatever the row's length: the columns' workgroups need them.
static hipError_t launch_norm_backward_few(const NormBackParams& p, float* dweight, int first, int grid, hipStream_t hs) {
  const int nv = p.k >> 3;
#define DG_FEW(V, T) hipLaunchKernelGGL((rms_norm_backward_few_kernel<V, T>), dim3(grid), dim3(T), 0, hs, p, dweight, first)
  if (p.m <= 256 && nv <= 512) DG_FEW(1, 512);
  else if (p.m <= 256 && nv <= 1024) DG_FEW(2, 512);
  else if (nv <= 1024) DG_FEW(1, 1024);
  else if (nv <= 2048) DG_FEW(2, 1024);
  else DG_FEW(4, 1024);
#undef DG_FEW
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
    // (a launch has fewer than 2^32 threads, and a row's workgroup at most this many)
    if ((long long)m * std::min(1024, (k / 8 + 63) / 64 * 64) >= 1LL << 32) return DG_ERR_UNSUPPORTED;
    DeviceInfo di = current_device_info();
    if (!di.ok) return DG_ERR_NO_DEVICE;
    NormParams p{x, residual, weight, h, q, sf, rstd, m, k, eps, 1.0 / k};
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    const hipError_t e = format == DG_QUANT_E4M3_F32     ? launch_norm<DG_QUANT_E4M3_F32>(p, hs)
                         : format == DG_QUANT_E4M3_UE8M0 ? launch_norm<DG_QUANT_E4M3_UE8M0>(p, hs)
                                                         : launch_norm<DG_QUANT_MXFP4>(p, hs);
    return e == hipSuccess ? DG_OK : DG_ERR_HIP;
  } catch (...) {
    return DG_ERR_HIP;
  }
}

size_t dg_add_rms_norm_backward_workspace_bytes(int m, int k) {
  if (m <= 0 || k <= 0 || !norm_backward_fits(m, k)) return 0;
  return norm_few(m) ? 0 : (size_t)norm_parts(m, k) * k * sizeof(float);
}

int dg_add_rms_norm_backward(const uint16_t* dy, const uint16_t* dh, const uint16_t* h, const uint16_t* weight,
                             const float* rstd, uint16_t* dx, float* dweight, int m, int k, void* workspace,
                             size_t workspace_bytes, void* stream) {
  try {
    if (!dy || !h || !weight || !rstd || !dx || !dweight) return DG_ERR_INVALID_ARG;
    if (m <= 0 || k <= 0) return DG_ERR_INVALID_ARG;
    if (misaligned(dy, 16) || misaligned(dh, 16) || misaligned(h, 16) || misaligned(weight, 16) ||
        misaligned(dx, 16) || misaligned(dweight, 16) || misaligned(rstd, 4))
      return DG_ERR_INVALID_ARG;
    if (!norm_backward_fits(m, k)) return DG_ERR_UNSUPPORTED;
    const size_t need = dg_add_rms_norm_backward_workspace_bytes(m, k);
    if (need && (!workspace || workspace_bytes < need || misaligned(workspace, 16))) return DG_ERR_INVALID_ARG;
    DeviceInfo di = current_device_info();
    if (!di.ok) return DG_ERR_NO_DEVICE;
    NormBackParams p{dy, dh, h, weight, rstd, dx, static_cast<float*>(workspace), m, k};
    hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
    hipError_t e;
    if (norm_few(m)) {
      const int dw = k / 64;
      if (dx == dy || dx == h) {
        e = launch_norm_backward_few(p, dweight, 0, dw, hs);
        if (e == hipSuccess) e = launch_norm_backward_few(p, dweight, dw, m, hs);
      } else {
        e = launch_norm_backward_few(p, dweight, 0, dw + m, hs);
      }
      return e == hipSuccess ? DG_OK : DG_ERR_HIP;
    }
    const int parts = norm_parts(m, k);
    e = launch_norm_backward(p, parts, hs);
    if (e != hipSuccess) return DG_ERR_HIP;
    hipLaunchKernelGGL(norm_dweight_kernel, dim3(k / 32), dim3(256), 0, hs, p.part, dweight, parts, k);
    return hipGetLastError() == hipSuccess ? DG_OK : DG_ERR_HIP;
  } catch (...) {
    return DG_ERR_HIP;
  }
}

}  // extern "C"
