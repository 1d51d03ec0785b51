// A 128 x 128 tile quantised to MXFP4 along its rows, its columns, or both (quant.hip,
// activation.hip, mxfp4_grouped.hip), and the row direction of eight values.
#pragma once

#include "dg_quant.hpp"

namespace dg {

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

// Where a tile's outputs go, from its first row and column; null: not wanted.
struct QuantOut {
  uint32_t* q;        // codes of eight values, `vecs` a row
  v4i* values;        // eight bf16 values, likewise
  int32_t* sf;        // scale words of the rows
  uint8_t* qt;        // transposed codes, `qt_stride` bytes a column
  int32_t* sft;       // scale words of the columns
  size_t vecs, qt_stride;
};

template <typename T>
struct QuantTile {
  __attribute__((aligned(16))) T tile[128][128];
  uint32_t words[128];
  __attribute__((aligned(4))) uint8_t bytes[128][4];
};

// Eight values of tile row r, columns c .. c + 7: quantised along the row on the way into LDS.
// All 16 lanes of a row take part; rows from `rows` on hold zeros.  Index: what a tile's offsets
// fit (32 bits take half the registers).
template <typename Index, typename T>
__device__ __forceinline__ void quantize_tile_row(QuantTile<T>& l, const Vec8<T>& v, int r, int c, int rows, const QuantOut& o) {
  v.to_lds(&l.tile[r][c]);
  if (o.q || o.values) {   // (uniform)
    const RowCodes w = quantize_row8(v);
    if (r < rows) {
      const Index at = (Index)r * (Index)o.vecs + (Index)(c >> 3);
      if (o.q) o.q[at] = w.w;
      if (o.values) o.values[at] = e2m1x8_to_bf16(w.w, w.scale);
    }
    if (c == 0) l.words[r] = w.word;
  }
}

// What is left when all rows are in LDS: the rows' scale words, and the columns.  With 256 threads
// one holds two columns of one block of 32 rows; with 512 (bf16) two columns of half a block, the
// other half 32 lanes apart.  ROWS = 32: the tile is one of the four blocks of 128 rows, whose
// places o.qt and o.sft are (then in bytes).
template <int THREADS, int ROWS = 128, typename T>
__device__ __forceinline__ void quantize_tile_columns(QuantTile<T>& l, int rows, const QuantOut& o) {
  const int tid = threadIdx.x;
  static_assert(ROWS == 128 || (ROWS == 32 && THREADS == 512), "tile");
  __syncthreads();
  if (o.sf && tid < rows) o.sf[tid] = (int32_t)l.words[tid];
  if (o.qt) {   // (uniform)
    uint8_t* stage = reinterpret_cast<uint8_t*>(l.tile);   // [128 columns][64 bytes, + 16 against bank conflicts]
    if constexpr (THREADS == 512) {
      static_assert(sizeof(T) == 2, "bf16");
      // (32 rows: the first two waves; the others repeat their reads and write nothing)
      const int c2 = ((tid >> 6) & 1) * 64 + (tid & 31) * 2, half = (tid >> 5) & 1, b = ROWS == 32 ? 0 : tid >> 7;
      uint32_t e[16];   // rows b*32 + half*16 .. of columns c2 (low half) and c2 + 1
      us2 am = us2{0, 0};
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        e[r] = *reinterpret_cast<const uint32_t*>(&l.tile[b * 32 + half * 16 + r][c2]);
        am = us2max(am, us2abs((int)e[r]));
      }
      am = us2max(am, __builtin_bit_cast(us2, __shfl_xor(__builtin_bit_cast(int, am), 32, 64)));
      v2i w[2];
      uint32_t byte[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        byte[h] = ue8m0_byte<false>((uint32_t)(h ? am.y : am.x) << 16);
        const float scale = ue8m0_value(byte[h]);
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          v4i pr;   // eight rows of the column
#pragma unroll
          for (int j = 0; j < 4; ++j)
            pr[j] = (int)__builtin_amdgcn_perm(e[8 * q + 2 * j + 1], e[8 * q + 2 * j], h ? 0x07060302u : 0x05040100u);
          w[h][q] = byte[h] == 255u ? 0 : (int)e2m1x8(pr, scale);
        }
      }
      __syncthreads();   // (the tile is read)
      if (ROWS == 128 || tid < 128) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          *reinterpret_cast<v2i*>(stage + (c2 + h) * 80 + b * 16 + half * 8) = w[h];
          if (half == 0) l.bytes[c2 + h][b] = (uint8_t)byte[h];
        }
      }
    } else {
      const int c2 = (tid & 63) * 2, b = tid >> 6;
      v4i w[2];
      uint32_t byte[2];
      if constexpr (sizeof(T) == 2) {
        uint32_t e[32];   // rows b*32 .. of columns c2 (low half) and c2 + 1
        us2 am = us2{0, 0};
#pragma unroll
        for (int r = 0; r < 32; ++r) {
          e[r] = *reinterpret_cast<const uint32_t*>(&l.tile[b * 32 + r][c2]);
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
          const float2 f = *reinterpret_cast<const float2*>(&l.tile[b * 32 + r][c2]);
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
      __syncthreads();   // (the tile is read)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        *reinterpret_cast<v4i*>(stage + (c2 + h) * 80 + b * 16) = w[h];
        l.bytes[c2 + h][b] = (uint8_t)byte[h];
      }
    }
    __syncthreads();
    // the codes leave through LDS: four lanes write the 64 bytes of a column, where each lane
    // writing its own would send 16-byte pieces of 64 lines
    if constexpr (ROWS == 32) {
      if (tid < 128) {
        *reinterpret_cast<v4i*>(o.qt + (size_t)tid * o.qt_stride) = *reinterpret_cast<const v4i*>(stage + tid * 80);
        reinterpret_cast<uint8_t*>(o.sft)[tid * 4] = l.bytes[tid][0];
      }
      __syncthreads();
      return;
    }
#pragma unroll
    for (int i = 0; i < 512 / THREADS; ++i) {
      const int col = i * (THREADS / 4) + (tid >> 2);
      *reinterpret_cast<v4i*>(o.qt + (size_t)col * o.qt_stride + (tid & 3) * 16) =
          *reinterpret_cast<const v4i*>(stage + col * 80 + (tid & 3) * 16);
    }
    if (tid < 128) o.sft[tid] = *reinterpret_cast<const int32_t*>(l.bytes[tid]);
  }
  __syncthreads();
}

// 256 threads: thread t holds columns 8 (t % 16) .. + 7 of rows t / 16 + 16 s in v[s].
template <typename T>
__device__ __forceinline__ void quantize_tile(QuantTile<T>& l, const Vec8<T> (&v)[8], int rows, const QuantOut& o) {
#pragma unroll
  for (int s = 0; s < 8; ++s) quantize_tile_row<size_t>(l, v[s], s * 16 + (threadIdx.x >> 4), (threadIdx.x & 15) * 8, rows, o);
  quantize_tile_columns<256>(l, rows, o);
}

}  // namespace dg
