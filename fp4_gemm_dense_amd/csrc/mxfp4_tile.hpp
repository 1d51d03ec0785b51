// The MXFP4 x MXFP4 product kernels (gfx950) as templates: the tile kernel and the one for few
// rows, by what becomes of a product (Mxfp4Params and the structs that follow it), and the
// plan of a dense call.
#pragma once

#include <atomic>

#include "dg_activation.hpp"
#include "dg_device.hpp"
#include "dg_internal.hpp"

namespace dg {

// What becomes of a product.
enum MxKind : int {
  MX_DENSE = 0,    // d = bf16(c + A.B^T)
  MX_LINEAR = 1,   // d = bf16(c + act(A.B^T + bias))
  MX_GATED = 2,    // d = bf16(c + act(gate) * up), gate and up the halves of A.B^T + bias
  MX_RAGGED = 3,   // rows in groups, each with a B of its own
  MX_KGROUP = 4    // K blocks in groups, each with a D of its own
};

struct Mxfp4Params {
  static constexpr MxKind KIND = MX_DENSE;
  const uint8_t* a;
  const int32_t* a_sf;
  const uint8_t* b;
  const int32_t* b_sf;
  const uint16_t* c;
  uint16_t* d;
  float* ws;
  int m, n, k;
  int tiles_m, tiles_n, group_m;
  int splits, kb_per_split;   // K slices of a split tile, K blocks per slice (even)
  int full_tiles;             // tiles [0, full_tiles) run whole, the others are split
  int units;                  // whole tiles and slices
};

template <bool GATED>
struct Mxfp4LinearParams : Mxfp4Params {
  static constexpr MxKind KIND = GATED ? MX_GATED : MX_LINEAR;
  const uint16_t* bias;   // [n] or null
  uint16_t* z;            // [m][n]: bf16 of A.B^T + bias, or null
  Activation act;
};

// Groups: m counts all rows of A (MX_RAGGED) or those of A^T.B's outputs (MX_KGROUP); units
// and full_tiles are the device's to find.
template <MxKind K>
struct Mxfp4GroupedParams : Mxfp4Params {
  static constexpr MxKind KIND = K;
  const int32_t* ms;      // [groups] rows of each group
  int groups;
};

__device__ __forceinline__ v4f mfma_mxfp4(const v4i& a, uint32_t sa, const v4i& b, uint32_t sb, const v4f& c) {
  const v8i a8 = {a.x, a.y, a.z, a.w, 0, 0, 0, 0}, b8 = {b.x, b.y, b.z, b.w, 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, b8, c, FMT_E2M1, FMT_E2M1, 0, (int)sa, 0, (int)sb);
}

// WM x WN waves of MT x NT blocks of 16 x 16; R ring slots; KG groups of such waves,
// each with a ring of its own, that take the stages of a tile in turn.
template <int MT_, int NT_, int WM_, int WN_, int R_, int KG_>
struct MxTile {
  static constexpr int MT = MT_, NT = NT_, WM = WM_, WN = WN_, R = R_, KG = KG_;
  static constexpr int NW = WM * WN, THREADS = NW * KG * 64;
  static constexpr int BM = WM * MT * 16, BN = WN * NT * 16;
  // a stage: A rows, B rows, then the scale words of both K blocks ([2][BM], [2][BN]) in
  // whole 1-KB copies
  static constexpr int NSA = (BM * 8 + 1023) / 1024, NSB = (BN * 8 + 1023) / 1024;
  static constexpr int OFF_B = BM * 128, OFF_SA = OFF_B + BN * 128, OFF_SB = OFF_SA + NSA * 1024;
  static constexpr int STAGE = OFF_SB + NSB * 1024, RING = R * STAGE;
  static constexpr int RA = BM / 8 / NW, RB = BN / 8 / NW;   // 1-KB copies (8 rows) per wave and stage
  static constexpr int LPS = RA + RB + 1;                    // copies per wave and stage, with one of scales
  static constexpr int NSTORE = MT * NT / 2;                 // 16-byte stores of D per lane
  static constexpr int BAR = 1;                              // column blocks ahead of the barrier
  // copies of a stage issued in the next stage's first K block, so that they spread over
  // both: with four column blocks half of them (4096 x 4096 x 7168 on 128x256 75 -> 69
  // us), with eight, or a ring of two slots, two (more come late: 3 % slower)
  static constexpr int LATE = NT == 8 || (KG > 1 && R == 2) ? 2 : NT == 4 ? 4 : 1;
  // One instance of the stage's code for a unit's first stage and the others, or two (the
  // first one's sums start from a constant).  With two the 256x256 tile runs out of
  // registers: 24 a lane go to memory as it starts (4001 x 4096 x 7168 63.3 us, 60.7 with
  // one).  The smaller tiles have room for both (200 x 4096 x 7168 13.4 us with one, 12.3
  // with two).
  static constexpr bool ONE = MT * NT == 32;
  static constexpr int LDS = KG * RING + (ONE ? 1024 : 0);   // and 1 KB that is written and not read
  // a linear layer's bias: BN values of R + 2 units behind that (with K groups: of one), in whole
  // copies of 128
  static constexpr int BIAS_COPIES = (BN + 127) / 128, BIAS_UNIT = BIAS_COPIES * 256;
  static constexpr int BIAS = (KG > 1 ? 1 : R + 2) * BIAS_UNIT;
  static_assert(LDS + BIAS <= 160 * 1024, "LDS");
  static_assert(NSA + NSB <= NW, "one scale copy per wave (some waves repeat another's)");
  static_assert(RA >= 1 && RB >= 1 && NT % 2 == 0 && LDS <= 160 * 1024 && NSTORE % KG == 0 && (KG == 1 || KG * BM * BN * 4 <= LDS),
                "tile shape");
};

// Chunk swizzles of an A and a B row.  A 16-byte LDS read serves lanes {0-3, 12-15,
// 20-27}, {4-11, 16-19, 28-31} and the same of the upper 32 together (measured: two
// lanes of one set on the same banks cost a cycle), over 64 banks, two rows.  With
// these the 16 lanes of a set meet 16 different 16-byte bank groups: A's fragment reads
// rows 0-15 by lane, B's rows 8a + b (a, b = 0..3; plus 4 in odd column blocks).
__device__ __forceinline__ int swz_a(int r) { return (r >> 1) & 7; }
__device__ __forceinline__ int swz_b(int r) { return ((r >> 1) & 1) | ((r >> 2) & 6); }

// The value x, opaque to the compiler: lane-dependent terms that only a change of tile
// needs are formed there, not held in registers through the K loop.
__device__ __forceinline__ int opaque(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// Waits until at most MORE (where first is set) or LESS vector-memory operations are in
// flight.  One asm block: a branch of the compiler's own would split the matrix
// instructions around it.
template <int LESS, int MORE>
__device__ __forceinline__ void wait_vmcnt_first(int first) {
  static_assert(LESS <= MORE && MORE < 64, "vmcnt");
  asm volatile(
      "s_cmp_lg_u32 %0, 0\n\t"
      "s_cbranch_scc1 .Lmore%=\n\t"
      "s_waitcnt vmcnt(%1)\n"
      ".Lmore%=:\n\t"
      "s_waitcnt vmcnt(%2)" ::"s"(first), "n"(LESS), "n"(MORE) : "memory", "scc");
}

// Columns of a gated product, so that one lane has the gate's and the other half's results of
// the same outputs.  W = 8 (waves of 64 columns or more): 32 gate columns of a tile and then the
// 32 of the same outputs' other half, eight a lane in each; W = 4: of 32 tile columns 16 gate
// columns and 16 of the other half, four by four.  Tile column c (from the product's first) ->
// its output, and whether it is the gate's (0) or the other half's (1).
template <int W>
__device__ __forceinline__ int gated_output(int c) {
  return W == 8 ? (c >> 6) * 32 + (c & 31) : (c >> 5) * 16 + ((c >> 3) & 3) * 4 + (c & 3);
}
template <int W>
__device__ __forceinline__ int gated_half(int c) {
  return W == 8 ? (c >> 5) & 1 : (c >> 2) & 1;
}

template <int N>
__device__ __forceinline__ void add_bf16(float (&v)[N], const int* w) {
#pragma unroll
  for (int e = 0; e < N; e += 2) {
    v[e] += __uint_as_float((uint32_t)w[e >> 1] << 16);
    v[e + 1] += __uint_as_float((uint32_t)w[e >> 1] & 0xffff0000u);
  }
}

// W neighbouring outputs of a linear layer from column `out` of row `row`, on to d and z: u is the
// product with the bias (gated: the gate's, and up the other half's), c the residual as load_c
// gave it.  Every lane takes part; ok: the place lies within d.
template <bool GATED, int W>
struct LinearOut {
  static_assert(W == 8 || (GATED && W == 4), "outputs a lane");
  typedef int Vec __attribute__((ext_vector_type(W / 2)));
  v4i rsD, rsC, rsZ;
  Activation act;
  int n, has_z;
  __device__ __forceinline__ LinearOut(const Mxfp4LinearParams<GATED>& p) : act(p.act), n(p.n), has_z(p.z != nullptr) {
    const uint32_t bytes = (uint32_t)p.m * (uint32_t)(GATED ? p.n >> 1 : p.n) * 2u;
    rsD = make_buffer_rsrc(p.d, bytes);
    rsC = make_buffer_rsrc(p.c, p.c ? bytes : 0u);   // (none: reads zeros, and no memory)
    rsZ = make_buffer_rsrc(p.z, p.z ? (uint32_t)p.m * (uint32_t)p.n * 2u : 0u);
  }
  static __device__ __forceinline__ Vec pack(const float (&v)[W]) {
    Vec r;
#pragma unroll
    for (int e = 0; e < W; e += 2) r[e >> 1] = (int)pack_bf16x2_rne(v[e], v[e + 1]);
    return r;
  }
  static __device__ __forceinline__ void store(const Vec& v, const v4i& rs, uint32_t off, int soff) {
    // (whole 16 bytes non-temporal: 4096 x 24576 x 1536 130 -> 121 us; with 8 they cost more
    // than they gain)
    if constexpr (W == 8) dg_raw_buffer_store_v4i32(v, rs, (int)off, soff, kStoreNonTemporal);
    else dg_raw_buffer_store_v2i32(v, rs, (int)off, soff, 0);
  }
  __device__ __forceinline__ uint32_t place(int row, int out, bool ok) const {
    return ok ? ((uint32_t)row * (uint32_t)(GATED ? n >> 1 : n) + (uint32_t)out) * 2u : kBufferOutOfRange;
  }
  __device__ __forceinline__ Vec load_c(uint32_t place) const {
    if constexpr (W == 8) return dg_raw_buffer_load_v4i32(rsC, (int)place, 0, 0);
    else return dg_raw_buffer_load_v2i32(rsC, (int)place, 0, 0);
  }
  __device__ __forceinline__ void operator()(int row, int out, bool ok, float (&u)[W], const float (&up)[W], const Vec& c) const {
    if (has_z) {
      const uint32_t oz = ok ? ((uint32_t)row * (uint32_t)n + (uint32_t)out) * 2u : kBufferOutOfRange;
      store(pack(u), rsZ, oz, 0);
      if constexpr (GATED) store(pack(up), rsZ, oz, n);   // (n / 2 columns on)
    }
    activate<W>(u, act);
    if constexpr (GATED) {
#pragma unroll
      for (int e = 0; e < W; ++e) u[e] *= up[e];
    }
    int w[W / 2];
#pragma unroll
    for (int e = 0; e < W / 2; ++e) w[e] = c[e];
    add_bf16(u, w);
    store(pack(u), rsD, place(row, out, ok), 0);
  }
};

// Inclusive sum over the wave's lanes.
__device__ __forceinline__ long long wave_scan(long long v, int lane) {
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const long long u = __shfl_up(v, o, 64);
    if (lane >= o) v += u;
  }
  return v;
}

// The groups' table: ends[g] = tiles of groups 0 .. g, starts[g] = first row (or K block) of
// group g, starts[groups] = the end.  Rows are cut at `limit` (rows, or K blocks), negative
// counts are 0.  One wave builds it.
template <MxKind K>
__device__ __forceinline__ void build_groups(const int32_t* ms, int groups, int limit, int bm, int tiles_m, int tiles_n, int* ends,
                                             int* starts, int lane) {
  long long at = 0, tiles = 0;
  for (int g0 = 0; g0 < groups; g0 += 64) {
    const int g = g0 + lane;
    long long n = g < groups ? max(ms[g], 0) : 0;
    if constexpr (K == MX_KGROUP) n = (n + 127) >> 7;
    const long long end = at + wave_scan(n, lane);
    const int s = (int)min(end - n, (long long)limit), e = (int)min(end, (long long)limit);
    const long long t = K == MX_KGROUP ? (e > s ? (long long)tiles_m * tiles_n : 0) : (long long)((e - s + bm - 1) / bm) * tiles_n;
    const long long tend = tiles + wave_scan(t, lane);
    if (g < groups) {
      starts[g] = s;
      ends[g] = (int)tend;
      if (g == groups - 1) starts[groups] = e;
    }
    at = __shfl(end, 63, 64);
    tiles = __shfl(tend, 63, 64);
  }
}

// The same with a third count, MOST where first is 2.
template <int LESS, int MORE, int MOST>
__device__ __forceinline__ void wait_vmcnt_first(int first) {
  static_assert(LESS <= MORE && MORE <= MOST && MOST < 64, "vmcnt");
  asm volatile(
      "s_cmp_gt_i32 %0, 1\n\t"
      "s_cbranch_scc1 .Lmost%=\n\t"
      "s_cmp_lg_u32 %0, 0\n\t"
      "s_cbranch_scc1 .Lmore%=\n\t"
      "s_waitcnt vmcnt(%1)\n"
      ".Lmore%=:\n\t"
      "s_waitcnt vmcnt(%2)\n"
      ".Lmost%=:\n\t"
      "s_waitcnt vmcnt(%3)" ::"s"(first), "n"(LESS), "n"(MORE), "n"(MOST) : "memory", "scc");
}

// The arguments, all read here: left to where each is first used, the reads wait for one
// another (96 x 24576 x 1536 9.2 us, 9.0 with them together).
__device__ __forceinline__ void read_arguments(const Mxfp4Params& p) {   // (of every kind)
  asm volatile("" ::"s"(p.a), "s"(p.a_sf), "s"(p.b), "s"(p.b_sf), "s"(p.c), "s"(p.d), "s"(p.ws), "s"(p.m), "s"(p.n), "s"(p.k),
               "s"(p.tiles_m), "s"(p.tiles_n), "s"(p.group_m), "s"(p.splits), "s"(p.kb_per_split), "s"(p.full_tiles),
               "s"(p.units));
}

template <typename T, typename P>
__global__ void __launch_bounds__(T::THREADS, 1) mxfp4_tile_kernel(P p) {
  constexpr int MT = T::MT, NT = T::NT, R = T::R;
  constexpr MxKind KIND = P::KIND;
  constexpr bool GROUPED = KIND == MX_RAGGED || KIND == MX_KGROUP;
  constexpr bool LINEAR = KIND == MX_LINEAR || KIND == MX_GATED;
  constexpr int W = KIND == MX_GATED && NT % 4 != 0 ? 4 : 8;   // outputs a lane has side by side
  extern __shared__ __attribute__((aligned(16))) uint8_t smem_all[];
  const int lane = threadIdx.x & 63;
  const int wave_all = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wave = wave_all % T::NW, grp = wave_all / T::NW;   // K group, and the wave in it
  uint8_t* const smem = smem_all + grp * T::RING;
  const int wave_m = wave / T::WN, wave_n = wave % T::WN;
  const int lrow = lane & 15, lgrp = lane >> 4;
  const int M = p.m, N = p.n;
  const uint32_t Kh = (uint32_t)p.k >> 1;   // bytes of an operand row
  const int KB = p.k >> 7;

  int G = gridDim.x;
  read_arguments(p);
  int units = p.units;
  int* const ends = reinterpret_cast<int*>(smem_all + T::LDS);
  if constexpr (GROUPED) {
    int* const starts = ends + p.groups;
    if (wave_all == 0)
      build_groups<KIND>(p.ms, p.groups, KIND == MX_KGROUP ? KB : M, T::BM, p.tiles_m, p.tiles_n, ends, starts, lane);
    __syncthreads();
    units = __builtin_amdgcn_readfirstlane(ends[p.groups - 1]);
    if constexpr (KIND == MX_KGROUP) {
      // D of a group without rows is zero
      const size_t vecs = (size_t)M * N / 8;
      for (int g = 0; g < p.groups; ++g) {
        if (starts[g] != starts[g + 1]) continue;   // (uniform)
        v4i* o = reinterpret_cast<v4i*>(p.d) + (size_t)g * vecs;
        for (size_t i = (size_t)blockIdx.x * T::THREADS + threadIdx.x; i < vecs; i += (size_t)G * T::THREADS) o[i] = v4i{0, 0, 0, 0};
      }
    }
    G = min(G, units);
    if ((int)blockIdx.x >= G) return;
  }
  // Workgroups go round the eight XCDs: one XCD's take units side by side, whose A and B
  // rows its L2 then holds once.
  const int xcd = blockIdx.x & 7;
  const int vb = xcd * (G >> 3) + min(xcd, G & 7) + (int)(blockIdx.x >> 3);
  if (vb >= units) return;

  // the lane, for terms formed where they are used
  auto lane_here = [&]() -> int {
    if constexpr (T::ONE && GROUPED) {
      // (formed anew each time: the builtin's value would be kept, in memory, and its reload
      // waits for every copy in flight)
      int ln;
      asm volatile("v_mbcnt_lo_u32_b32 %0, -1, 0\n\tv_mbcnt_hi_u32_b32 %0, -1, %0" : "=v"(ln));
      return ln;
    }
    return opaque(T::ONE ? (int)__builtin_amdgcn_mbcnt_hi(-1, __builtin_amdgcn_mbcnt_lo(-1, 0)) : lane);
  };

  struct Unit {
    int m0, n0, kb0, nkb, part;
    int g, m_end;   // the group, and the end of its rows
  };
  auto decode = [&](int t) -> Unit {
    Unit w{0, 0, 0, KB, -1, 0, M};
    if constexpr (GROUPED) {
      // the first group that ends past t
      const int ln = lane_here();
      int g = 0;
      for (int c = 0; c < p.groups; c += 64) g += __popcll(__ballot(c + ln < p.groups && ends[c + ln] <= t));
      const int* const starts = ends + p.groups;
      w.g = g = __builtin_amdgcn_readfirstlane(g);
      const int s = __builtin_amdgcn_readfirstlane(starts[g]), e = __builtin_amdgcn_readfirstlane(starts[g + 1]);
      if (g > 0) t -= __builtin_amdgcn_readfirstlane(ends[g - 1]);
      int tm, tn;
      raster_tile(t, KIND == MX_KGROUP ? p.tiles_m : (e - s + T::BM - 1) / T::BM, p.tiles_n, p.group_m, &tm, &tn);
      w.n0 = tn * T::BN;
      w.m0 = tm * T::BM;
      if constexpr (KIND == MX_KGROUP) {
        w.kb0 = s;
        w.nkb = e - s;
      } else {
        w.m0 += s;
        w.m_end = e;
      }
      return w;
    }
    if (t >= p.full_tiles) {
      const int u = t - p.full_tiles;
      w.kb0 = (u % p.splits) * p.kb_per_split;
      w.nkb = min(p.kb_per_split, KB - w.kb0);
      w.part = u;
      t = p.full_tiles + u / p.splits;
    }
    int tm, tn;
    raster_tile(t, p.tiles_m, p.tiles_n, p.group_m, &tm, &tn);
    w.m0 = tm * T::BM;
    w.n0 = tn * T::BN;
    return w;
  };

  const v4i rsA = make_buffer_rsrc(p.a, (uint32_t)M * Kh);
  v4i rsB = make_buffer_rsrc(p.b, (uint32_t)N * Kh);   // (MX_RAGGED: of the cursor's group)
  // The copy cursor: the unit and stage copied next.  Copy j of a wave fills rows
  // 8 (RA wave + j) .. + 7 of the A tile: lane l position l % 8 of row (..) + l / 8,
  // which holds chunk (l % 8) ^ swizzle(row).  Rows past M lie past the buffer and read zeros, and so does the second
  // K block of a stage at an odd end of K: a zero code under a finite scale adds nothing.
  int cu = vb, cs = 0, c_kb = 0, c_nkb = 0;   // unit, stage of this group, its first K block, K blocks of the unit
  uint32_t slot_w = 0;   // the slot copied into next
  uint32_t off[T::LPS];
  // per-lane offset of copy idx within its buffer, from tile row 0's bytes; chunks 4-7
  // (bit 6 of the chunk's offset) are the stage's second K block
  auto chunk_a = [&](int ln, int j) -> uint32_t {
    return (uint32_t)((ln & 7) ^ swz_a((wave * T::RA + j) * 8 + (ln >> 3))) << 4;
  };
  auto chunk_b = [&](int ln, int j) -> uint32_t {
    return (uint32_t)((ln & 7) ^ swz_b((wave * T::RB + j) * 8 + (ln >> 3))) << 4;
  };
  // this wave's scale copy: 1 KB of A's words or of B's
  const int sc = wave % (T::NSA + T::NSB);
  const bool sc_b = sc >= T::NSA;
  v4i rsS = make_buffer_rsrc(sc_b ? p.b_sf : p.a_sf, (uint32_t)KB * (uint32_t)(sc_b ? N : M) * 4u);
  const uint32_t s_stride = (uint32_t)(sc_b ? N : M) * 4u;   // bytes of one K block's words
  const uint32_t s_dst = sc_b ? T::OFF_SB + (sc - T::NSA) * 1024 : T::OFF_SA + sc * 1024;
  // B's row of a gated product's column (N: none)
  auto gated_row = [&](int c) -> int {
    const int out = gated_output<W>(c), half = N >> 1;
    return out < half ? gated_half<W>(c) * half + out : N;
  };
  auto scale_offset = [&](int ln, int m0, int n0, bool odd_end) -> uint32_t {
    const int bt = sc_b ? T::BN : T::BM, rows = sc_b ? N : M, r0 = sc_b ? n0 : m0;
    const int q = (sc_b ? sc - T::NSA : sc) * 256 + ln * 4, half = q / bt;
    int row = r0 + q % bt;
    if (KIND == MX_GATED && sc_b) row = gated_row(row);   // (four rows side by side)
    // (rows past the end, lanes past the two K blocks, a second K block past the end)
    return row < rows && half < (odd_end ? 1 : 2) ? (uint32_t)half * s_stride + (uint32_t)row * 4u : kBufferOutOfRange;
  };
  int c_m0 = 0, c_n0 = 0;
  // The bias of a unit's columns, in their order: a copy ahead of the unit's first stage, so that
  // it has landed with that (and the waits, which do not count it, only wait for more).  The
  // cursor is at most R units ahead of the slowest wave's unit, and one more at its barrier.
  uint32_t bias_w = 0, bias_r = 0;   // the places of the cursor's unit, and of the present one
  auto next_bias = [&](uint32_t at) { return at + T::BIAS_UNIT == T::BIAS ? 0u : at + T::BIAS_UNIT; };
  auto cursor_to = [&](const Unit& w) {
    if constexpr (LINEAR) {
      if (p.bias && wave_all < T::BIAS_COPIES) {
        const int c = w.n0 + wave_all * 128 + 2 * lane_here();
        const int col = KIND == MX_GATED ? gated_row(c) : c;
        buf4_to_lds(make_buffer_rsrc(p.bias, (uint32_t)N * 2u), col < N ? (uint32_t)col * 2u : kBufferOutOfRange, 0u,
                    smem_all + T::LDS + bias_w + wave_all * 256);
      }
      bias_w = next_bias(bias_w);
    }
    c_m0 = w.m0;
    c_n0 = w.n0;
    c_kb = w.kb0 + 2 * grp;
    c_nkb = w.nkb;
    cs = 0;
    const int ln = lane_here();
#pragma unroll
    for (int j = 0; j < T::RA; ++j)
      off[j] = (uint32_t)(w.m0 + (wave * T::RA + j) * 8 + (ln >> 3)) * Kh + chunk_a(ln, j);
#pragma unroll
    for (int j = 0; j < T::RB; ++j) {
      const int row = w.n0 + (wave * T::RB + j) * 8 + (ln >> 3);
      if constexpr (KIND == MX_GATED)
        off[T::RA + j] = (uint32_t)gated_row(row) * Kh + chunk_b(ln, j);
      else
        off[T::RA + j] = (uint32_t)row * Kh + chunk_b(ln, j);
    }
    if constexpr (KIND == MX_RAGGED) {
      rsB = make_buffer_rsrc(p.b + (size_t)w.g * (size_t)N * Kh, (uint32_t)N * Kh);
      if (sc_b) rsS = make_buffer_rsrc(p.b_sf + (size_t)w.g * (size_t)KB * (size_t)N, (uint32_t)KB * (uint32_t)N * 4u);
    }
    // scale words: copy sc of the stage, four words (rows) of one K block per lane
    off[T::RA + T::RB] = scale_offset(ln, w.m0, w.n0, false);
  };
  // the cursor's stage is a unit's last and has one K block only: its second one is
  // out of range (the offsets are formed anew for the next unit)
  auto cursor_odd_end = [&]() {
    const int ln = lane_here();
#pragma unroll
    for (int j = 0; j < T::RA; ++j) off[j] |= (chunk_a(ln, j) & 64u) << 25;
#pragma unroll
    for (int j = 0; j < T::RB; ++j) off[T::RA + j] |= (chunk_b(ln, j) & 64u) << 25;
    off[T::RA + T::RB] = scale_offset(ln, c_m0, c_n0, true);
  };
  // copy idx of a stage: where to in the slot's LDS; per-lane offset o, first K block kb
  auto dst_of = [&](auto idx_tag, uint32_t slot) -> uint32_t {
    constexpr int idx = decltype(idx_tag)::value;
    if constexpr (idx < T::RA) return slot + (wave * T::RA + idx) * 1024;
    else if constexpr (idx < T::RA + T::RB) return slot + T::OFF_B + (wave * T::RB + idx - T::RA) * 1024;
    else return slot + s_dst;
  };
  auto issue_at = [&](auto idx_tag, uint32_t o, int kb, uint32_t dst, const v4i& from_b, const v4i& from_s) {
    constexpr int idx = decltype(idx_tag)::value;
    if constexpr (idx < T::RA) {
      buf16_to_lds(rsA, o, (uint32_t)kb * 64u, smem + dst);
    } else if constexpr (idx < T::RA + T::RB) {
      buf16_to_lds(from_b, o, (uint32_t)kb * 64u, smem + dst);
    } else {
      // (the K block in the lane's offset: a lane's last words may lie past the end, and
      // the range check of each then needs no scalar offset)
      buf16_to_lds(from_s, o == kBufferOutOfRange ? o : o + (uint32_t)kb * s_stride, 0u, smem + dst);
    }
  };
  // copy idx of the cursor's stage
  auto issue = [&](auto idx_tag) {
    issue_at(idx_tag, off[decltype(idx_tag)::value], c_kb, dst_of(idx_tag, slot_w), rsB, rsS);
  };
  // The last LATE copies of a stage are issued in the next one, from these.  A unit's
  // last stage issues them itself, ahead of the stores, so the next unit's first stage
  // has none: where it is no instance of its own, it copies zeros to where nothing is
  // read.
  uint32_t late_off[T::LATE], late_dst[T::LATE];
  int late_kb = 0;
  v4i late_b = rsB, late_s = rsS;   // (MX_RAGGED: the cursor may be in another group by then)
  auto keep_late = [&](int first) {
    static_for<T::LATE>([&](auto i) {
      using Idx = std::integral_constant<int, T::LPS - T::LATE + decltype(i)::value>;
      late_off[decltype(i)::value] = first ? kBufferOutOfRange : off[Idx::value];
      late_dst[decltype(i)::value] = first ? (uint32_t)(T::KG * T::RING - grp * T::RING) : dst_of(Idx{}, slot_w);
    });
    late_kb = first ? 0 : c_kb;
    if constexpr (KIND == MX_RAGGED) {
      late_b = rsB;
      late_s = rsS;
    }
  };
  auto issue_late = [&](auto i_tag) {
    constexpr int i = decltype(i_tag)::value;
    using Idx = std::integral_constant<int, T::LPS - T::LATE + i>;
    if constexpr (KIND == MX_RAGGED) issue_at(Idx{}, late_off[i], late_kb, late_dst[i], late_b, late_s);
    else issue_at(Idx{}, late_off[i], late_kb, late_dst[i], rsB, rsS);
  };
  // nothing more to copy: out of range from here on (the instructions still count), with
  // a scalar offset of 0, so that the range check sees the lane's offset alone
  auto cursor_none = [&]() {
    c_kb = 0;
#pragma unroll
    for (int j = 0; j < T::LPS; ++j) off[j] = kBufferOutOfRange;
  };
  // the cursor's stage st: its second K block may be past the end, or all of it (the
  // last stage of the last K group)
  auto cursor_check = [&]() {
    const int st = cs * T::KG + grp;
    if (2 * st + 1 == c_nkb) cursor_odd_end();
    if (T::KG > 1 && 2 * st >= c_nkb) cursor_none();
  };
  // to the next stage, of the next unit if this one has no more
  auto advance = [&]() {
    slot_w = slot_w + T::STAGE == T::RING ? 0u : slot_w + T::STAGE;
    ++cs;
    c_kb += 2 * T::KG;
    if (2 * cs * T::KG >= c_nkb) {
      if (T::KG == 1 && cu + G < units) {
        cu += G;
        cursor_to(decode(cu));
        cursor_check();
      } else {
        cursor_none();
      }
    } else {
      cursor_check();
    }
  };

  // fragment addresses within a slot; K block 1 of a stage is chunks 4-7
  const uint32_t a_rd = (uint32_t)(wave_m * MT * 16 + lrow) * 128u + (uint32_t)((lgrp ^ swz_a(lrow)) << 4);
  const int brow = (lrow >> 2) * 8 + (lrow & 3);   // (+ 4 in odd column blocks, + 32 per pair: the same swizzle)
  const uint32_t b_rd =
      T::OFF_B + (uint32_t)(wave_n * NT * 16 + brow) * 128u + (uint32_t)((lgrp ^ swz_b(brow)) << 4);
  const uint32_t sa_rd = T::OFF_SA + (uint32_t)(wave_m * MT * 16 + lrow) * 4u;
  const uint32_t sb_rd = T::OFF_SB + (uint32_t)(wave_n * NT * 16 + brow) * 4u;
  const int sh = 8 * lgrp;

  v4i af[2][MT], bf[NT];
  uint32_t sa[2][MT], sb[NT];   // scale words; the byte is taken at use
  // The 256x256 tile's grouped kinds hold more than the dense one, whose registers are all taken:
  // they form the addresses of a stage's K block 1 and of B's scale words (row * 4, from the
  // fragments' row * 128) where they are used.  (With three registers in memory, reloaded in every
  // stage, 16384 rows along K in 8 groups, 4096 x 7168, took 382 us, 335 so.)
  constexpr bool FORM = T::ONE && GROUPED;
  auto sb_at = [&]() {
    return FORM ? ((uint32_t)opaque((int)b_rd) >> 5 & ~3u) + (T::OFF_SB - T::OFF_B / 32) : sb_rd;
  };
  auto of_half = [&](uint32_t x, auto half_tag) -> uint32_t {
    constexpr uint32_t flip = decltype(half_tag)::value * 64u;
    if constexpr (FORM && flip != 0) return (uint32_t)opaque((int)x) ^ flip;
    else return x ^ flip;
  };
  // Reads of K block H of the slot at byte offset rd, in two sets of parts.
  auto read_a = [&](uint32_t rd, auto half_tag, auto mt_tag) {
    constexpr int H = decltype(half_tag)::value, mt = decltype(mt_tag)::value;
    af[H][mt] = *reinterpret_cast<const v4i*>(smem + rd + of_half(a_rd, half_tag) + mt * 2048);
  };
  auto read_sa = [&](uint32_t rd, auto half_tag) {
    constexpr int H = decltype(half_tag)::value;
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
      sa[H][mt] = *reinterpret_cast<const uint32_t*>(smem + rd + sa_rd + H * (T::BM * 4) + mt * 64);
  };
  // what column block nt's registers take over after their last use: its fragment,
  // and after the last of a half of the column blocks that half's scale words
  auto read_b = [&](uint32_t rd, auto half_tag, auto nt_tag) {
    constexpr int H = decltype(half_tag)::value, nt = decltype(nt_tag)::value, NH = NT / 2;
    bf[nt] = *reinterpret_cast<const v4i*>(smem + rd + of_half(b_rd, half_tag) + (nt >> 1) * 4096 + (nt & 1) * 512);
    if constexpr (nt % NH == NH - 1) {
      const uint32_t at = sb_at();
#pragma unroll
      for (int e = nt - NH + 1; e <= nt; ++e)
        sb[e] = *reinterpret_cast<const uint32_t*>(smem + rd + at + H * (T::BN * 4) + (e >> 1) * 128 + (e & 1) * 16);
    }
  };
  using I0 = std::integral_constant<int, 0>;
  using I1 = std::integral_constant<int, 1>;

  // prologue: R stages in flight, the first one's fragments
  cursor_to(decode(cu));
  cursor_check();
  static_for<R>([&](auto r) {
    static_for<T::LPS>([&](auto i) { issue(i); });
    if constexpr (decltype(r)::value + 1 < R) advance();
  });
  wait_vmcnt<T::KG == 1 ? 0 : (R - 1) * T::LPS>();   // (KG 1: the first stage below counts on all of them)
  block_barrier();
  uint32_t rd = 0;
  read_sa(0u, I0{});
  static_for<MT>([&](auto mt) { read_a(0u, I0{}, mt); });
  static_for<NT>([&](auto nt) { read_b(0u, I0{}, nt); });

  v4f acc[MT][NT];
  // One stage.  The first of a unit (FIRST in an instance of its own, first otherwise):
  // the unit before stored D after the copies of the stage waited for here.
  auto stage = [&](auto first_tag, int first) {
    constexpr bool FIRST = decltype(first_tag)::value;
    if constexpr (!FIRST) keep_late(first);
    advance();   // (ahead of the matrix instructions: its branch must not split them)
    const uint32_t nx = rd + T::STAGE == T::RING ? 0u : rd + T::STAGE;
    // first K block: read the second one's fragments
    static_for<NT>([&](auto nt_tag) {
      constexpr int nt = decltype(nt_tag)::value;
      const uint32_t sbv = sb[nt] >> sh;
      static_for<MT>([&](auto mt_tag) {
        constexpr int mt = decltype(mt_tag)::value;
        if constexpr (nt == 0) sa[0][mt] >>= sh;
        acc[mt][nt] = mfma_mxfp4(bf[nt], sbv, af[0][mt], sa[0][mt], acc[mt][nt]);
      });
      read_b(rd, I1{}, nt_tag);
      if constexpr (nt == 0) read_sa(rd, I1{});
      if constexpr (nt < MT) read_a(rd, I1{}, nt_tag);
      if constexpr (nt == NT - 1 && MT > NT)
        static_for<(MT > NT ? MT - NT : 0)>([&](auto e) { read_a(rd, I1{}, std::integral_constant<int, NT + decltype(e)::value>{}); });
      if constexpr (!FIRST && nt < T::LATE) issue_late(nt_tag);
      __builtin_amdgcn_sched_barrier(0);
    });
    // second K block: after BAR column blocks the barrier, then the next stage's
    // fragments and the copies into this slot
    static_for<NT>([&](auto nt_tag) {
      constexpr int nt = decltype(nt_tag)::value;
      const uint32_t sbv = sb[nt] >> sh;
      static_for<MT>([&](auto mt_tag) {
        constexpr int mt = decltype(mt_tag)::value;
        if constexpr (nt == 0) sa[1][mt] >>= sh;
        acc[mt][nt] = mfma_mxfp4(bf[nt], sbv, af[1][mt], sa[1][mt], acc[mt][nt]);
      });
      if constexpr (nt == T::BAR - 1) {
        __builtin_amdgcn_sched_barrier(0);
        wait_lgkmcnt0();
        // (a gated lane's eight outputs come of two such pairs of column blocks)
        constexpr int more = (R - 2) * T::LPS, stores = T::KG > 1 ? 0 : KIND == MX_GATED && W == 8 ? T::NSTORE / 2 : T::NSTORE;
        // (with z, first is 2: its stores are younger than the copies, too)
        constexpr int z_stores = KIND == MX_GATED && W == 8 ? T::NSTORE : T::NSTORE * (KIND == MX_GATED ? 2 : 1);
        if constexpr (T::ONE && LINEAR) wait_vmcnt_first<more, more + T::LATE + stores, more + T::LATE + stores + z_stores>(first);
        else if constexpr (T::ONE) wait_vmcnt_first<more, more + T::LATE + stores>(first);
        else wait_vmcnt<more + (FIRST ? stores : 0)>();
        block_barrier();
        read_sa(nx, I0{});
        static_for<T::BAR>([&](auto e) {
          read_b(nx, I0{}, e);
          if constexpr (decltype(e)::value < MT) read_a(nx, I0{}, e);
        });
      } else if constexpr (nt >= T::BAR) {
        read_b(nx, I0{}, nt_tag);
        if constexpr (nt < MT) read_a(nx, I0{}, nt_tag);
      }
      if constexpr (nt == NT - 1 && MT > NT)
        static_for<(MT > NT ? MT - NT : 0)>([&](auto e) { read_a(nx, I0{}, std::integral_constant<int, NT + decltype(e)::value>{}); });
      if constexpr (nt >= T::BAR - 1) {
        // the copies, spread over the column blocks from the barrier on
        constexpr int parts = NT - T::BAR + 1, q = nt - (T::BAR - 1);
        constexpr int now = T::LPS - T::LATE, lo = now * q / parts, hi = now * (q + 1) / parts;
        static_for<hi - lo>([&](auto e) { issue(std::integral_constant<int, lo + decltype(e)::value>{}); });
      }
      __builtin_amdgcn_sched_barrier(0);
    });
    rd = nx;
  };

  for (int u = vb; u < units; u += G) {
    const Unit cur = decode(u);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = v4f{0.f, 0.f, 0.f, 0.f};

    const int S = ((cur.nkb + 1) / 2 + T::KG - 1) / T::KG;   // stages of this group
    int s = 0, first = 1;
    if constexpr (T::ONE) {
      // (of the unit before: a whole tile with z, or a slice, which has as many stores as z and D)
      if constexpr (LINEAR) first = p.z ? 2 : 1;
      asm volatile("" : "+s"(first));   // (the first stage is not peeled off the loop)
    } else {
      stage(std::true_type{}, 0);
      s = 1;
      first = 0;
    }
#pragma clang loop unroll(disable)
    for (; s < S; ++s) {
      stage(std::false_type{}, first);
      first = 0;
    }
    // The last stage's late copies go out ahead of the stores: the next unit's first wait
    // counts the stores as younger (a store that moved ahead of a copy would let that stage
    // read LDS before the copy has landed).
    keep_late(0);
    static_for<T::LATE>([&](auto i) { issue_late(i); });
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);

    // the pairs of column blocks (mt, np) that this group stores: every KG-th share of them
    auto mine = [&](int mt, int np) {
      if (KIND == MX_GATED && W == 8) return T::KG == 1 || (mt * (NT / 4) + np / 2) % T::KG == grp;
      return T::KG == 1 || (mt * (NT / 2) + np) / (T::NSTORE / T::KG) == grp;
    };
    if constexpr (T::KG > 1) {
      // the groups' sums meet: each hands the others' pairs over in LDS, and adds theirs to
      // its own in order (one unit per workgroup: the rings are done with)
      wait_vmcnt<0>();
      wait_lgkmcnt0();
      block_barrier();
      v4f* xch = reinterpret_cast<v4f*>(smem_all) + wave * 64 + lane;   // [group][MT][NT][wave][lane]
      auto at = [&](int g, int mt, int nt) -> v4f& { return xch[((g * MT + mt) * NT + nt) * (T::NW * 64)]; };
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
          if (!mine(mt, nt >> 1)) at(grp, mt, nt) = acc[mt][nt];
      wait_lgkmcnt0();
      block_barrier();
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (!mine(mt, nt >> 1)) continue;
#pragma unroll
          for (int g = 1; g < T::KG; ++g) acc[mt][nt] += at((grp + g) % T::KG, mt, nt);
        }
    }
    const int ln = T::ONE ? lane_here() : lane;
    if (LINEAR && cur.part >= 0) bias_r = next_bias(bias_r);
    if (cur.part >= 0) {
      // fp32 partial tile of this slice: ws[part][BM][BN]
      const v4i rsW = make_buffer_rsrc(p.ws + (size_t)cur.part * (T::BM * T::BN), (uint32_t)(T::BM * T::BN * 4));
      const int at = ((wave_m * MT * 16 + (ln & 15)) * T::BN + wave_n * NT * 16 + (ln >> 4) * 8) * 4;
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          if (!mine(mt, nt >> 1)) continue;
          const v4i w = {__float_as_int(acc[mt][nt][0]), __float_as_int(acc[mt][nt][1]),
                         __float_as_int(acc[mt][nt][2]), __float_as_int(acc[mt][nt][3])};
          dg_raw_buffer_store_v4i32(w, rsW, at, (mt * 16 * T::BN + (nt >> 1) * 32 + (nt & 1) * 4) * 4, 0);
        }
    } else if constexpr (LINEAR) {
      const LinearOut<KIND == MX_GATED, W> out(p);
      using Vec = typename LinearOut<KIND == MX_GATED, W>::Vec;
      // items of a lane's W outputs, their residual read PRE items ahead (a load behind a store is
      // waited for with it; the 256x256 tile has registers for four, gated for two: with four, seven
      // others were in memory, and their reloads waited for the stores)
      constexpr int ITEMS = KIND == MX_GATED && W == 8 ? NT / 4 : NT / 2, STEP = NT / 2 / ITEMS;
      const int c0 = wave_n * NT * 16 + (ln >> 4) * 8;   // the tile's column of item 0
      auto column = [&](int i) { return KIND == MX_GATED ? gated_output<W>(cur.n0 + c0 + i * STEP * 32) : cur.n0 + c0 + i * 32; };
      auto row_of = [&](int mt) { return cur.m0 + wave_m * MT * 16 + mt * 16 + (ln & 15); };
      const int cols = KIND == MX_GATED ? N >> 1 : N;
      constexpr int ALL = MT * ITEMS, PRE = T::ONE && KIND == MX_GATED ? 2 : ALL < 4 ? ALL : 4;
      Vec cv[PRE];
      auto read_c = [&](auto item_tag) {
        constexpr int mt = decltype(item_tag)::value / ITEMS, i = decltype(item_tag)::value % ITEMS;
        if (mine(mt, i * STEP))
          cv[decltype(item_tag)::value % PRE] = out.load_c(out.place(row_of(mt), column(i), row_of(mt) < M && column(i) < cols));
      };
      static_for<PRE>([&](auto f) { read_c(f); });
      const uint8_t* const bias = smem_all + T::LDS + bias_r + c0 * 2;
      static_for<ALL>([&](auto item_tag) {
        constexpr int f = decltype(item_tag)::value, mt = f / ITEMS, i = f % ITEMS;
        const int row = row_of(mt);
        if (mine(mt, i * STEP)) {
          auto product = [&](int np) {
            struct { float v[8]; } r;
            const v4f lo = acc[mt][2 * np], hi = acc[mt][2 * np + 1];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              r.v[e] = lo[e];
              r.v[4 + e] = hi[e];
            }
            if (p.bias) {   // (uniform)
              const v4i b = *reinterpret_cast<const v4i*>(bias + np * 64);
              const int w[4] = {b.x, b.y, b.z, b.w};
              add_bf16(r.v, w);
            }
            return r;
          };
          auto first = product(i * STEP);
          float u[W], up[W];
#pragma unroll
          for (int e = 0; e < W; ++e) u[e] = up[e] = first.v[e];
          if constexpr (KIND == MX_GATED) {
            const auto other = STEP == 2 ? product(i * STEP + 1) : first;
#pragma unroll
            for (int e = 0; e < W; ++e) up[e] = other.v[W == 8 ? e : 4 + e];
          }
          out(row, column(i), row < M && column(i) < cols, u, up, cv[f % PRE]);
        }
        if constexpr (f + PRE < ALL) read_c(std::integral_constant<int, f + PRE>{});
      });
      bias_r = next_bias(bias_r);
    } else {
      const v4i rsD = make_buffer_rsrc(p.d + (KIND == MX_KGROUP ? (size_t)cur.g * M * N : 0), (uint32_t)M * (uint32_t)N * 2u);
      const v4i rsC = make_buffer_rsrc(p.c, p.c ? (uint32_t)M * (uint32_t)N * 2u : 0u);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int row = cur.m0 + wave_m * MT * 16 + mt * 16 + (ln & 15);
#pragma unroll
        for (int np = 0; np < NT / 2; ++np) {
          if (!mine(mt, np)) continue;
          const int col = cur.n0 + wave_n * NT * 16 + np * 32 + (ln >> 4) * 8;
          const uint32_t off = row < (KIND == MX_RAGGED ? cur.m_end : M) && col < N ? ((uint32_t)row * (uint32_t)N + (uint32_t)col) * 2u : kBufferOutOfRange;
          v4f lo = acc[mt][2 * np], hi = acc[mt][2 * np + 1];
          if (!GROUPED && p.c) {
            const v4i cv = dg_raw_buffer_load_v4i32(rsC, (int)off, 0, 0);
            const uint32_t cw[4] = {(uint32_t)cv.x, (uint32_t)cv.y, (uint32_t)cv.z, (uint32_t)cv.w};
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              lo[2 * e] += __uint_as_float(cw[e] << 16);
              lo[2 * e + 1] += __uint_as_float(cw[e] & 0xffff0000u);
              hi[2 * e] += __uint_as_float(cw[2 + e] << 16);
              hi[2 * e + 1] += __uint_as_float(cw[2 + e] & 0xffff0000u);
            }
          }
          const v4i w = {(int)pack_bf16x2_rne(lo[0], lo[1]), (int)pack_bf16x2_rne(lo[2], lo[3]),
                         (int)pack_bf16x2_rne(hi[0], hi[1]), (int)pack_bf16x2_rne(hi[2], hi[3])};
          dg_raw_buffer_store_v4i32(w, rsD, (int)off, 0, 0);
        }
      }
    }
  }
  wait_vmcnt<0>();   // the copies past the last stage: LDS is not given back before they have landed
}

// ---------------------------------------------------------------------------
// Few rows (decode): the product streams B once, bound by how much of it is in
// flight, and by the launch.  A workgroup takes 16 columns and all rows of A (MT blocks
// of 16); its four waves split K between them, pair of K blocks by pair (a 128-byte
// line of each row), with fragments and scale words loaded straight into registers, P
// pairs ahead.  The waves' sums meet in LDS, added in wave order, so no second launch
// and no workspace is needed.  (1 x 4096 x 7168: 6.1 us, 2.7 of them the launch, at 4.6
// TB/s of B in between; 32 x 4096 x 7168 8.3-8.5 us, 32 x 1024 x 8192 8.5-9, on 64 workgroups; eight waves and 32 columns measured 4-40 % slower.)
// ---------------------------------------------------------------------------
extern "C" __device__ int dg_raw_buffer_load_i32_mx(v4i rsrc, int voffset, int soffset,
                                                    int aux) __asm("llvm.amdgcn.raw.buffer.load.i32");

constexpr int MX_SKINNY_WAVES = 4;

// The same for a linear layer: v holds four columns of a row; a gated one's halves lie in
// lanes 32 apart, which take part together.
__device__ __forceinline__ void add_bf16x4(v4f& v, const uint16_t* t) {
  const uint2 w = *reinterpret_cast<const uint2*>(t);
  v[0] += __uint_as_float(w.x << 16);
  v[1] += __uint_as_float(w.x & 0xffff0000u);
  v[2] += __uint_as_float(w.y << 16);
  v[3] += __uint_as_float(w.y & 0xffff0000u);
}
template <bool GATED>
__device__ __forceinline__ void skinny_linear_out(const Mxfp4LinearParams<GATED>& p, v4f v, int row, int n0, int lgrp) {
  const int half = p.n >> 1;
  const int col = GATED ? (lgrp >> 1) * half + (n0 >> 1) + (lgrp & 1) * 4 : n0 + 4 * lgrp;
  if (p.bias) add_bf16x4(v, p.bias + col);
  if (p.z) *reinterpret_cast<uint2*>(p.z + (size_t)row * p.n + col) = uint2{pack_bf16x2_rne(v[0], v[1]), pack_bf16x2_rne(v[2], v[3])};
  float a[4] = {v[0], v[1], v[2], v[3]};
  activate<4>(a, p.act);
  if constexpr (GATED) {
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] *= __shfl_xor(v[e], 32, 64);
    if (lgrp >= 2) return;
  }
  v = v4f{a[0], a[1], a[2], a[3]};
  const size_t at = (size_t)row * (GATED ? half : p.n) + col;
  if (p.c) add_bf16x4(v, p.c + at);
  *reinterpret_cast<uint2*>(p.d + at) = uint2{pack_bf16x2_rne(v[0], v[1]), pack_bf16x2_rne(v[2], v[3])};
}

template <int MT, int P, typename Params>
__global__ void __launch_bounds__(MX_SKINNY_WAVES * 64) mxfp4_skinny_kernel(Params p) {
  constexpr MxKind KIND = Params::KIND;
  constexpr int NW = MX_SKINNY_WAVES;
  __shared__ v4f red[NW][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lrow = lane & 15, lgrp = lane >> 4, sh = 8 * lgrp;
  const int M = p.m, N = p.n;
  const uint32_t Kh = (uint32_t)p.k >> 1;
  const int KB = p.k >> 7, PAIRS = (KB + 1) >> 1;
  const int n0 = blockIdx.x * 16;   // (N % 16 == 0: every column is there)
  const v4i rsA = make_buffer_rsrc(p.a, (uint32_t)M * Kh);
  const v4i rsB = make_buffer_rsrc(p.b, (uint32_t)N * Kh);
  const v4i rsSA = make_buffer_rsrc(p.a_sf, (uint32_t)KB * (uint32_t)M * 4u);
  const v4i rsSB = make_buffer_rsrc(p.b_sf, (uint32_t)KB * (uint32_t)N * 4u);
  // per-lane offsets; a row past the end reads zeros (and its results are not stored)
  uint32_t a_off[MT], sa_off[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) {
    const int r = i * 16 + lrow;
    a_off[i] = r < M ? (uint32_t)r * Kh + (uint32_t)lgrp * 16u : kBufferOutOfRange;
    sa_off[i] = r < M ? (uint32_t)r * 4u : kBufferOutOfRange;
  }
  // (gated: the gate's eight rows, and then the other half's of the same outputs)
  const int b_row = KIND == MX_GATED ? (lrow >> 3) * (N >> 1) + (n0 >> 1) + (lrow & 7) : n0 + lrow;
  const uint32_t b_off = (uint32_t)b_row * Kh + (uint32_t)lgrp * 16u, sb_off = (uint32_t)b_row * 4u;
  v4i af[P][2][MT], bf[P][2];
  uint32_t sa[P][2][MT], sb[P][2];
  // pair j of this wave (pair j NW + wave of K); K blocks past the end read zeros
  auto load = [&](int j, auto set_tag) {
    constexpr int S = decltype(set_tag)::value;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int kb = (j * NW + wave) * 2 + h;
      const bool in = kb < KB;
      const int ko = in ? kb * 64 : 0;
      const uint32_t none = in ? 0u : kBufferOutOfRange;
      bf[S][h] = dg_raw_buffer_load_v4i32(rsB, (int)(b_off | none), ko, 0);
      sb[S][h] = (uint32_t)dg_raw_buffer_load_i32_mx(rsSB, (int)(sb_off | none), in ? kb * N * 4 : 0, 0);
#pragma unroll
      for (int i = 0; i < MT; ++i) {
        af[S][h][i] = dg_raw_buffer_load_v4i32(rsA, (int)(a_off[i] | none), ko, 0);
        sa[S][h][i] = (uint32_t)dg_raw_buffer_load_i32_mx(rsSA, (int)(sa_off[i] | none), in ? kb * M * 4 : 0, 0);
      }
    }
  };
  v4f acc[MT];
#pragma unroll
  for (int i = 0; i < MT; ++i) acc[i] = v4f{0.f, 0.f, 0.f, 0.f};
  const int mine = (PAIRS - wave + NW - 1) / NW;   // (0 for a wave past the last pair)
  static_for<P>([&](auto s) { load(decltype(s)::value, s); });
  for (int j = 0; j < mine; j += P) {
    static_for<P>([&](auto s) {
      constexpr int S = decltype(s)::value;
#pragma unroll
      for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
          acc[mt] = mfma_mxfp4(bf[S][h], sb[S][h] >> sh, af[S][h][mt], sa[S][h][mt] >> sh, acc[mt]);
      load(j + P + S, s);
    });
  }
#pragma unroll
  for (int mt = 0; mt < MT; ++mt) {
    if (mt > 0) __syncthreads();
    red[wave][lane] = acc[mt];
    __syncthreads();
    const int row = mt * 16 + lrow;
    if (wave == 0 && row < M) {
      v4f v = red[0][lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) v += red[w][lane];
      if constexpr (KIND == MX_LINEAR || KIND == MX_GATED) {
        skinny_linear_out(p, v, row, n0, lgrp);
        continue;
      }
      const size_t at = (size_t)row * N + n0 + 4 * lgrp;
      if (p.c) {
        const uint2 cv = *reinterpret_cast<const uint2*>(p.c + at);
        v[0] += __uint_as_float(cv.x << 16);
        v[1] += __uint_as_float(cv.x & 0xffff0000u);
        v[2] += __uint_as_float(cv.y << 16);
        v[3] += __uint_as_float(cv.y & 0xffff0000u);
      }
      *reinterpret_cast<uint2*>(p.d + at) = uint2{pack_bf16x2_rne(v[0], v[1]), pack_bf16x2_rne(v[2], v[3])};
    }
  }
}

// Groups of one call, and the bytes of their table (ends and starts) in LDS behind a tile's
// ring; not every ring leaves room for the table of many.
constexpr int kMaxGroups = 1024, kLdsBytes = 160 * 1024;
inline size_t group_table_bytes(int groups) { return (size_t)(2 * groups + 1) * 4; }

// id, MT, NT, WM, WN, ring slots, K groups
#define DG_MXFP4_TILES(X) \
  X(0, 4, 8, 4, 2, 2, 1)  \
  X(1, 4, 4, 2, 4, 3, 1)  \
  X(2, 2, 4, 4, 2, 4, 1)  \
  X(3, 2, 2, 2, 4, 6, 1)  \
  X(4, 2, 4, 2, 2, 3, 2)  \
  X(5, 3, 4, 2, 2, 2, 2)  \
  X(6, 2, 2, 2, 2, 4, 2)  \
  X(7, 4, 4, 2, 2, 2, 2)
// and of the grouped kinds alone (whose rounds it fills better: mxfp4_grouped.hip)
#define DG_MXFP4_GROUPED_TILES(X) X(8, 3, 8, 4, 2, 2, 1)

// Raises kernel f's limit of dynamic LDS on the current device, once for each (done: their bits).
static hipError_t allow_lds(const void* f, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  const hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = 1ull << (dev & 63);   // (the entry points refuse device 64 and beyond)
  if (done.load(std::memory_order_relaxed) & bit) return hipSuccess;
  const hipError_t set = hipFuncSetAttribute(f, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (set == hipSuccess) done.fetch_or(bit, std::memory_order_relaxed);
  return set;
}

template <typename P>
static hipError_t launch_mxfp4_tile(const P& p, int id, int grid, hipStream_t stream, size_t table_bytes = 0) {
  switch (id) {
#define X(i, MT, NT, WM, WN, R, KG)                                                                               \
  case i: {                                                                                                       \
    using T = MxTile<MT, NT, WM, WN, R, KG>;                                                                      \
    static std::atomic<uint64_t> allowed{0};                                                                      \
    const hipError_t attr =                                                                                       \
        allow_lds(reinterpret_cast<const void*>(&mxfp4_tile_kernel<T, P>),                                        \
                  P::KIND >= MX_RAGGED ? kLdsBytes : P::KIND == MX_DENSE ? T::LDS : T::LDS + T::BIAS, allowed);   \
    if (attr != hipSuccess) return attr;                                                                          \
    const size_t lds = T::LDS + (P::KIND == MX_LINEAR || P::KIND == MX_GATED ? T::BIAS : table_bytes);           \
    hipLaunchKernelGGL((mxfp4_tile_kernel<T, P>), dim3(grid), dim3(T::THREADS), lds, stream, p);                  \
    return hipGetLastError();                                                                                     \
  }
    DG_MXFP4_TILES(X)
  default:
    if constexpr (P::KIND >= MX_RAGGED) {
      switch (id) { DG_MXFP4_GROUPED_TILES(X) }
    }
#undef X
  }
  return hipErrorInvalidValue;
}

// id, MT, pairs in flight per wave
#define DG_MXFP4_SKINNY(X) \
  X(0, 1, 4)               \
  X(1, 2, 4)

template <typename Params>
static hipError_t launch_mxfp4_skinny(const Params& p, int id, hipStream_t stream) {
  switch (id) {
#define X(i, MT, P)                                                                                                       \
  case i:                                                                                                                 \
    hipLaunchKernelGGL((mxfp4_skinny_kernel<MT, P, Params>), dim3(p.n / 16), dim3(MX_SKINNY_WAVES * 64), 0, stream, p); \
    return hipGetLastError();
    DG_MXFP4_SKINNY(X)
#undef X
  }
  return hipErrorInvalidValue;
}

struct Mxfp4Plan {
  int skinny, tile, tiles_m, tiles_n, splits, kb_per_split, full_tiles, units, grid;
  size_t ws_bytes;
};

Mxfp4Plan plan_mxfp4(int m, int n, int k, int cus);
bool mxfp4_sizes_fit(int m, int n, int k);
void log_mxfp4_plan(const char* call, int m, int n, int k, const Mxfp4Plan& pl);   // (with DG_LOG=1)
struct Mxfp4TileInfo {
  int bm, bn, kg, lds;
  bool narrow;   // its waves have fewer than 64 columns
};
Mxfp4TileInfo mxfp4_tile_info(int id);
constexpr int kMxTileCount = 8, kMxGroupedTileCount = 9, kMxSkinnyIdBase = 100;
int mxfp4_forced();   // the kernel that DG_FORCE_MXFP4 pins (kMxSkinnyIdBase and up: a streaming one), or -1
// Estimated microseconds of `units` whole tiles of kb K blocks each.
double mxfp4_tile_time(int id, long long units, int kb, int cus);

}  // namespace dg
