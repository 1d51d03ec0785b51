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
  float* ws;
  int m, n, k;
  int tiles_m, tiles_n, group_m;
  int splits, kb_per_split;   // K slices of a split tile, K blocks per slice (even)
  int full_tiles;             // tiles [0, full_tiles) run whole, the others are split
  int units;                  // whole tiles and slices
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

// The arguments, all read here: left to where each is first used, the reads wait for one
// another (96 x 24576 x 1536 9.2 us, 9.0 with them together).
__device__ __forceinline__ void read_arguments(const Mxfp4Params& p) {
  asm volatile("" ::"s"(p.a), "s"(p.a_sf), "s"(p.b), "s"(p.b_sf), "s"(p.c), "s"(p.d), "s"(p.ws), "s"(p.m), "s"(p.n), "s"(p.k),
               "s"(p.tiles_m), "s"(p.tiles_n), "s"(p.group_m), "s"(p.splits), "s"(p.kb_per_split), "s"(p.full_tiles),
               "s"(p.units));
}

template <typename T>
__global__ void __launch_bounds__(T::THREADS, 1) mxfp4_tile_kernel(Mxfp4Params p) {
  constexpr int MT = T::MT, NT = T::NT, R = T::R;
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

  const int G = gridDim.x;
  read_arguments(p);
  // Workgroups go round the eight XCDs: one XCD's take units side by side, whose A and B
  // rows its L2 then holds once.
  const int xcd = blockIdx.x & 7;
  const int vb = xcd * (G >> 3) + min(xcd, G & 7) + (int)(blockIdx.x >> 3);
  if (vb >= p.units) return;

  // the lane, for terms formed where they are used
  auto lane_here = [&]() -> int {
    return opaque(T::ONE ? (int)__builtin_amdgcn_mbcnt_hi(-1, __builtin_amdgcn_mbcnt_lo(-1, 0)) : lane);
  };

  struct Unit {
    int m0, n0, kb0, nkb, part;
  };
  auto decode = [&](int t) -> Unit {
    Unit w{0, 0, 0, KB, -1};
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
  const v4i rsB = make_buffer_rsrc(p.b, (uint32_t)N * Kh);
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
  const v4i rsS = make_buffer_rsrc(sc_b ? p.b_sf : p.a_sf, (uint32_t)KB * (uint32_t)(sc_b ? N : M) * 4u);
  const uint32_t s_stride = (uint32_t)(sc_b ? N : M) * 4u;   // bytes of one K block's words
  const uint32_t s_dst = sc_b ? T::OFF_SB + (sc - T::NSA) * 1024 : T::OFF_SA + sc * 1024;
  auto scale_offset = [&](int ln, int m0, int n0, bool odd_end) -> uint32_t {
    const int bt = sc_b ? T::BN : T::BM, rows = sc_b ? N : M, r0 = sc_b ? n0 : m0;
    const int q = (sc_b ? sc - T::NSA : sc) * 256 + ln * 4, half = q / bt, row = r0 + q % bt;
    // (rows past the end, lanes past the two K blocks, a second K block past the end)
    return row < rows && half < (odd_end ? 1 : 2) ? (uint32_t)half * s_stride + (uint32_t)row * 4u : kBufferOutOfRange;
  };
  int c_m0 = 0, c_n0 = 0;
  auto cursor_to = [&](const Unit& w) {
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
    for (int j = 0; j < T::RB; ++j)
      off[T::RA + j] = (uint32_t)(w.n0 + (wave * T::RB + j) * 8 + (ln >> 3)) * Kh + chunk_b(ln, j);
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
  auto issue_at = [&](auto idx_tag, uint32_t o, int kb, uint32_t dst) {
    constexpr int idx = decltype(idx_tag)::value;
    if constexpr (idx < T::RA) {
      buf16_to_lds(rsA, o, (uint32_t)kb * 64u, smem + dst);
    } else if constexpr (idx < T::RA + T::RB) {
      buf16_to_lds(rsB, o, (uint32_t)kb * 64u, smem + dst);
    } else {
      // (the K block in the lane's offset: a lane's last words may lie past the end, and
      // the range check of each then needs no scalar offset)
      buf16_to_lds(rsS, o == kBufferOutOfRange ? o : o + (uint32_t)kb * s_stride, 0u, smem + dst);
    }
  };
  // copy idx of the cursor's stage
  auto issue = [&](auto idx_tag) { issue_at(idx_tag, off[decltype(idx_tag)::value], c_kb, dst_of(idx_tag, slot_w)); };
  // The last LATE copies of a stage are issued in the next one, from these.  A unit's
  // last stage issues them itself, ahead of the stores, so the next unit's first stage
  // has none: where it is no instance of its own, it copies zeros to where nothing is
  // read.
  uint32_t late_off[T::LATE], late_dst[T::LATE];
  int late_kb = 0;
  auto keep_late = [&](int first) {
    static_for<T::LATE>([&](auto i) {
      using Idx = std::integral_constant<int, T::LPS - T::LATE + decltype(i)::value>;
      late_off[decltype(i)::value] = first ? kBufferOutOfRange : off[Idx::value];
      late_dst[decltype(i)::value] = first ? (uint32_t)(T::KG * T::RING - grp * T::RING) : dst_of(Idx{}, slot_w);
    });
    late_kb = first ? 0 : c_kb;
  };
  auto issue_late = [&](auto i_tag) {
    constexpr int i = decltype(i_tag)::value;
    issue_at(std::integral_constant<int, T::LPS - T::LATE + i>{}, late_off[i], late_kb, late_dst[i]);
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
      if (T::KG == 1 && cu + G < p.units) {
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
  // Reads of K block H of the slot at byte offset rd, in two sets of parts.
  auto read_a = [&](uint32_t rd, auto half_tag, auto mt_tag) {
    constexpr int H = decltype(half_tag)::value, mt = decltype(mt_tag)::value;
    af[H][mt] = *reinterpret_cast<const v4i*>(smem + rd + (a_rd ^ (H * 64u)) + mt * 2048);
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
    bf[nt] = *reinterpret_cast<const v4i*>(smem + rd + (b_rd ^ (H * 64u)) + (nt >> 1) * 4096 + (nt & 1) * 512);
    if constexpr (nt % NH == NH - 1) {
#pragma unroll
      for (int e = nt - NH + 1; e <= nt; ++e)
        sb[e] = *reinterpret_cast<const uint32_t*>(smem + rd + sb_rd + H * (T::BN * 4) + (e >> 1) * 128 + (e & 1) * 16);
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
        constexpr int more = (R - 2) * T::LPS, stores = T::KG == 1 ? T::NSTORE : 0;
        if constexpr (T::ONE) wait_vmcnt_first<more, more + T::LATE + stores>(first);
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

  for (int u = vb; u < p.units; u += G) {
    const Unit cur = decode(u);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) acc[mt][nt] = v4f{0.f, 0.f, 0.f, 0.f};

    const int S = ((cur.nkb + 1) / 2 + T::KG - 1) / T::KG;   // stages of this group
    int s = 0, first = 1;
    if constexpr (T::ONE) {
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
    auto mine = [&](int mt, int np) { return T::KG == 1 || (mt * (NT / 2) + np) / (T::NSTORE / T::KG) == grp; };
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
    } else {
      const v4i rsD = make_buffer_rsrc(p.d, (uint32_t)M * (uint32_t)N * 2u);
      const v4i rsC = make_buffer_rsrc(p.c, p.c ? (uint32_t)M * (uint32_t)N * 2u : 0u);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt) {
        const int row = cur.m0 + wave_m * MT * 16 + mt * 16 + (ln & 15);
#pragma unroll
        for (int np = 0; np < NT / 2; ++np) {
          if (!mine(mt, np)) continue;
          const int col = cur.n0 + wave_n * NT * 16 + np * 32 + (ln >> 4) * 8;
          const uint32_t off = row < M && col < N ? ((uint32_t)row * (uint32_t)N + (uint32_t)col) * 2u : kBufferOutOfRange;
          v4f lo = acc[mt][2 * np], hi = acc[mt][2 * np + 1];
          if (p.c) {
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

struct Mxfp4TileInfo {
  int bm, bn, kg;
};
static const Mxfp4TileInfo kMxTiles[] = {
#define X(id, MT, NT, WM, WN, R, KG) {MxTile<MT, NT, WM, WN, R, KG>::BM, MxTile<MT, NT, WM, WN, R, KG>::BN, KG},
    DG_MXFP4_TILES(X)
#undef X
};

static hipError_t launch_mxfp4_tile(const Mxfp4Params& p, int id, int grid, hipStream_t stream) {
  switch (id) {
#define X(i, MT, NT, WM, WN, R, KG)                                                                      \
  case i: {                                                                                              \
    using T = MxTile<MT, NT, WM, WN, R, KG>;                                                             \
    static const hipError_t attr = hipFuncSetAttribute(reinterpret_cast<const void*>(&mxfp4_tile_kernel<T>), \
                                                       hipFuncAttributeMaxDynamicSharedMemorySize, T::LDS);  \
    if (attr != hipSuccess) return attr;                                                                 \
    hipLaunchKernelGGL(mxfp4_tile_kernel<T>, dim3(grid), dim3(T::THREADS), T::LDS, stream, p);           \
    return hipGetLastError();                                                                            \
  }
    DG_MXFP4_TILES(X)
#undef X
  }
  return hipErrorInvalidValue;
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
template <int MT, int P>
__global__ void __launch_bounds__(MX_SKINNY_WAVES * 64) mxfp4_skinny_kernel(Mxfp4Params p) {
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
  const uint32_t b_off = (uint32_t)(n0 + lrow) * Kh + (uint32_t)lgrp * 16u, sb_off = (uint32_t)(n0 + lrow) * 4u;
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

// id, MT, pairs in flight per wave
#define DG_MXFP4_SKINNY(X) \
  X(0, 1, 4)               \
  X(1, 2, 4)
constexpr int kMxSkinnyIdBase = 100;   // in DG_FORCE_MXFP4

static int skinny_rows(int id) {
  switch (id) {
#define X(i, MT, P) case i: return MT * 16;
    DG_MXFP4_SKINNY(X)
#undef X
  }
  return 0;
}

static hipError_t launch_mxfp4_skinny(const Mxfp4Params& p, int id, hipStream_t stream) {
  switch (id) {
#define X(i, MT, P)                                                                                       \
  case i:                                                                                                 \
    hipLaunchKernelGGL((mxfp4_skinny_kernel<MT, P>), dim3(p.n / 16), dim3(MX_SKINNY_WAVES * 64), 0, stream, p); \
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

// Up to 32 rows: the streaming kernel reads all of A once per 16 columns, so it is taken
// while row blocks x columns stay small (measured against the best tile: 1 x 4096 x 7168
// 6.0 against 9.7 us, 16 x 7168 x 2048 5.9 / 5.7, 32 x 4096 x 7168 8.5 / 9.9; past the
// limit 1 x 24576 x 1536 10.7 / 7.5, 32 x 7168 x 16384 28.8 / 19.7).  Otherwise the tile
// with the least estimated time in microseconds: rounds of units, each its stages at the
// tile's pace and a fixed share (pipeline fill, D); a split plan's partials' round trip
// and second launch; and the rate at which the units' CUs stream B.  The constants fit
// 247 shapes, M 1 to 8192, 512 x 2048 to 32768 x 512 and 7168 x 16384 (geometric mean
// 0.2 % over the best tile of each; worst 64 x 7168 x 16384, 18 %).
static Mxfp4Plan plan_mxfp4(int m, int n, int k, int cus) {
  constexpr double kStage[] = {1.85, 1.12, 0.76, 0.69, 0.57, 0.81, 0.52, 1.05};
  constexpr double kUnit[] = {4.5, 2.0, 1.0, 1.0, 1.8, 1.9, 1.6, 2.5};
  constexpr double kSplit = 5.7, kPartialRate = 3.6e6, kStreamRate = 40.0e3;   // us, bytes per us
  constexpr int kTiles = (int)(sizeof(kMxTiles) / sizeof(kMxTiles[0]));
  int force = -1;
  if (const char* f = std::getenv("DG_FORCE_MXFP4")) force = std::atoi(f);   // pins the kernel (for tuning)
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
  for (int id = 0; id < kTiles; ++id) {
    const int kg = kMxTiles[id].kg;
    const Mxfp4Plan pl = plan_mxfp4_tile(m, n, k, cus, id);
    if (kg > 1 && pl.units > cus) continue;   // one unit per workgroup (a pinned one is passed over, too)
    const int whole = ((k / 128 + 1) / 2 + kg - 1) / kg;
    double t = (double)((pl.full_tiles + cus - 1) / cus) * (whole * kStage[id] + kUnit[id]);
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

static bool mxfp4_sizes_fit(int m, int n, int k) {
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
    if (const char* log = std::getenv("DG_LOG"); log && log[0] == '1') {
      if (pl.skinny >= 0)
        std::fprintf(stderr, "[dg] mxfp4_gemm_nt m=%d n=%d k=%d -> streaming kernel, %d rows\n", m, n, k, skinny_rows(pl.skinny));
      else
        std::fprintf(stderr, "[dg] mxfp4_gemm_nt m=%d n=%d k=%d -> tile %dx%d, %d K group%s, %d tiles (%d whole, the rest x %d K slices), "
                     "%d workgroups, workspace %zu bytes\n", m, n, k, kMxTiles[pl.tile].bm, kMxTiles[pl.tile].bn,
                     kMxTiles[pl.tile].kg, kMxTiles[pl.tile].kg > 1 ? "s" : "", pl.tiles_m * pl.tiles_n, pl.full_tiles, pl.splits, pl.grid, pl.ws_bytes);
    }
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
