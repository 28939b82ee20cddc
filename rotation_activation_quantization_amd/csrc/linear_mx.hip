// The product of MXFP4 operands,
//
//   out[t][k] = sum_j x[t][j] w[k][j] + b[k],
//
// on v_mfma_scale_f32_16x16x128_f8f6f4, which multiplies the codes and applies
// both blocks' scales; the sum is binary32.  The weights are the MFMA's A
// operand and the tokens its B operand, so that a lane's four results are
// consecutive output channels of one token.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>
#include <utility>

#include "internal.h"
#include "mx_ops.h"
#include "row_ops.h"
#include "wave_ops.h"

namespace signrot {
namespace {

typedef __attribute__((__vector_size__(8 * sizeof(int32_t)))) int32_t i32x8_t;
typedef __attribute__((__vector_size__(4 * sizeof(int32_t)))) int32_t i32x4_t;
using wave::f32x4_t;

constexpr int kCus = 256;  // of an MI355X: the plans do not depend on the device asked
constexpr int kFp4 = 4;    // format number of E2M1 in the MFMA

template <int N, class F>
__device__ __forceinline__ void unrolled(F&& f) {
  [&]<int... I>(std::integer_sequence<int, I...>) { (f(std::integral_constant<int, I>{}), ...); }
  (std::make_integer_sequence<int, N>{});
}

// OA, OB: the byte of sa and sb that holds the lane's block scales.  The
// operand's upper four registers are not read for four-bit formats.
template <int OA, int OB>
__device__ __forceinline__ f32x4_t mfma(const i32x4_t& a, const i32x4_t& b, const f32x4_t& c, uint32_t sa,
                                        uint32_t sb) {
  const i32x8_t wa = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, wb = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, wb, c, kFp4, kFp4, OA, static_cast<int>(sa), OB,
                                                          static_cast<int>(sb));
}

// acc += a b in place, for the tiles: left to itself the compiler gives results
// and sums registers of their own, which a tile that takes nearly all of them
// does not have, and moves them about.  The leading s_nop covers a VALU write of an
// operand just before.  The reader of a sum has to wait for the last one (settle).
template <int OA, int OB>
__device__ __forceinline__ void mfma_to(f32x4_t& acc, const i32x4_t& a, const i32x4_t& b, uint32_t sa, uint32_t sb) {
  asm volatile("s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%6,0] "
               "op_sel_hi:[%7,%8,0] cbsz:4 blgp:4"
               : "+v"(acc)
               : "v"(a), "v"(b), "v"(sa), "v"(sb), "n"(OA & 1), "n"(OB & 1), "n"(OA >> 1), "n"(OB >> 1));
}
// Waits for the sums and hands them on, so that no reader, nor a move of them, comes before.
template <int FK, int FT>
__device__ __forceinline__ void settle(f32x4_t (&acc)[FK][FT]) {
  asm volatile("s_nop 15\n\ts_nop 15" ::: "memory");
#pragma unroll
  for (int f = 0; f < FK; ++f)
#pragma unroll
    for (int j = 0; j < FT; ++j) asm volatile("" : "+v"(acc[f][j]));
}

// Four results of token t from channel k on: a vector at whatever address it has,
// single ones at the row's end.
__device__ __forceinline__ void store_results(const MxArgs& a, int t, int k, const float (&o)[4]) {
  const int64_t at = static_cast<int64_t>(t) * a.ldo + k;
  const bool whole = k + 4 <= a.R;
  if (whole && a.out_bf16) {
    row::store_as<false>(static_cast<uint16_t*>(a.out) + at,
                         wave::u32x2_t{row::pack_bf16(o[0], o[1]), row::pack_bf16(o[2], o[3])});
  } else if (whole) {
    row::store_as<false>(static_cast<float*>(a.out) + at, f32x4_t{o[0], o[1], o[2], o[3]});
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (k + e < a.R) row::store_elem(a.out, at + e, o[e], a.out_bf16);
  }
}

// ---- tiles --------------------------------------------------------------------
//
// Tile p of the order -> (token tile, channel tile): token tiles fastest over
// groups of eight, so that neighbours share a few panels of tokens and weights
// in an L2.
__device__ __forceinline__ void tile_at(int p, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int kGroup = 8;
  const int per_group = kGroup * tiles_n;
  const int group = p / per_group;
  const int first = group * kGroup;
  const int gm = min(tiles_m - first, kGroup);
  const int r = p - group * per_group;
  tm = first + r % gm;
  tn = r / gm;
}

constexpr int kDeep = 64;               // bytes of a row that one MFMA takes: four blocks
constexpr int kStage = 2 * kDeep;       // of a stage: a whole 128-byte line
constexpr int kQuadBytes = 2 * kStage;  // of a quad, the depths whose scales are handled together

// Channel of a 64-channel group in slot 16 f + i.
__device__ __forceinline__ int channel_of(int f, int i) { return 32 * (f >> 1) + 8 * (i >> 2) + 4 * (f & 1) + (i & 3); }

// The words of scales of four 16-row groups, depth s (lane (s, i): d[f] of row
// 16 f + i), as those of the MFMA: o[b] for lane (b, i) of that depth.
__device__ __forceinline__ void turned_words(const uint32_t (&d)[4], uint32_t (&o)[4]) {
  const uint32_t a0 = __builtin_amdgcn_perm(d[1], d[0], 0x05010400u), a1 = __builtin_amdgcn_perm(d[1], d[0], 0x07030602u);
  const uint32_t b0 = __builtin_amdgcn_perm(d[3], d[2], 0x05010400u), b1 = __builtin_amdgcn_perm(d[3], d[2], 0x07030602u);
  o[0] = __builtin_amdgcn_perm(b0, a0, 0x05040100u);
  o[1] = __builtin_amdgcn_perm(b0, a0, 0x07060302u);
  o[2] = __builtin_amdgcn_perm(b1, a1, 0x05040100u);
  o[3] = __builtin_amdgcn_perm(b1, a1, 0x07060302u);
}

// WK x WT waves of FK x FT 16 x 16 results each, a ring of S stages of two
// MFMAs' depth.
template <int WK, int WT, int FK, int FT, int S>
struct Tile {
  static constexpr int kWaves = WK * WT;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kBN = 16 * WK * FK;  // channels
  static constexpr int kBM = 16 * WT * FT;  // tokens
  // LDS bytes of a stage, and its 1 KiB loads per wave
  static constexpr int kWStage = kBN * kStage, kTStage = kBM * kStage;
  static constexpr int kWLoads = kWStage / 1024 / kWaves, kTLoads = kTStage / 1024 / kWaves;
  static constexpr int kLoads = kWLoads + kTLoads;
  static constexpr int kPart = 256 * FK * FT * kWaves;  // floats of a tile's partial sums
  // scales: groups of 64 rows (weights, then tokens), a word of four rows' for
  // each lane and depth
  static constexpr int kGroupsW = kBN / 64, kGroups = (kBN + kBM) / 64;
  static constexpr int kScales = kGroups * 4 * 256;
  static constexpr int kPer = kGroups > kWaves ? kGroups / kWaves : 1;  // groups that a wave lays out
  static constexpr int kRing = S * (kWStage + kTStage);
  static constexpr int kLds = kRing + 2 * kScales + 2048 * kWaves;  // and a unit of results for each wave
  // work-groups to a CU: as many as its LDS holds, at most eight waves
  static constexpr int kFit = 160 * 1024 / kLds < 8 / kWaves ? 160 * 1024 / kLds : 8 / kWaves;
  static_assert(kWLoads * kWaves * 1024 == kWStage && kTLoads * kWaves * 1024 == kTStage, "whole loads per wave");
  static_assert(FK % 4 == 0 && kBM % 64 == 0, "rows come in groups of 64");
  static_assert(S == 2 || S == 4, "ring");
  static_assert(FT % 4 == 0 || 4 % FT == 0, "a wave's tokens lie in whole words of scales or in one");
  static_assert(kGroups <= kWaves || kPer * kWaves == kGroups, "whole groups of scales per wave");
  static_assert(kGroupsW % kPer == 0, "a wave's groups are of one operand");
  static_assert(kFit > 0, "LDS");
};

// Both operands stream global -> LDS (16 bytes a lane, no registers), a whole
// 128-byte line of a row at a time, through a ring of S stages of two MFMA
// depths.  A depth is FK blocks of FT MFMAs, one block for each of the wave's
// 16-row groups of weights; operands are read two blocks (weights) or a depth
// (tokens) ahead.  One barrier a stage, before its last two blocks: by then
// every wave has read all of the stage, whose place the loads of stage s + S may
// take, and stage s + 1 has landed (the wait before the barrier), so that its
// first operands are read in the last two blocks.
//
// A work-group takes the tiles p, p + stride, ... below `end`, and the ring
// runs on from tile to tile: the last stages of a tile load the first ones of
// the next, which arrive while its results are stored.  With two stages the second
// stage's loads all go out before the stores, so that the wait in the next tile's
// first stage can leave the stores on their way (8192 x 4096 x 4096 71.2 us, 72.9
// with the wait for them).
//
// What bounds a large product: 8192 x 4096 x 14336 takes 230 to 250 us (3.9 to 4.2
// PFLOP/s), the tiles 215 of them in a loop over the same operands.  There the matrix
// units are busy 60 % of the cycles (8192 x 14336 x 4096: 65 %) at 1.8 GHz, on all zeros
// for as many cycles at 2.2 GHz, 176 us: the power that real operands take costs a fifth.
// The other 40 % of the cycles are the tiles' own.  LDS serves reads and writes by index in
// 30 % of them, the L2s deliver 21 bytes a cycle and CU, and a wave waits 38 % of its time;
// none of that is full, but in every tile a quad's time follows the bytes staged, 22 to 25
// ns a KiB, more than its products.  A tile's start and stores cost what two quads do.
// Alone, on values in registers, the instruction reaches 7.0 PFLOP/s of random codes and
// 9.3 of zeros.  Four waves of 128 x 128 (a third fewer LDS reads) were slower, as were
// stores past the caches and staggered starts.
//
// A row is cut into quads of four depths (512 channels, two stages).  Quad 0 of
// a tile is the row's last, possibly short one.  Its chunks beyond n are read
// from the quad's first chunk, and the scales of both operands there are
// 2^-127: the products, below 2^-248, are zero in binary32.
//
// LDS rows of 128 bytes, eight 16-byte chunks: logical chunk c of row r sits at
// physical chunk c ^ ((r >> 1) & 7), so that the sixteen lanes a
// 16-byte read serves at a time cover the 64 banks once.  A lane (g = lane / 16,
// i = lane % 16) reads row i, chunk 4 u + g of a 16-row group: block g of depth
// u for both operands.
//
// Slot 16 f + i of a 64-channel group holds channel 32 (f / 2) + 8 (i / 4) +
// 4 (f % 2) + i % 4: two 16 x 16 results then leave a lane eight consecutive
// channels of a token.
//
// Scales.  An MFMA takes a lane's scale from one byte of a register, the byte
// fixed in the instruction, so a word for lane (g, i) holds block g of the rows
// i of four 16-row groups f: one 4-byte LDS read serves four operands.  A row's
// scales of a quad are sixteen bytes.  For each quad a wave takes the scales of
// 64 rows into registers (lane (s, i): the word of depth s of rows 16 f + i, so
// that a cache line is touched once for four depths) with the quad's first
// loads, and before a barrier whose wait has seen them arrive turns the four by
// four bytes with eight permutes and writes them to LDS.  That work is a tenth of a
// large product's time (8192 x 28672 x 4096 436 us, 392 without); so for the
// largest tiles (ORDERED) a kernel of its own turns all scales once, into
// 1 KiB for 64 rows and a quad, which a wave loads straight to LDS.
__device__ __forceinline__ int swizzle_of(int r) { return (r >> 1) & 7; }

template <int WK, int WT, int FK, int FT, int S, bool SPLIT, bool ORDERED>
__device__ __forceinline__ void mx_tile(const MxArgs& a, int tiles_m, int tiles_n, int splits) {
  using C = Tile<WK, WT, FK, FT, S>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds];
  uint8_t* const lds_w = lds;
  uint8_t* const lds_t = lds + S * C::kWStage;
  uint8_t* const lds_s = lds + C::kRing;
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wid % WK, wt = wid / WK;
  const int g = lane >> 4, i = lane & 15;

  // Item p is part p / tiles of tile p % tiles.  Consecutive block ids go to
  // different XCDs: each XCD takes one contiguous range of the items, its
  // work-groups (gridDim / 8 of them) the items of that range in turn.  A grid
  // that is not a multiple of eight is one item each.
  const int tiles = tiles_m * tiles_n;
  int p, end, stride;
  {
    const int items = tiles * splits;
    const int q = items >> 3, rem = items & 7;
    const int x = blockIdx.x & 7;
    const int start = x < rem ? x * (q + 1) : rem * (q + 1) + (x - rem) * q;
    p = start + (blockIdx.x >> 3);
    end = start + q + (x < rem ? 1 : 0);
    stride = (gridDim.x & 7) ? items : gridDim.x >> 3;
  }
  const int bytes = a.n / 2;  // of a row
  const int blocks = a.n / mx::kBlock;
  const int quads = (bytes + kQuadBytes - 1) / kQuadBytes;
  // part j of a row: quads first(j) .. first(j + 1) - 1
  auto first = [&](int j) { return static_cast<int>(static_cast<int64_t>(quads) * j / splits); };

  // What is loaded next: quad lq of item src_p.  Rows beyond the tensor are
  // clamped (their results are not stored).  Load l of a wave fills eight rows.
  const int row8 = lane >> 3;
  // (an opaque copy of the lane where its constants are used once a quad or less, so
  // that they are formed there and not kept in registers)
  auto lane_here = [&]() {
    int here = lane;
    asm volatile("" : "+v"(here));
    return here;
  };
  int src_p = p, lq, lq_end;
  const uint8_t *base_w, *base_t, *base_s;
  int rows_w, rows_t;
  uint32_t size_w, size_t_;
  uint32_t off_w[C::kWLoads], off_t[C::kTLoads];  // of the lane's rows
  uint32_t off_s[C::kPer][4];                     // of its rows of scales
  // byte of the lane's chunk in a stage: rows 8 (k wave + l) + lane / 8
  auto chunk_of = [&](int lines) { return 16 * ((lane & 7) ^ swizzle_of(8 * lines + row8)); };
  // This wave's first group of 64 rows of scales (waves beyond the groups repeat the last).
  const int group = min(C::kPer * wid, C::kGroups - 1);
  const bool of_w = group < C::kGroupsW;
  auto set_source = [&]() {
    const int row8 = lane_here() >> 3;
    const int part = SPLIT ? src_p / tiles : 0;
    lq = __builtin_amdgcn_readfirstlane(first(part));
    lq_end = __builtin_amdgcn_readfirstlane(first(part + 1));
    int tm, tn;
    tile_at(src_p - part * tiles, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * C::kBM, n0 = tn * C::kBN;
    rows_w = min(C::kBN, a.R - n0);
    rows_t = min(C::kBM, a.T - m0);
    base_w = a.w + static_cast<int64_t>(n0) * a.ldw;
    base_t = a.a + static_cast<int64_t>(m0) * a.lda;
    size_w = static_cast<uint32_t>(rows_w - 1) * static_cast<uint32_t>(a.ldw) + bytes;
    size_t_ = static_cast<uint32_t>(rows_t - 1) * static_cast<uint32_t>(a.lda) + bytes;
    if (ORDERED)
      base_s = of_w ? a.w_scale + 1024 * static_cast<int64_t>(quads) * (n0 / 64 + group)
                    : a.scale + 1024 * static_cast<int64_t>(quads) * (m0 / 64 + group - C::kGroupsW);
    else
      base_s = of_w ? a.w_scale + static_cast<int64_t>(n0) * a.ldws : a.scale + static_cast<int64_t>(m0) * a.lds;
#pragma unroll
    for (int l = 0; l < C::kWLoads; ++l) {
      const int slot = 8 * (C::kWLoads * wid + l) + row8;
      const int ch = (slot & ~63) + channel_of((slot >> 4) & 3, slot & 15);
      off_w[l] = static_cast<uint32_t>(min(ch, rows_w - 1)) * static_cast<uint32_t>(a.ldw);
    }
#pragma unroll
    for (int l = 0; l < C::kTLoads; ++l) {
      const int r = 8 * (C::kTLoads * wid + l) + row8;
      off_t[l] = static_cast<uint32_t>(min(r, rows_t - 1)) * static_cast<uint32_t>(a.lda);
    }
    if (ORDERED) return;
    const int i = lane_here() & 15;
#pragma unroll
    for (int x = 0; x < C::kPer; ++x)
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int r = 64 * (group + x - (of_w ? 0 : C::kGroupsW)) + (of_w ? channel_of(f, i) : 16 * f + i);
        off_s[x][f] =
            static_cast<uint32_t>(min(r, (of_w ? rows_w : rows_t) - 1)) * static_cast<uint32_t>(of_w ? a.ldws : a.lds);
      }
  };
  int at_quad;  // its first byte in a row
  int left;     // bytes of it
  auto place = [&]() {
    at_quad = __builtin_amdgcn_readfirstlane(kQuadBytes * (lq == 0 ? quads - 1 : lq - 1));
    left = __builtin_amdgcn_readfirstlane(min(bytes - at_quad, kQuadBytes));
  };
  // Past the last item the loads go on with that item's: every stage issues the
  // same number, so the vmcnt thresholds are exact.
  auto advance = [&]() {
    lq = __builtin_amdgcn_readfirstlane(lq + 1);
    if (lq == lq_end) {
      src_p = src_p + stride < end ? src_p + stride : src_p;
      set_source();
    }
    place();
  };
  // The lane's chunk sits in an even or an odd line of eight rows: two values.
  const int chunk_even = chunk_of(0), chunk_odd = chunk_of(1);
  // load l of stage j of the quad, into ring position `to`
  auto issue = [&](int l, int j, int to) {
    const bool w = l < C::kWLoads;
    const int k = w ? l : l - C::kWLoads;
    const int line = (w ? C::kWLoads : C::kTLoads) * wid + k;
    const int chunk = ((w ? C::kWLoads : C::kTLoads) % 2 == 0 ? k : line) % 2 == 0 ? chunk_even : chunk_odd;
    const uint32_t in = (w ? off_w[k] : off_t[k]) + (chunk < left - kStage * j ? chunk + kStage * j : 0);
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        w ? wave::buffer_rsrc(base_w, size_w) : wave::buffer_rsrc(base_t, size_t_),
        (__attribute__((address_space(3))) void*)((w ? lds_w + C::kWStage * to : lds_t + C::kTStage * to) + 1024 * line),
        16, in, at_quad, 0, 0);
  };

  // The scales of the quad, words s = g of the rows; those beyond n read the quad's first.
  // Words at any address: a row's last one ends at its end, shifted into place later
  // (rows of fewer than four blocks start on words).  Laying them out on words first
  // took 3.3 us of the 11.1 of 613 x 1120 x 777.
  typedef uint32_t any_u32_t __attribute__((aligned(1)));
  uint32_t raw[C::kPer][4], raw_shift = 0;
  int raw_left = 0;
  auto load_scales = [&](int half) {
    if (ORDERED) {
#pragma unroll
      for (int x = 0; x < C::kPer; ++x)
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            wave::buffer_rsrc(base_s + 1024 * static_cast<int64_t>(quads) * x, 1024u * static_cast<uint32_t>(quads)),
            (__attribute__((address_space(3))) void*)(lds_s + half * C::kScales + 1024 * (group + x)), 16, 16 * lane,
            1024 / kQuadBytes * at_quad, 0, 0);
      return;
    }
    raw_left = left / mx::kBlockBytes;
    const int word = at_quad / mx::kBlockBytes + (4 * g < raw_left ? 4 * g : 0);
    const int from = min(word, max(blocks - 4, 0));
    raw_shift = 8 * (word - from);
#pragma unroll
    for (int x = 0; x < C::kPer; ++x)
#pragma unroll
      for (int f = 0; f < 4; ++f)
        raw[x][f] = *reinterpret_cast<const any_u32_t*>(base_s + (off_s[x][f] + static_cast<uint32_t>(from)));
  };
  auto turn_scales = [&](int half) {
    uint32_t* const turned = reinterpret_cast<uint32_t*>(lds_s + 1024 * group + 256 * g) + i;
#pragma unroll
    for (int x = 0; x < C::kPer; ++x) {
      uint32_t d[4], o[4];
#pragma unroll
      for (int f = 0; f < 4; ++f) d[f] = raw[x][f] >> raw_shift;
      turned_words(d, o);
#pragma unroll
      for (int b = 0; b < 4; ++b)
        turned[half * (C::kScales / 4) + 256 * x + 16 * b] = 4 * g + b < raw_left ? o[b] : 0;
    }
  };

  // the lane's bytes in a 16-row group: depth 0; depth 1 is chunk ^ 4
  const int read = i * kStage + 16 * (g ^ swizzle_of(i));
  const int read_w = 16 * wk * FK * kStage + read, read_t = 16 * wt * FT * kStage + read;
  auto weight = [&](int pos, int u, int f) {
    return *reinterpret_cast<const i32x4_t*>(lds_w + C::kWStage * pos + 16 * kStage * f + (read_w ^ (64 * u)));
  };
  auto token = [&](int pos, int u, int j) {
    return *reinterpret_cast<const i32x4_t*>(lds_t + C::kTStage * pos + 16 * kStage * j + (read_t ^ (64 * u)));
  };
  // scales of a depth: a word for four of the wave's 16-row groups
  constexpr int kSW = FK / 4, kST = FT >= 4 ? FT / 4 : 1;
  const int scale_w = 1024 * (wk * FK / 4) + 4 * lane;
  const int scale_t = 1024 * (C::kGroupsW + wt * FT / 4) + 4 * lane;
  const int shift_t = FT >= 4 ? 0 : 8 * (wt * FT % 4);  // a wave with fewer than four: its bytes lowest
  uint32_t sw[2][kSW], st[2][kST];                      // of this and the next depth
  auto read_scales = [&](int to, int half, int e) {
#pragma unroll
    for (int q = 0; q < kSW; ++q)
      sw[to][q] = *reinterpret_cast<const uint32_t*>(lds_s + half * C::kScales + scale_w + 1024 * q + 256 * e);
#pragma unroll
    for (int q = 0; q < kST; ++q)
      st[to][q] = *reinterpret_cast<const uint32_t*>(lds_s + half * C::kScales + scale_t + 1024 * q + 256 * e) >> shift_t;
  };

  f32x4_t acc[FK][FT];
  i32x4_t tok[2][FT];  // token operands of this and the next depth
  i32x4_t wf[FK + 2];

  // Loads of a stage: the first kLate after the barrier that frees its place, in
  // that stage's last two blocks, the others in the next stage's first blocks.
  constexpr int kLate = C::kLoads / 2, kEarly = C::kLoads - kLate;
  static_assert(kEarly <= 2 * FK - 2, "a load a block before the barrier");
  static_assert(!ORDERED || S == 2, "loaded to LDS in the stage before their quad");

  constexpr int kScaleLoads = (ORDERED ? 1 : 4) * C::kPer;
  set_source();
  place();
  load_scales(0);
#pragma unroll
  for (int s = 0; s < S; ++s) {
    if (s == 2) {
      advance();
      wave::wait_vmcnt<2 * C::kLoads>();
      __builtin_amdgcn_sched_barrier(0);
      turn_scales(0);
      load_scales(1);
    }
#pragma unroll
    for (int l = 0; l < (S > 2 && s == S - 1 ? kLate : C::kLoads); ++l) issue(l, s % 2, s);
  }
  if (S == 2 && !ORDERED) {
    wave::wait_vmcnt<2 * C::kLoads>();
    __builtin_amdgcn_sched_barrier(0);
    turn_scales(0);
  }
  wave::wait_vmcnt<S == 2 ? C::kLoads : 2 * C::kLoads + kLate + kScaleLoads>();
  wave::lds_barrier();
  wf[0] = weight(0, 0, 0);
  wf[1] = weight(0, 0, 1);
#pragma unroll
  for (int j = 0; j < FT; ++j) tok[0][j] = token(0, 0, j);
  read_scales(0, 0, 0);

  // Stores that the results of the tile before have on their way behind the loads of
  // the first stage (S = 2), when their number is certain.
  int stored = 0;
  constexpr int kStores = FK * FT / 2;  // of bf16 results; binary32: twice as many

  // Stage j of a quad at ring position pos; fresh: a tile's first with S = 2, before
  // which all loads of the next have been issued.
  auto stage = [&](auto J, bool fresh, int pos, int half) {
    constexpr int j = decltype(J)::value;
    const int next = (pos + 1) % S, before = (pos + S - 1) % S;
    unrolled<2>([&](auto UC) {
      constexpr int u = decltype(UC)::value;
      i32x4_t(&now)[FT] = tok[u];
      i32x4_t(&then)[FT] = tok[u ^ 1];
      unrolled<FK>([&](auto F) {
        constexpr int f = decltype(F)::value, b = u * FK + f;
        if constexpr (b == 2 * FK - 2) {
          // S = 2: the next stage's loads have landed, S = 4: those of the two after it
          // may be in flight, with the scales that one of them began with.  The
          // scales loaded two (S = 2: one) stages ago go to LDS.
          constexpr bool turn = !ORDERED && j == (S == 2 ? 1 : 0);
          if (S == 2 && j == 0 && fresh && stored == kStores)
            wave::wait_vmcnt<kStores>();
          else if (S == 2 && j == 0 && fresh && stored == 2 * kStores)
            wave::wait_vmcnt<2 * kStores>();
          else
            wave::wait_vmcnt<(S - 2) * C::kLoads + (S == 4 && j == 1 ? kScaleLoads : 0)>();
          __builtin_amdgcn_sched_barrier(0);
          if (turn) turn_scales(half ^ 1);
          wave::lds_barrier();
          __builtin_amdgcn_sched_barrier(0);
          if (j == 0) {
            advance();
            load_scales(half ^ 1);
          }
        }
        // The reads follow the block's first MFMA: the wait before that one is
        // then for reads a whole block old.
        mfma_to<f % 4, 0>(acc[f][0], wf[f], now[0], sw[u][f / 4], st[u][0]);
        __builtin_amdgcn_sched_barrier(0);
        wf[f + 2] = f + 2 < FK ? weight(pos, u, f + 2) : weight(u == 0 ? pos : next, u ^ 1, f + 2 - FK);
        if (u == 0) {
#pragma unroll
          for (int t = f * FT / FK; t < (f + 1) * FT / FK; ++t) then[t] = token(pos, 1, t);
          if (f == FK - 1) read_scales(1, half, 2 * j + 1);
        } else if (f >= FK - 2) {
#pragma unroll
          for (int t = (f - FK + 2) * FT / 2; t < (f - FK + 3) * FT / 2; ++t) then[t] = token(next, 0, t);
          if (f == FK - 1) read_scales(0, half ^ j, 2 * (j ^ 1));
        }
        if constexpr (b < kEarly) {
          if (S != 2 || j == 1 || !fresh) issue(kLate + b, j ^ 1, before);
        }
        if (b >= 2 * FK - 2) {
#pragma unroll
          for (int l = (b - 2 * FK + 2) * kLate / 2; l < (b - 2 * FK + 3) * kLate / 2; ++l) issue(l, j, pos);
        }
        unrolled<FT - 1>([&](auto T) {
          constexpr int t = decltype(T)::value + 1;
          mfma_to<f % 4, t % 4>(acc[f][t], wf[f], now[t], sw[u][f / 4], st[u][t / 4]);
        });
        __builtin_amdgcn_sched_barrier(0);
      });
      wf[0] = wf[FK];
      wf[1] = wf[FK + 1];
    });
  };

  int pos = 0, half = 0;
  for (; p < end; p += stride) {
    int tm, tn;
    tile_at(SPLIT ? p % tiles : p, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * C::kBM, n0 = tn * C::kBN;
#pragma unroll
    for (int f = 0; f < FK; ++f)
#pragma unroll
      for (int j = 0; j < FT; ++j) acc[f][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    const int part = SPLIT ? p / tiles : 0;
    const int count = first(part + 1) - first(part);
#pragma clang loop unroll(disable)
    for (int q = 0; q < count; ++q) {
      unrolled<2>([&](auto J) { stage(J, q == 0, (S == 2 ? 0 : pos) + J, half); });
      if (S != 2) pos ^= 2;
      half ^= 1;
    }
    if (S == 2) {
      // the rest of the next tile's second stage, before the stores that its first
      // need not wait for
#pragma unroll
      for (int l = kLate; l < C::kLoads; ++l) issue(l, 1, 1);
    }

    settle(acc);
    if (SPLIT) {
      // partial sums in operand order, [part][tile][wave][f][j][lane]
      f32x4_t* const out = reinterpret_cast<f32x4_t*>(a.workspace) +
                           (static_cast<int64_t>(p) * C::kPart + 256 * FK * FT * wid) / 4 + lane;
#pragma unroll
      for (int f = 0; f < FK; ++f)
#pragma unroll
        for (int j = 0; j < FT; ++j) out[64 * (FT * f + j)] = acc[f][j];
      continue;
    }

    // Lane (g, i): token 16 j + i, channels 8 g .. 8 g + 7 of every 32.  Stored from
    // there, neighbouring lanes would write sixteen rows, 16 bytes a request; so
    // sixteen rows of 128 bytes at a time, a unit, go through 2 KiB of LDS of the
    // wave's own and leave as whole lines.  Chunk c of row r sits at chunk
    // c ^ ((r >> 1) & 7): the sixteen lanes that an access serves at a time cover the
    // banks once.  A wave's LDS accesses are done in order, so the next unit is
    // written as soon as the reads of this one are on their way.
    uint8_t* const mine = lds + C::kRing + 2 * C::kScales + 2048 * wid;
    const int lane = lane_here(), g = lane >> 4, i = lane & 15;
    auto chunk_at = [&](int r, int c) {
      return reinterpret_cast<wave::u32x4_t*>(mine + 128 * r + 16 * (c ^ ((r >> 1) & 7)));
    };
    const int t_wave = m0 + 16 * wt * FT, k_wave = n0 + 16 * wk * FK;
    float bias[FK / 4][16];
#pragma unroll
    for (int q = 0; q < FK / 4; ++q)
#pragma unroll
      for (int e = 0; e < 16; ++e) bias[q][e] = 0.f;
    if (a.bias) {
#pragma unroll
      for (int q = 0; q < FK / 4; ++q)
#pragma unroll
        for (int e = 0; e < 16; ++e)
          bias[q][e] = a.bias[min(k_wave + 64 * q + 32 * (e >> 3) + 8 * g + (e & 7), a.R - 1)];
      wave::wait_vmcnt<0>();  // here, or the compiler waits for it, and all stores, in the next tile
    }
    auto results = [&](auto BF16, auto WHOLE) {
      constexpr int per = BF16 ? 8 : 4;    // results of a chunk
      constexpr int parts = BF16 ? 1 : 2;  // units of 64 channels
      constexpr int units = FK / 4 * FT * parts;
      auto put = [&](auto U) {
        constexpr int u = decltype(U)::value, part = u % parts, j = u / parts % FT, q = u / parts / FT;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          wave::u32x4_t v;
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            if constexpr (BF16)
              v[e] = row::pack_bf16(
                  acc[4 * q + 2 * h + (e >> 1)][j][2 * (e & 1)] + bias[q][8 * h + 2 * e],
                  acc[4 * q + 2 * h + (e >> 1)][j][2 * (e & 1) + 1] + bias[q][8 * h + 2 * e + 1]);
            else
              v[e] = __float_as_uint(acc[4 * q + 2 * part + h][j][e] +
                                     bias[q][8 * part + 4 * h + e]);
          }
          *chunk_at(i, BF16 ? 4 * h + g : 2 * g + h) = v;
        }
      };
      const int r0 = lane >> 3, c = lane & 7;
      uint8_t* const to = static_cast<uint8_t*>(a.out) +
                          (static_cast<int64_t>(t_wave + r0) * a.ldo + k_wave + per * c) * (16 / per);
      wave::u32x4_t got[2][2];
      auto send = [&](auto U) {
        constexpr int u = decltype(U)::value, part = u % parts, j = u / parts % FT, q = u / parts / FT;
        const int k = k_wave + 64 * q + 32 * part + per * c;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const int t = t_wave + 16 * j + 8 * h + r0;
          uint8_t* const at = to + (static_cast<int64_t>(16 * j + 8 * h) * a.ldo + 64 * q + 32 * part) * (16 / per);
          const wave::u32x4_t v = got[u & 1][h];
          if (WHOLE || (t < a.T && k + per <= a.R)) {
            row::store_as<false>(at, v);
          } else if (t < a.T) {
#pragma unroll
            for (int e = 0; e < per; ++e) {
              if (k + e >= a.R) continue;
              if constexpr (BF16)
                reinterpret_cast<uint16_t*>(at)[e] = static_cast<uint16_t>(v[e >> 1] >> (16 * (e & 1)));
              else
                reinterpret_cast<uint32_t*>(at)[e] = v[e];
            }
          }
        }
      };
      unrolled<units>([&](auto U) {
        constexpr int u = decltype(U)::value;
        put(U);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int h = 0; h < 2; ++h) got[u & 1][h] = *chunk_at(8 * h + r0, c);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if constexpr (u > 0) send(std::integral_constant<int, u - 1>{});
      });
      send(std::integral_constant<int, units - 1>{});
    };
    const bool whole = m0 + C::kBM <= a.T && n0 + C::kBN <= a.R;
    stored = !whole ? 0 : a.out_bf16 ? kStores : 2 * kStores;
    if (a.out_bf16 && whole)
      results(std::true_type{}, std::true_type{});
    else if (a.out_bf16)
      results(std::true_type{}, std::false_type{});
    else if (whole)
      results(std::false_type{}, std::true_type{});
    else
      results(std::false_type{}, std::false_type{});
  }
  wave::wait_vmcnt<0>();
}

// Scales of all 64-row groups of tokens and weights in the order that the tiles
// read them, [group][quad][depth][lane]: a wave takes a group and a quad.  Blocks
// beyond n get 2^-127.
struct Order {
  const uint8_t* src[2];  // tokens, weights
  int64_t ld[2];
  uint8_t* dst[2];
  int rows[2], groups[2];
  int blocks, quads;
  int words;  // 1: rows of aligned words
};
__global__ __launch_bounds__(256) void mx_order_kernel(Order o) {
  const int lane = threadIdx.x & 63, s = lane >> 4, i = lane & 15;
  const int q = 4 * static_cast<int>(blockIdx.x) + static_cast<int>(threadIdx.x >> 6);
  if (q >= o.quads) return;
  const int total = o.groups[0] + o.groups[1];
  for (int g = blockIdx.y; g < total; g += gridDim.y) {
    const int of_w = g >= o.groups[0];
    const int group = of_w ? g - o.groups[0] : g;
    const int at = 16 * q + 4 * s;
    uint32_t d[4], t[4];
#pragma unroll
    for (int f = 0; f < 4; ++f) {
      const int r = min(64 * group + (of_w ? channel_of(f, i) : 16 * f + i), o.rows[of_w] - 1);
      const uint8_t* const p = o.src[of_w] + r * o.ld[of_w] + at;
      d[f] = 0;
      if (o.words) {
        if (at < o.blocks) d[f] = *reinterpret_cast<const uint32_t*>(p);
      } else {
#pragma unroll
        for (int b = 0; b < 4; ++b)
          if (at + b < o.blocks) d[f] |= static_cast<uint32_t>(p[b]) << (8 * b);
      }
    }
    turned_words(d, t);
    uint32_t* const to = reinterpret_cast<uint32_t*>(o.dst[of_w] + 1024 * (static_cast<int64_t>(group) * o.quads + q)) +
                         64 * s + i;
#pragma unroll
    for (int b = 0; b < 4; ++b) to[16 * b] = at + b < o.blocks ? t[b] : 0;
  }
}

template <int WK, int WT, int FK, int FT, int S, bool SPLIT, bool ORDERED>
__global__ __launch_bounds__(64 * WK * WT) __attribute__((
    amdgpu_waves_per_eu(Tile<WK, WT, FK, FT, S>::kWaves * Tile<WK, WT, FK, FT, S>::kFit / 4)))
void mx_tile_kernel(MxArgs a, int tiles_m, int tiles_n, int splits) {
  mx_tile<WK, WT, FK, FT, S, SPLIT, ORDERED>(a, tiles_m, tiles_n, SPLIT ? splits : 1);
}

// Sums the parts of a tile's results and finishes them: a thread takes one
// lane's four channels of a 16 x 16 result.
template <int WK, int WT, int FK, int FT, int S>
__global__ __launch_bounds__(256) void mx_join_kernel(MxArgs a, int tiles_m, int tiles_n, int splits) {
  using C = Tile<WK, WT, FK, FT, S>;
  const int tiles = tiles_m * tiles_n;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;  // f32x4 of a part
  const int tile = static_cast<int>(e / (C::kPart / 4));
  const int at = static_cast<int>(e - static_cast<int64_t>(tile) * (C::kPart / 4));
  const int lane = at & 63, j = (at >> 6) % FT, f = (at >> 6) / FT % FK, wid = (at >> 6) / (FT * FK);
  int tm, tn;
  tile_at(tile, tiles_m, tiles_n, tm, tn);
  const int t = tm * C::kBM + 16 * ((wid / WK) * FT + j) + (lane & 15);
  const int k = tn * C::kBN + 16 * (wid % WK) * FK + 64 * (f >> 2) + channel_of(f & 3, 4 * (lane >> 4));
  if (t >= a.T || k >= a.R) return;
  const f32x4_t* src = reinterpret_cast<const f32x4_t*>(a.workspace) + e;
  const int64_t pitch = static_cast<int64_t>(tiles) * (C::kPart / 4);
  f32x4_t sum = src[0];
  for (int s = 1; s < splits; ++s) sum += src[s * pitch];
  float o[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) o[c] = sum[c] + (a.bias ? a.bias[min(k + c, a.R - 1)] : 0.f);
  store_results(a, t, k, o);
}

template <int WK, int WT, int FK, int FT, int S, bool ORDERED>
hipError_t run_tile(const MxArgs& a, int splits, hipStream_t stream) {
  using C = Tile<WK, WT, FK, FT, S>;
  const int tiles_m = (a.T + C::kBM - 1) / C::kBM, tiles_n = (a.R + C::kBN - 1) / C::kBN;
  const int items = tiles_m * tiles_n * splits;
  const int most = (device_cu_count() & ~7) * C::kFit;
  const dim3 grid(static_cast<unsigned>(most > 0 && items > most ? most : items)), block(C::kThreads);
  if (splits == 1) {
    mx_tile_kernel<WK, WT, FK, FT, S, false, ORDERED><<<grid, block, 0, stream>>>(a, tiles_m, tiles_n, 1);
    return hipGetLastError();
  }
  mx_tile_kernel<WK, WT, FK, FT, S, true, ORDERED><<<grid, block, 0, stream>>>(a, tiles_m, tiles_n, splits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  mx_join_kernel<WK, WT, FK, FT, S><<<dim3(static_cast<unsigned>(tiles_m * tiles_n * (C::kPart / 1024))), dim3(256), 0,
                                       stream>>>(a, tiles_m, tiles_n, splits);
  return hipGetLastError();
}

// The tiles there are, and what they cost: microseconds for a quad with one
// work-group on a CU and with two side by side, and for a tile's start and stores,
// fitted to 1021 timings of 23 shapes (40 x 4096 x 4096 to 8192 x 4096 x 4096; 9 %
// rms) beside the call's 5.5 us.  The least estimate picked the fastest of the timed
// choices or one within 3 % of it at 22 of them (128 x 14336 x 4096 20.0 us, the
// best 19.1).
struct TileCost {
  int bm, bn, fit;
  double one, two, tile;
};
constexpr TileCost kTiles[] = {{256, 256, 1, 3.2, 0, 6.0},       // 4 x 2 waves of 64 channels x 128 tokens
                               {128, 128, 1, 1.38, 0, 0.63},     // 2 x 2 waves of 64 x 64, four stages
                               {128, 128, 2, 1.65, 2.66, 0.44},  // the same, two stages
                               {64, 128, 1, 1.10, 0, 0.58},      // 2 x 2 waves of 64 x 32
                               {64, 64, 2, 0.88, 1.54, 0.84}};   // 1 x 4 waves of 64 x 16


// The least estimate over the tiles and over parts of the row joined by a second
// kernel (3.4 us, and 3.6 TB/s over the partial sums), or what the bytes take.
MxPlan tile_plan(int64_t T, int64_t n, int64_t R) {
  MxPlan best{0, 1};
  double least = 1e30;
  const double bytes = static_cast<double>(T + R) * n * 17 / 32 + 2.0 * T * R;
  const int64_t quads = (n + 511) / 512;
  for (int c = 0; c < 5; ++c) {
    const TileCost& t = kTiles[c];
    const double tiles = static_cast<double>((T + t.bm - 1) / t.bm) * static_cast<double>((R + t.bn - 1) / t.bn);
    for (const int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (splits > 1 && (splits > quads || tiles * splits > 4 * kCus)) break;
      const double per_cu = ceil(tiles * splits / kCus);
      const double k = static_cast<double>(quads) / splits;
      double us = t.fit == 1 ? per_cu * (k * t.one + t.tile)
                             : floor(per_cu / 2) * (k * t.two + t.tile) + fmod(per_cu, 2) * (k * t.one + t.tile);
      us = fmax(us, bytes / 6.6e6) + (splits > 1 ? 3.4 + tiles * splits * t.bm * t.bn * 4 / 3.6e6 : 0);
      if (us < least) {
        least = us;
        best = {c, splits};
      }
    }
  }
  return best;
}

// ---- few tokens ---------------------------------------------------------------
//
// The weights are read once and bound the time (1 x 28672 x 8192 22.8 us, 5.4 TB/s).  A work-group takes 16 FK
// channels and all tokens (FT groups of sixteen); its waves share the row: wave w
// takes the 128-byte units w, w + waves, ... of the codes (eight blocks), so that
// the work-group reads its rows side by side.  Each wave has a ring of D units of
// its own in LDS, codes and scales, and waits for its own loads only; the partial
// sums meet in LDS at the end, joined in the waves' order.
//
// The loads go through LDS because a lane (g, i) holds 16 bytes of row i: sixteen
// neighbouring lanes would read sixteen rows, 64 cache accesses an instruction
// instead of eight whole lines.
//
// LDS rows of 128 bytes: chunk c of row r sits at chunk c ^ h(r), h(r) = (r & 7) ^
// ((r >> 3) & 1): lane (g, i) reads chunks 2 g and 2 g + 1 of row i, the sixteen
// lanes a read serves at a time on banks of their own.  So its blocks of MFMA s = 0,
// 1 are 2 g + s, and their scales the bytes of one 16-bit word; a row's eight
// scales of a unit are loaded as two words.  Beyond n the codes are the unit's
// first and the scales of both operands 2^-127: products that are zero in binary32.
//
// BYTES: rows of scales at any address (16 x 28704 x 8192 35.8 us, 33.8 on words).  A
// row's eight lie in three words then.
constexpr int kUnit = 128;
constexpr int64_t kMaxPitch = 1 << 23;  // a tile's offsets stay below 2^32

template <int FK, int FT, int D, bool BYTES>
struct Few {
  static constexpr int kWBytes = 16 * FK * kUnit, kTBytes = 16 * FT * kUnit;
  static constexpr int kWLoads = kWBytes / 1024, kTLoads = kTBytes / 1024;
  // scales: words of a row's eight, and loads of 64 of them
  static constexpr int kWords = BYTES ? 3 : 2;
  static constexpr int kSLoads = (16 * kWords * (FK + FT) + 63) / 64;
  static constexpr int kLoads = kWLoads + kTLoads + kSLoads;
  static constexpr int kSlot = kWBytes + kTBytes + 256 * kSLoads;
  static constexpr int kWave = D * kSlot;
  static_assert(8 * kWave <= 160 * 1024, "eight waves");
  static_assert(1024 * FK * FT <= kWave, "a wave's partial sums take its ring's place");
};

template <int FK, int FT, int D, bool BYTES>
__device__ __forceinline__ void mx_few(const MxArgs& a, uint8_t* few_lds) {
  using C = Few<FK, FT, D, BYTES>;
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int g = lane >> 4, i = lane & 15;
  const int n0 = 16 * FK * blockIdx.x;
  const int bytes = a.n / 2, blocks = a.n / mx::kBlock;
  const int units = (bytes + kUnit - 1) / kUnit;
  const int count = units > wid ? (units - wid - 1) / waves + 1 : 0;
  uint8_t* const ring = few_lds + wid * C::kWave;

  // rows and tokens beyond the tensors are clamped (their results are not stored)
  const int rows_w = min(16 * FK, a.R - n0);
  const __amdgpu_buffer_rsrc_t src_w =
      wave::buffer_rsrc(a.w + static_cast<int64_t>(n0) * a.ldw,
                        static_cast<uint32_t>(rows_w - 1) * static_cast<uint32_t>(a.ldw) + bytes);
  const __amdgpu_buffer_rsrc_t src_t =
      wave::buffer_rsrc(a.a, static_cast<uint32_t>(a.T - 1) * static_cast<uint32_t>(a.lda) + bytes);
  auto h = [](int r) { return (r & 7) ^ ((r >> 3) & 1); };
  // sources of the lane: load l of either operand fills rows 8 l .. 8 l + 7
  uint32_t off_w[C::kWLoads], off_t[C::kTLoads];
  auto chunk_at = [&](int l) { return 16 * ((lane & 7) ^ h((8 * l + (lane >> 3)) & 15)); };
#pragma unroll
  for (int l = 0; l < C::kWLoads; ++l)
    off_w[l] = static_cast<uint32_t>(min(8 * l + (lane >> 3), rows_w - 1)) * static_cast<uint32_t>(a.ldw);
#pragma unroll
  for (int l = 0; l < C::kTLoads; ++l)
    off_t[l] = static_cast<uint32_t>(min(8 * l + (lane >> 3), a.T - 1)) * static_cast<uint32_t>(a.lda);
  // words of scales, weights' rows first: of the word that a row starts in, and the
  // row's end from there
  auto scales_of = [&](int r) {
    return r < 16 * FK ? a.w_scale + static_cast<int64_t>(n0 + min(r, rows_w - 1)) * a.ldws
                       : a.scale + static_cast<int64_t>(min(r - 16 * FK, a.T - 1)) * a.lds;
  };
  auto shift_of = [&](int r) {
    return BYTES ? static_cast<int>(reinterpret_cast<uintptr_t>(scales_of(r)) & 3) : 0;
  };
  const uint8_t* src_s[C::kSLoads];
  int end_s[C::kSLoads];
#pragma unroll
  for (int q = 0; q < C::kSLoads; ++q) {
    const int r = (64 * q + lane) / C::kWords;
    src_s[q] = scales_of(r) - shift_of(r);
    end_s[q] = blocks + shift_of(r);
  }
  // unit x of this wave into ring slot x % D
  auto issue = [&](int x) {
    const int u = wid + x * waves;
    const int left = bytes - u * kUnit;
    uint8_t* const slot = ring + (x % D) * C::kSlot;
#pragma unroll
    for (int l = 0; l < C::kWLoads; ++l)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(src_w, (__attribute__((address_space(3))) void*)(slot + 1024 * l), 16,
                                               off_w[l] + (chunk_at(l) < left ? chunk_at(l) : 0), kUnit * u, 0, 0);
#pragma unroll
    for (int l = 0; l < C::kTLoads; ++l)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(src_t,
                                               (__attribute__((address_space(3))) void*)(slot + C::kWBytes + 1024 * l), 16,
                                               off_t[l] + (chunk_at(l) < left ? chunk_at(l) : 0), kUnit * u, 0, 0);
#pragma unroll
    for (int q = 0; q < C::kSLoads; ++q) {
      const int word = 4 * ((64 * q + lane) % C::kWords);
      __builtin_amdgcn_global_load_lds(
          (const __attribute__((address_space(1))) void*)(src_s[q] + 8 * u + (8 * u + word < end_s[q] ? word : 0)),
          (__attribute__((address_space(3))) void*)(slot + C::kWBytes + C::kTBytes + 256 * q), 4, 0, 0);
    }
  };
  // the lane's rows of scales in a slot, blocks 2 g and 2 g + 1
  int at_w[FK], at_t[FT];
#pragma unroll
  for (int f = 0; f < FK; ++f) at_w[f] = 4 * C::kWords * (16 * f + i) + shift_of(16 * f + i) + 2 * g;
#pragma unroll
  for (int j = 0; j < FT; ++j)
    at_t[j] = 4 * C::kWords * (16 * (FK + j) + i) + shift_of(16 * (FK + j) + i) + 2 * g;
  // (16-bit accesses: bytes would alias the loads to LDS, and the compiler wait for all)
  typedef uint16_t any_u16_t __attribute__((aligned(1)));
  auto pair_at = [](const uint8_t* p) -> uint32_t { return *reinterpret_cast<const any_u16_t*>(p); };

  f32x4_t acc[FK][FT];
#pragma unroll
  for (int f = 0; f < FK; ++f)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[f][j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int x = 0; x < min(D, count); ++x) issue(x);
  for (int x = 0; x < count; ++x) {
    if (x + D <= count)
      wave::wait_vmcnt<(D - 1) * C::kLoads>();
    else
      wave::wait_vmcnt<0>();
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* const sw = ring + (x % D) * C::kSlot;
    const uint8_t* const st = sw + C::kWBytes;
    const uint8_t* const ss = st + C::kTBytes;
    i32x4_t w[2][FK], tok[2][FT];
    uint32_t cw[FK], ct[FT];
#pragma unroll
    for (int f = 0; f < FK; ++f) cw[f] = pair_at(ss + at_w[f]);
#pragma unroll
    for (int j = 0; j < FT; ++j) ct[j] = pair_at(ss + at_t[j]);
#pragma unroll
    for (int s = 0; s < 2; ++s) {
#pragma unroll
      for (int f = 0; f < FK; ++f)
        w[s][f] = *reinterpret_cast<const i32x4_t*>(sw + 2048 * f + kUnit * i + 16 * ((2 * g + s) ^ h(i)));
#pragma unroll
      for (int j = 0; j < FT; ++j)
        tok[s][j] = *reinterpret_cast<const i32x4_t*>(st + 2048 * j + kUnit * i + 16 * ((2 * g + s) ^ h(i)));
    }
    // The slot is free once the reads are done; they are not ordered with the loads.
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    if (x + D < count) issue(x + D);
    __builtin_amdgcn_sched_barrier(0);
    const int here = blocks - 8 * (wid + x * waves);  // blocks from this unit on
    if (here < 8) {
      const uint32_t keep = 2 * g + 1 < here ? 0xffffu : 2 * g < here ? 0xffu : 0u;
#pragma unroll
      for (int f = 0; f < FK; ++f) cw[f] &= keep;
#pragma unroll
      for (int j = 0; j < FT; ++j) ct[j] &= keep;
    }
#pragma unroll
    for (int f = 0; f < FK; ++f)
#pragma unroll
      for (int j = 0; j < FT; ++j) {
        acc[f][j] = mfma<0, 0>(w[0][f], tok[0][j], acc[f][j], cw[f], ct[j]);
        acc[f][j] = mfma<1, 1>(w[1][f], tok[1][j], acc[f][j], cw[f], ct[j]);
      }
  }
#pragma unroll
  for (int f = 0; f < FK; ++f)
#pragma unroll
    for (int j = 0; j < FT; ++j)
      *reinterpret_cast<f32x4_t*>(ring + 16 * ((f * FT + j) * 64 + lane)) = acc[f][j];
  __syncthreads();
  // sums [FK][FT][64][4] of each wave: result e is channel e % 4 + 4 (e / 64 % 4) of group
  // e / 256 / FT, token e / 4 % 16 of group e / 256 % FT
  for (int e = threadIdx.x; e < 256 * FK * FT; e += blockDim.x) {
    const int k = n0 + 16 * ((e >> 8) / FT) + (e & 3) + 4 * ((e >> 6) & 3);
    const int t = 16 * ((e >> 8) % FT) + ((e >> 2) & 15);
    if (k >= a.R || t >= a.T) continue;
    float sum = reinterpret_cast<const float*>(few_lds)[e];
    for (int v = 1; v < waves; ++v) sum += reinterpret_cast<const float*>(few_lds + v * C::kWave)[e];
    row::store_elem(a.out, static_cast<int64_t>(t) * a.ldo + k, sum + (a.bias ? a.bias[k] : 0.f), a.out_bf16);
  }
}

template <int FK, int FT, int D, bool BYTES>
__global__ __launch_bounds__(512) void mx_few_kernel(MxArgs a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t few_lds[];
  mx_few<FK, FT, D, BYTES>(a, few_lds);
}

template <int FK, int FT, int D, bool BYTES>
hipError_t run_few_rows(const MxArgs& a, hipStream_t s) {
  using C = Few<FK, FT, D, BYTES>;
  const int groups = (a.R + 16 * FK - 1) / (16 * FK), units = (a.n / 2 + kUnit - 1) / kUnit;
  int waves = 8;
  while (waves > 2 && (groups * waves > 8 * kCus || units < waves)) waves /= 2;
  mx_few_kernel<FK, FT, D, BYTES><<<dim3(static_cast<unsigned>(groups)), dim3(static_cast<unsigned>(64 * waves)),
                            static_cast<unsigned>(waves * C::kWave), s>>>(a);
  return hipGetLastError();
}

bool aligned_rows(const uint8_t* p, int64_t ld, int64_t to) {
  return ld % to == 0 && (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0 && ld < kMaxPitch;
}

template <int FK, int FT, int D>
hipError_t run_few_as(const MxArgs& a, hipStream_t s) {
  return aligned_rows(a.scale, a.lds, 4) && aligned_rows(a.w_scale, a.ldws, 4) ? run_few_rows<FK, FT, D, false>(a, s)
                                                                               : run_few_rows<FK, FT, D, true>(a, s);
}

// 32 channels a work-group halve what it reads of the tokens, which up to sixteen
// tokens' rows is as much as the weights (16 x 28672 x 8192 26.8 us, 30.3 with sixteen
// channels; 32 tokens 32.5 and 40.8), where that still gives more than half of the CUs
// a work-group (16 x 14336 x 4096 12.8 and 9.7); up to four tokens it gains nothing
// (2 x 28672 x 8192 24.0 and 22.8).  Times on weights that no cache holds.
bool few_wide(int64_t T, int64_t R) { return T > 4 && R > 16 * kCus; }

// Beyond sixteen tokens and two work-groups a CU the tiles are faster (32 x 8192 x
// 20480 26.5 us, 30.3 here; 32 x 8192 x 7168 here 11.1).
bool takes_few(int64_t T, int64_t R) { return (T <= 16 && R <= (int64_t{1} << 24)) || (T <= 32 && R <= 64 * kCus); }

hipError_t run_few(const MxArgs& a, hipStream_t s) {
  if (few_wide(a.T, a.R)) return a.T <= 16 ? run_few_as<2, 1, 2>(a, s) : run_few_as<2, 2, 2>(a, s);
  return a.T <= 16 ? run_few_as<1, 1, 4>(a, s) : run_few_as<1, 2, 2>(a, s);
}

// ---- any stride and alignment ---------------------------------------------------
//
// Rows that do not start on 16-byte boundaries (codes), or 4-byte ones (fewer than four
// scales), are laid out anew in the workspace, in rows of whole 16-byte chunks.
struct Copy {
  const uint8_t* src;
  int64_t ld;
  uint8_t* dst;
  int64_t rows;
  int bytes;  // of a row
};
struct Copies {
  Copy c[4];
};
__host__ __device__ __forceinline__ int64_t copy_pitch(int bytes) { return (bytes + 15) & ~15; }

__global__ __launch_bounds__(256) void mx_copy_kernel(Copies all) {
  const Copy c = all.c[blockIdx.y];
  const int per = static_cast<int>(copy_pitch(c.bytes) / 16);
  const int64_t most = c.rows * per;
  for (int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; e < most;
       e += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t r = e / per;
    const int at = 16 * static_cast<int>(e - r * per);
    const uint8_t* const src = c.src + r * c.ld + at;
    wave::u32x4_t v = {0, 0, 0, 0};
    if (at + 16 <= c.bytes) {
      v = row::load_as<false, wave::u32x4_t>(src);
    } else {
#pragma unroll
      for (int b = 0; b < 16; ++b)
        if (at + b < c.bytes) v[b >> 2] |= static_cast<uint32_t>(src[b]) << (8 * (b & 3));
    }
    *reinterpret_cast<wave::u32x4_t*>(c.dst + 16 * e) = v;
  }
}

// The workspace after the partial sums: the copies that the operands need and, for
// tiles that take them so, the ordered scales.  a takes what is laid out anew.
struct Layout {
  Copies copies = {};
  int count = 0;
  Order order = {};
  int64_t end = 0;
  Layout(MxArgs& a, int64_t at, bool ordered) : end(at) {
    copy(a, a.a, a.lda, a.T, a.n / 2, 16);
    copy(a, a.w, a.ldw, a.R, a.n / 2, 16);
    if (!ordered) {
      const int blocks = a.n / mx::kBlock;
      copy(a, a.scale, a.lds, a.T, blocks, blocks < 4 ? 4 : 1);
      copy(a, a.w_scale, a.ldws, a.R, blocks, blocks < 4 ? 4 : 1);
      return;
    }
    order.blocks = a.n / mx::kBlock;
    order.quads = (order.blocks + 15) / 16;
    order.words = aligned_rows(a.scale, a.lds, 4) && aligned_rows(a.w_scale, a.ldws, 4);
    end = (end + 15) & ~int64_t{15};
    sort(a, 0, a.scale, a.lds, a.T);
    sort(a, 1, a.w_scale, a.ldws, a.R);
  }

 private:
  void copy(const MxArgs& a, const uint8_t*& p, int64_t& ld, int64_t rows, int bytes, int64_t to) {
    if (aligned_rows(p, ld, to)) return;
    uint8_t* const dst = a.workspace + end;
    copies.c[count++] = {p, ld, dst, rows, bytes};
    p = dst;
    ld = copy_pitch(bytes);
    end += rows * ld;
  }
  void sort(const MxArgs& a, int k, const uint8_t*& p, int64_t ld, int rows) {
    order.src[k] = p;
    order.ld[k] = ld;
    order.dst[k] = a.workspace + end;
    order.rows[k] = rows;
    order.groups[k] = (rows + 255) / 256 * 4;  // whole tiles
    p = order.dst[k];
    end += int64_t{1024} * order.quads * order.groups[k];
  }
};

int64_t partial_bytes(const MxArgs& a, const MxPlan& p) {
  if (p.splits == 1) return 0;
  const TileCost& t = kTiles[p.kind];
  const int64_t tiles = static_cast<int64_t>((a.T + t.bm - 1) / t.bm) * ((a.R + t.bn - 1) / t.bn);
  return tiles * p.splits * t.bm * t.bn * 4;
}

}  // namespace

MxPlan mx_plan(const MxArgs& a) {
  if (a.T == 0 || a.R == 0 || takes_few(a.T, a.R)) return {-1, 1};
  return tile_plan(a.T, a.n, a.R);
}

int64_t mx_workspace(const MxArgs& a, const MxPlan& plan) {
  if (a.T == 0 || a.R == 0) return 0;
  MxArgs b = a;
  b.workspace = nullptr;
  return Layout(b, partial_bytes(a, plan), plan.kind == 0).end;
}

const char* mx_name(const MxArgs& a) {
  static const char* const names[] = {"mx_tile256x256", "mx_tile128x128_s4", "mx_tile128x128_s2", "mx_tile64x128",
                                      "mx_tile64x64"};
  const MxPlan plan = mx_plan(a);
  if (plan.kind >= 0) return names[plan.kind];
  if (few_wide(a.T, a.R)) return a.T <= 16 ? "mx_few16_k32" : "mx_few32_k32";
  return a.T <= 16 ? "mx_few16" : "mx_few32";
}

hipError_t launch_mx(const MxArgs& args, const MxPlan& plan, hipStream_t s) {
  MxArgs a = args;
  const bool ordered = plan.kind == 0;
  const Layout lay(a, partial_bytes(args, plan), ordered);
  if (lay.count > 0) {
    mx_copy_kernel<<<dim3(1024, static_cast<unsigned>(lay.count)), 256, 0, s>>>(lay.copies);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (plan.kind < 0) return run_few(a, s);
  if (ordered) {
    const int groups = lay.order.groups[0] + lay.order.groups[1];
    mx_order_kernel<<<dim3(static_cast<unsigned>((lay.order.quads + 3) / 4),
                           static_cast<unsigned>(groups < 65535 ? groups : 65535)),
                      256, 0, s>>>(lay.order);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  switch (plan.kind) {
    case 0: return run_tile<4, 2, 4, 8, 2, true>(a, plan.splits, s);
    case 1: return run_tile<2, 2, 4, 4, 4, false>(a, plan.splits, s);
    case 2: return run_tile<2, 2, 4, 4, 2, false>(a, plan.splits, s);
    case 3: return run_tile<2, 2, 4, 2, 4, false>(a, plan.splits, s);
    default: return run_tile<1, 4, 4, 1, 4, false>(a, plan.splits, s);
  }
}

}  // namespace signrot
