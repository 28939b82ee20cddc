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
// does not have, and moves them about.  AGPR: the sums are accumulation
// registers.  The leading s_nop covers a VALU write of an operand just before.
// The reader of a sum has to wait for the last one (settle).
template <int OA, int OB, bool AGPR>
__device__ __forceinline__ void mfma_to(f32x4_t& acc, const i32x4_t& a, const i32x4_t& b, uint32_t sa, uint32_t sb) {
#define SR_MFMA "s_nop 1\n\tv_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[%5,%6,0] op_sel_hi:[%7,%8,0] cbsz:4 blgp:4"
  if constexpr (AGPR)
    asm volatile(SR_MFMA
                 : "+a"(acc)
                 : "v"(a), "v"(b), "v"(sa), "v"(sb), "n"(OA & 1), "n"(OB & 1), "n"(OA >> 1), "n"(OB >> 1));
  else
    asm volatile(SR_MFMA
                 : "+v"(acc)
                 : "v"(a), "v"(b), "v"(sa), "v"(sb), "n"(OA & 1), "n"(OB & 1), "n"(OA >> 1), "n"(OB >> 1));
#undef SR_MFMA
}
// A sum's value, read where it is asked for and not before.
template <bool AGPR>
__device__ __forceinline__ float value_of(float sum) {
  if constexpr (!AGPR) return sum;
  float v;
  asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v) : "a"(sum));
  return v;
}
__device__ __forceinline__ void settle() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

// Results of token t from channel k on: vectors at whatever address they have,
// single ones at the row's end.
template <int N>
__device__ __forceinline__ void store_results(const MxArgs& a, int t, int k, const float (&o)[N]) {
  const int64_t at = static_cast<int64_t>(t) * a.ldo + k;
  const bool whole = k + N <= a.R;
  if (whole && a.out_bf16) {
    uint16_t* const out = static_cast<uint16_t*>(a.out) + at;
    uint32_t h[N / 2];
#pragma unroll
    for (int e = 0; e < N / 2; ++e) h[e] = row::pack_bf16(o[2 * e], o[2 * e + 1]);
    if (N == 4) row::store_as<false>(out, wave::u32x2_t{h[0], h[1]});
#pragma unroll
    for (int e = 0; e < N / 8; ++e)
      row::store_as<false>(out + 8 * e, wave::u32x4_t{h[4 * e], h[4 * e + 1], h[4 * e + 2], h[4 * e + 3]});
  } else if (whole) {
    float* const out = static_cast<float*>(a.out) + at;
#pragma unroll
    for (int e = 0; e < N; e += 4) row::store_as<false>(out + e, f32x4_t{o[e], o[e + 1], o[e + 2], o[e + 3]});
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
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
constexpr int kQuad = 4;                // MFMA depths whose scales are handled together
constexpr int kQuadBytes = kQuad * kDeep;

// WK x WT waves of FK x FT 16 x 16 results each, a ring of four steps of KU
// MFMAs' depth.
template <int WK, int WT, int FK, int FT, int KU>
struct Tile {
  static constexpr int S = 4;
  static constexpr int kStep = KU * kDeep;  // bytes of a row per step
  static constexpr int kSteps = kQuad / KU; // of a quad
  static constexpr int kWaves = WK * WT;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kBN = 16 * WK * FK;  // channels
  static constexpr int kBM = 16 * WT * FT;  // tokens
  // LDS bytes of one MFMA's depth, its 1 KiB loads, and the loads per wave and step
  static constexpr int kWDeep = kBN * kDeep, kTDeep = kBM * kDeep;
  static constexpr int kWBlocks = kWDeep / 1024, kTBlocks = kTDeep / 1024;
  static constexpr int kWLoads = KU * kWBlocks / kWaves, kTLoads = KU * kTBlocks / kWaves;
  static constexpr int kLoads = kWLoads + kTLoads;
  static constexpr int kWStage = KU * kWDeep, kTStage = KU * kTDeep;
  static constexpr bool kAgpr = FK * FT > 32;
  static constexpr int kPart = 256 * FK * FT * kWaves;  // floats of a tile's partial sums
  // scales: groups of 64 rows (weights, then tokens), a word of four rows' for
  // each lane and depth
  static constexpr int kGroupsW = kBN / 64, kGroups = (kBN + kBM) / 64;
  static constexpr int kScales = kGroups * kQuad * 256;
  static constexpr int kPer = kGroups > kWaves ? kGroups / kWaves : 1;  // groups that a wave lays out
  static constexpr int kRing = S * (kWStage + kTStage);
  static constexpr int kLds = kRing + 2 * kScales;
  // work-groups to a CU: as many as its LDS holds, at most eight waves
  static constexpr int kFit = 160 * 1024 / kLds < 8 / kWaves ? 160 * 1024 / kLds : 8 / kWaves;
  static_assert(kWLoads * kWaves == KU * kWBlocks && kTLoads * kWaves == KU * kTBlocks, "whole loads per wave");
  static_assert(kWBlocks * 1024 == kWDeep && kTBlocks * 1024 == kTDeep, "whole loads");
  static_assert(FK % 4 == 0 && kBM % 64 == 0, "rows come in groups of 64");
  static_assert(KU == 1 || KU == 2, "two to four steps a quad");
  static_assert(FT % 4 == 0 || 4 % FT == 0, "a wave's tokens lie in whole words of scales or in one");
  static_assert(kGroups <= kWaves || kPer * kWaves == kGroups, "whole groups of scales per wave");
  static_assert(kGroupsW % kPer == 0, "a wave's groups are of one operand");
  static_assert(kFit > 0, "LDS");
  static_assert(kWLoads >= 2 && kTLoads >= 2, "a wave's own 2 KiB of either operand");
};

// Both operands stream global -> LDS (16 bytes a lane, no registers) through a
// ring of four steps; one barrier a step.  Step s: the MFMAs of step s, the
// loads of step s + 3 into the buffers step s - 1 used, and towards its end the
// first operand reads of step s + 1 (which has landed: the barrier at the end
// of step s - 1 came after every wave's wait for it).
//
// A work-group takes the tiles p, p + stride, ... below `end`, and the ring
// runs on from tile to tile: the last steps of a tile load the first ones of
// the next, which arrive while its results are stored.
//
// A row is cut into quads of four MFMA depths (512 channels).  Quad 0 of a tile
// is the row's last, possibly short one.  Its chunks beyond n are read from the
// quad's first chunk, and the scales of both operands there are 2^-127: the
// products, below 2^-248, are zero in binary32.
//
// LDS rows of 64 bytes, four 16-byte chunks: logical chunk c of row r sits at
// physical chunk c ^ 2 ((r >> 3) & 1), so that the sixteen lanes a 16-byte read
// serves at a time cover the 64 banks once.  A lane (g = lane / 16, i = lane %
// 16) reads row i, chunk g of a 16-row group: block g of the depth for both
// operands.
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
// that a cache line is touched once for four depths), turns the four by four
// bytes with eight permutes two steps later, when a step's wait has seen them
// arrive, and writes them to LDS a step before they are read.
__device__ __forceinline__ int channel_of(int f, int i) { return 32 * (f >> 1) + 8 * (i >> 2) + 4 * (f & 1) + (i & 3); }

template <int WK, int WT, int FK, int FT, int KU, bool SPLIT>
__device__ __forceinline__ void mx_tile(const MxArgs& a, int tiles_m, int tiles_n, int splits) {
  using C = Tile<WK, WT, FK, FT, KU>;
  constexpr int S = C::S;
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
  // clamped (their results are not stored).
  // Load l of a wave is block kLoads * wave + l of the step's, counted through
  // the depths: sixteen rows of weights or tokens.
  const int chunk = 16 * ((lane & 3) ^ (2 * (lane >> 5)));  // byte of the lane's slot (row lane / 4 of 16) in a depth
  int src_p = p, lq, lq_end;
  const uint8_t *base_w, *base_t, *base_s;
  int rows_w, rows_t;
  uint32_t off_w[C::kWLoads], off_t[C::kTLoads];
  auto depth_w = [&](int l) { return (C::kWLoads * wid + l) / C::kWBlocks; };
  auto depth_t = [&](int l) { return (C::kTLoads * wid + l) / C::kTBlocks; };
  // This wave's first group of 64 rows of scales (waves beyond the groups repeat the last).
  const int group = min(C::kPer * wid, C::kGroups - 1);
  const bool of_w = group < C::kGroupsW;
  // (an opaque copy of the lane where its constants are used once a quad or less, so
  // that they are formed there and not kept in registers)
  auto lane_here = [&]() {
    int here = lane;
    asm volatile("" : "+v"(here));
    return here;
  };
  auto set_source = [&]() {
    const int lane = lane_here();
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
    base_s = of_w ? a.w_scale + static_cast<int64_t>(n0) * a.ldws : a.scale + static_cast<int64_t>(m0) * a.lds;
#pragma unroll
    for (int l = 0; l < C::kWLoads; ++l) {
      const int slot = 16 * ((C::kWLoads * wid + l) % C::kWBlocks) + (lane >> 2);
      const int ch = (slot & ~63) + channel_of((slot >> 4) & 3, slot & 15);
      off_w[l] = static_cast<uint32_t>(min(ch, rows_w - 1)) * static_cast<uint32_t>(a.ldw) + kDeep * depth_w(l) + chunk;
    }
#pragma unroll
    for (int l = 0; l < C::kTLoads; ++l) {
      const int r = 16 * ((C::kTLoads * wid + l) % C::kTBlocks) + (lane >> 2);
      off_t[l] = static_cast<uint32_t>(min(r, rows_t - 1)) * static_cast<uint32_t>(a.lda) + kDeep * depth_t(l) + chunk;
    }
  };
  int at_quad;  // its first byte in a row
  int left;     // bytes of it
  auto place = [&]() {
    at_quad = __builtin_amdgcn_readfirstlane(kQuadBytes * (lq == 0 ? quads - 1 : lq - 1));
    left = __builtin_amdgcn_readfirstlane(min(bytes - at_quad, kQuadBytes));
  };
  // Past the last item the loads go on with that item's: every step issues the
  // same number, so the vmcnt thresholds are exact.
  auto advance = [&]() {
    lq = __builtin_amdgcn_readfirstlane(lq + 1);
    if (lq == lq_end) {
      src_p = src_p + stride < end ? src_p + stride : src_p;
      set_source();
    }
    place();
  };
  // load l of step lj of the quad, into ring position `to`
  auto issue = [&](int l, int lj, int to) {
    const bool w = l < C::kWLoads;
    const int k = w ? l : l - C::kWLoads;
    const int depth = w ? depth_w(k) : depth_t(k);
    const uint32_t off = w ? off_w[k] : off_t[k];
    const uint32_t in = chunk < left - C::kStep * lj - kDeep * depth ? off + C::kStep * lj : off - kDeep * depth - chunk;
    __builtin_amdgcn_raw_ptr_buffer_load_lds(
        w ? wave::buffer_rsrc(base_w, static_cast<uint32_t>(rows_w - 1) * static_cast<uint32_t>(a.ldw) + bytes)
          : wave::buffer_rsrc(base_t, static_cast<uint32_t>(rows_t - 1) * static_cast<uint32_t>(a.lda) + bytes),
        (__attribute__((address_space(3))) void*)(w ? lds_w + C::kWStage * to + 1024 * (C::kWLoads * wid + k)
                                                    : lds_t + C::kTStage * to + 1024 * (C::kTLoads * wid + k)),
        16, in, at_quad, 0, 0);
  };

  // The scales of the quad, words s = g of the rows; those beyond n read the quad's first.
  uint32_t raw[C::kPer][4];
  int raw_left = 0;
  auto load_scales = [&]() {
    const uint32_t ld = static_cast<uint32_t>(of_w ? a.ldws : a.lds);
    const int rows = of_w ? rows_w : rows_t;
    const int here = lane_here(), g = here >> 4, i = here & 15;
    const int r0 = 64 * (of_w ? group : group - C::kGroupsW);
    raw_left = left / mx::kBlockBytes;
    const uint32_t word = 4 * g < raw_left ? 4 * g : 0;
    const __amdgpu_buffer_rsrc_t src =
        wave::buffer_rsrc(base_s, static_cast<uint32_t>(rows - 1) * ld + ((blocks + 3) & ~3));
#pragma unroll
    for (int x = 0; x < C::kPer; ++x)
#pragma unroll
      for (int f = 0; f < 4; ++f) {
        const int r = r0 + 64 * x + (of_w ? channel_of(f, i) : 16 * f + i);
        raw[x][f] = __builtin_amdgcn_raw_buffer_load_b32(src, static_cast<uint32_t>(min(r, rows - 1)) * ld + word,
                                                         at_quad / mx::kBlockBytes, 0);
      }
  };
  auto turn_scales = [&](int half) {
    const int here = lane_here(), g = here >> 4;
    uint32_t* const turned = reinterpret_cast<uint32_t*>(lds_s + 1024 * group + 256 * g) + (here & 15);
#pragma unroll
    for (int x = 0; x < C::kPer; ++x) {
      const uint32_t(&d)[4] = raw[x];
      const uint32_t a0 = __builtin_amdgcn_perm(d[1], d[0], 0x05010400u);
      const uint32_t a1 = __builtin_amdgcn_perm(d[1], d[0], 0x07030602u);
      const uint32_t b0 = __builtin_amdgcn_perm(d[3], d[2], 0x05010400u);
      const uint32_t b1 = __builtin_amdgcn_perm(d[3], d[2], 0x07030602u);
      const uint32_t o[4] = {__builtin_amdgcn_perm(b0, a0, 0x05040100u), __builtin_amdgcn_perm(b0, a0, 0x07060302u),
                             __builtin_amdgcn_perm(b1, a1, 0x05040100u), __builtin_amdgcn_perm(b1, a1, 0x07060302u)};
#pragma unroll
      for (int b = 0; b < 4; ++b)
        turned[half * (C::kScales / 4) + 256 * x + 16 * b] = 4 * g + b < raw_left ? o[b] : 0;
    }
  };

  const int read_w = 16 * wk * FK * kDeep + i * kDeep + 16 * (g ^ (2 * (i >> 3)));
  const int read_t = 16 * wt * FT * kDeep + i * kDeep + 16 * (g ^ (2 * (i >> 3)));
  auto weight = [&](int pos, int depth, int f) {
    return *reinterpret_cast<const i32x4_t*>(lds_w + C::kWStage * pos + C::kWDeep * depth + read_w + 16 * kDeep * f);
  };
  auto token = [&](int pos, int depth, int j) {
    return *reinterpret_cast<const i32x4_t*>(lds_t + C::kTStage * pos + C::kTDeep * depth + read_t + 16 * kDeep * j);
  };
  // scales of a depth: a word for four of the wave's 16-row groups
  constexpr int kSW = FK / 4, kST = FT >= 4 ? FT / 4 : 1;
  const int scale_w = 1024 * (wk * FK / 4) + 4 * lane;
  const int scale_t = 1024 * (C::kGroupsW + wt * FT / 4) + 4 * lane;
  const int shift_t = FT >= 4 ? 0 : 8 * (wt * FT % 4);  // a wave with fewer than four: its bytes lowest
  uint32_t sw[kSW], st[kST];
  auto read_scales = [&](int half, int e) {
#pragma unroll
    for (int q = 0; q < kSW; ++q)
      sw[q] = *reinterpret_cast<const uint32_t*>(lds_s + half * C::kScales + scale_w + 1024 * q + 256 * e);
#pragma unroll
    for (int q = 0; q < kST; ++q)
      st[q] = *reinterpret_cast<const uint32_t*>(lds_s + half * C::kScales + scale_t + 1024 * q + 256 * e) >> shift_t;
  };

  f32x4_t acc[FK][FT];
  i32x4_t tok[2][FT];  // token operands of this and the next depth
  i32x4_t wf[FK + 2];

  set_source();
  place();
  load_scales();
#pragma unroll
  for (int s = 0; s < S - 1; ++s) {
    if (s == C::kSteps) {
      advance();
      wave::wait_vmcnt<C::kSteps * C::kLoads>();
      __builtin_amdgcn_sched_barrier(0);
      turn_scales(0);
      load_scales();
    }
#pragma unroll
    for (int l = 0; l < C::kLoads; ++l) issue(l, s % C::kSteps, s);
  }
  if (C::kSteps >= S - 1) {
    wave::wait_vmcnt<(S - 1) * C::kLoads>();
    __builtin_amdgcn_sched_barrier(0);
    turn_scales(0);
  }
  wave::wait_vmcnt<(S - 3) * C::kLoads>();
  wave::lds_barrier();
  wf[0] = weight(0, 0, 0);
  wf[1] = weight(0, 0, 1);
#pragma unroll
  for (int j = 0; j < FT; ++j) tok[0][j] = token(0, 0, j);

  // Step j of a quad at ring position pos: its depths, and the loads of the step
  // three ahead, in step 1 the first of a quad.  The scales of a quad's first depth
  // are read as it starts (published by the barrier before), the others' a depth
  // ahead.
  auto step = [&](auto J, int pos, int half) {
    constexpr int j = decltype(J)::value;
    const int next = (pos + 1) % S, to = (pos + 3) % S;
    if (j == 0) read_scales(half, 0);
    if (j == 3 % C::kSteps) turn_scales(half ^ 1);  // loaded two steps ago
    if (j == 1) load_scales();
    unrolled<KU>([&](auto UC) {
      constexpr int u = decltype(UC)::value, e = j * KU + u;
      i32x4_t(&now)[FT] = tok[e & 1];
      i32x4_t(&then)[FT] = tok[(e + 1) & 1];
      const int then_pos = u + 1 < KU ? pos : next, then_depth = u + 1 < KU ? u + 1 : 0;
      uint32_t cw[kSW], ct[kST];
#pragma unroll
      for (int q = 0; q < kSW; ++q) cw[q] = sw[q];
#pragma unroll
      for (int q = 0; q < kST; ++q) ct[q] = st[q];
      unrolled<FK>([&](auto F) {
        constexpr int f = decltype(F)::value;
        // The reads follow the block's first MFMA: the wait before that one is
        // then for reads a whole block old.
        mfma_to<f % 4, 0, C::kAgpr>(acc[f][0], wf[f], now[0], cw[f / 4], ct[0]);
        __builtin_amdgcn_sched_barrier(0);
        // two reads ahead, the last two from the next depth or step
        wf[f + 2] = f + 2 < FK ? weight(pos, u, f + 2) : weight(then_pos, then_depth, f + 2 - FK);
#pragma unroll
        for (int t = f * FT / FK; t < (f + 1) * FT / FK; ++t) then[t] = token(then_pos, then_depth, t);
        if (f == FK - 1 && e + 1 < kQuad) read_scales(half, e + 1);
        constexpr int kBlocks = KU * FK, b = u * FK + f;
#pragma unroll
        for (int l = b * C::kLoads / kBlocks; l < (b + 1) * C::kLoads / kBlocks; ++l) issue(l, (j + 3) % C::kSteps, to);
        unrolled<FT - 1>([&](auto T) {
          constexpr int t = decltype(T)::value + 1;
          mfma_to<f % 4, t % 4, C::kAgpr>(acc[f][t], wf[f], now[t], cw[f / 4], ct[t / 4]);
        });
        __builtin_amdgcn_sched_barrier(0);
      });
      wf[0] = wf[FK];
      wf[1] = wf[FK + 1];
    });
    if (j == 0) advance();
    wave::wait_vmcnt<(S - 3) * C::kLoads + (j == 1 ? 4 * C::kPer : 0)>();
    if (j == 3 % C::kSteps)
      wave::lds_barrier();  // the scales are written
    else
      __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
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
      unrolled<C::kSteps>([&](auto J) { step(J, (C::kSteps == S ? 0 : pos) + J, half); });
      if (C::kSteps != S) pos ^= C::kSteps;
      half ^= 1;
    }

    settle();
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
    // sixteen rows of 128 bytes at a time, a unit, go through LDS and leave as whole
    // lines: through the places that the wave itself fills next in the ring position
    // of the last step, which all waves have done with.  Chunk c of row r sits at
    // chunk c ^ ((r >> 1) & 7): the sixteen lanes that an access serves at a time
    // cover the banks once.  Units alternate between two places; a wave's LDS
    // accesses are done in order, so that the next unit is written before this
    // one has been read back.
    const int last = C::kSteps == S ? S - 1 : (pos ^ C::kSteps) + C::kSteps - 1;
    auto chunk_at = [&](int odd, int r, int c) {
      uint8_t* const mine = odd ? lds_t + C::kTStage * last + 1024 * C::kTLoads * wid
                                : lds_w + C::kWStage * last + 1024 * C::kWLoads * wid;
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
    }
    auto results = [&](auto BF16) {
      constexpr int per = BF16 ? 8 : 4;                   // results of a chunk
      constexpr int parts = BF16 ? 1 : 2;                 // units of 64 channels
      constexpr int units = FK / 4 * FT * parts;
      auto put = [&](auto U) {
        constexpr int u = decltype(U)::value, part = u % parts, j = u / parts % FT, q = u / parts / FT;
        if constexpr (BF16) {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            wave::u32x4_t v;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = row::pack_bf16(
                  value_of<C::kAgpr>(acc[4 * q + 2 * h + (e >> 1)][j][2 * (e & 1)]) + bias[q][8 * h + 2 * e],
                  value_of<C::kAgpr>(acc[4 * q + 2 * h + (e >> 1)][j][2 * (e & 1) + 1]) + bias[q][8 * h + 2 * e + 1]);
            *chunk_at(u & 1, i, 4 * h + g) = v;
          }
        } else {
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            wave::u32x4_t v;
#pragma unroll
            for (int e = 0; e < 4; ++e)
              v[e] = __float_as_uint(value_of<C::kAgpr>(acc[4 * q + 2 * part + h][j][e]) +
                                     bias[q][8 * part + 4 * h + e]);
            *chunk_at(u & 1, i, 2 * g + h) = v;
          }
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
          if (t < a.T && k + per <= a.R) {
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
      put(std::integral_constant<int, 0>{});
      unrolled<units>([&](auto U) {
        constexpr int u = decltype(U)::value;
        if constexpr (u + 1 < units) put(std::integral_constant<int, u + 1>{});
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int h = 0; h < 2; ++h) got[u & 1][h] = *chunk_at(u & 1, 8 * h + r0, c);
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if constexpr (u > 0) send(std::integral_constant<int, u - 1>{});
      });
      send(std::integral_constant<int, units - 1>{});
    };
    if (a.out_bf16)
      results(std::true_type{});
    else
      results(std::false_type{});
  }
  wave::wait_vmcnt<0>();
}

template <int WK, int WT, int FK, int FT, int KU, bool SPLIT>
__global__ __launch_bounds__(64 * WK * WT) __attribute__((
    amdgpu_waves_per_eu(Tile<WK, WT, FK, FT, KU>::kWaves * Tile<WK, WT, FK, FT, KU>::kFit / 4)))
void mx_tile_kernel(MxArgs a, int tiles_m, int tiles_n, int splits) {
  mx_tile<WK, WT, FK, FT, KU, SPLIT>(a, tiles_m, tiles_n, SPLIT ? splits : 1);
}

// Sums the parts of a tile's results and finishes them: a thread takes one
// lane's four channels of a 16 x 16 result.
template <int WK, int WT, int FK, int FT, int KU>
__global__ __launch_bounds__(256) void mx_join_kernel(MxArgs a, int tiles_m, int tiles_n, int splits) {
  using C = Tile<WK, WT, FK, FT, KU>;
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

template <int WK, int WT, int FK, int FT, int KU>
hipError_t run_tile(const MxArgs& a, int splits, hipStream_t s) {
  using C = Tile<WK, WT, FK, FT, KU>;
  const int tiles_m = (a.T + C::kBM - 1) / C::kBM, tiles_n = (a.R + C::kBN - 1) / C::kBN;
  const int items = tiles_m * tiles_n * splits;
  const int most = (device_cu_count() & ~7) * C::kFit;
  const dim3 grid(static_cast<unsigned>(most > 0 && items > most ? most : items)), block(C::kThreads);
  if (splits == 1) {
    mx_tile_kernel<WK, WT, FK, FT, KU, false><<<grid, block, 0, s>>>(a, tiles_m, tiles_n, 1);
    return hipGetLastError();
  }
  mx_tile_kernel<WK, WT, FK, FT, KU, true><<<grid, block, 0, s>>>(a, tiles_m, tiles_n, splits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  mx_join_kernel<WK, WT, FK, FT, KU><<<dim3(static_cast<unsigned>(tiles_m * tiles_n * (C::kPart / 1024))), dim3(256), 0,
                                       s>>>(a, tiles_m, tiles_n, splits);
  return hipGetLastError();
}

struct TileCost {
  int bm, bn, fit;
  double one, two, tile;
};
constexpr TileCost kTiles[] = {{256, 256, 1, 1.35, 0, 2.8},      // 4 x 2 waves of 64 channels x 128 tokens
                               {128, 128, 1, 0.453, 0, 1.4},     // 2 x 2 waves of 64 x 64
                               {64, 128, 1, 0.280, 0, 1.2},      // 2 x 2 waves of 64 x 32
                               {64, 64, 2, 0.184, 0.341, 1.4}};  // 1 x 4 waves of 64 x 16

struct Plan {
  int kind, splits;
  double us;
};

Plan tile_plan(int64_t T, int64_t n, int64_t R) {
  Plan best{0, 1, 1e30};
  const double bytes = static_cast<double>(T + R) * n * 17 / 32 + 2.0 * T * R;
  for (int c = 0; c < 4; ++c) {
    const TileCost& t = kTiles[c];
    const double tiles = static_cast<double>((T + t.bm - 1) / t.bm) * static_cast<double>((R + t.bn - 1) / t.bn);
    const int64_t quads = (n + 511) / 512;
    for (const int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (splits > 1 && (splits > quads || tiles * splits > 4 * kCus)) break;
      const double per_cu = ceil(tiles * splits / kCus);
      const double k = 2.0 * quads / splits;  // 256 channels
      double us = t.fit == 1 ? per_cu * (k * t.one + t.tile)
                             : floor(per_cu / 2) * (k * t.two + t.tile) + fmod(per_cu, 2) * (k * t.one + t.tile);
      us = fmax(us, bytes / 7e6) + (splits > 1 ? 3.5 + tiles * splits * t.bm * t.bn * 4 / 3.3e6 : 0);
      if (us < best.us) best = {c, splits, us};
    }
  }
  return best;
}

constexpr int64_t kMaxPitch = 1 << 23;  // a tile's offsets stay below 2^32

// ---- any stride and alignment ---------------------------------------------------
//
// Rows that do not start on 16-byte boundaries (codes) or 4-byte ones (scales)
// are laid out anew in the workspace, in rows of whole 16-byte chunks.
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

bool aligned_rows(const uint8_t* p, int64_t ld, int64_t to) {
  return ld % to == 0 && (reinterpret_cast<uintptr_t>(p) & (to - 1)) == 0 && ld < kMaxPitch;
}

// The copies that the operands need, from `at` of the workspace on; a takes them.
int lay_out(MxArgs& a, int64_t& at, Copies& all) {
  int count = 0;
  auto need = [&](const uint8_t*& p, int64_t& ld, int64_t rows, int bytes, int64_t to) {
    if (aligned_rows(p, ld, to)) return;
    uint8_t* const dst = a.workspace + at;
    all.c[count++] = {p, ld, dst, rows, bytes};
    p = dst;
    ld = copy_pitch(bytes);
    at += rows * ld;
  };
  need(a.a, a.lda, a.T, a.n / 2, 16);
  need(a.scale, a.lds, a.T, a.n / 32, 4);
  need(a.w, a.ldw, a.R, a.n / 2, 16);
  need(a.w_scale, a.ldws, a.R, a.n / 32, 4);
  return count;
}

int64_t partial_bytes(const MxArgs& a) {
  const Plan p = tile_plan(a.T, a.n, a.R);
  if (p.splits == 1) return 0;
  const TileCost& t = kTiles[p.kind];
  const int64_t tiles = static_cast<int64_t>((a.T + t.bm - 1) / t.bm) * ((a.R + t.bn - 1) / t.bn);
  return tiles * p.splits * t.bm * t.bn * 4;
}

}  // namespace

int64_t mx_workspace(const MxArgs& a) {
  if (a.T == 0 || a.R == 0) return 0;
  MxArgs b = a;
  b.workspace = nullptr;
  Copies all;
  int64_t at = partial_bytes(a);
  lay_out(b, at, all);
  return at;
}

const char* mx_name(const MxArgs& a) {
  static const char* const names[] = {"mx_tile256x256", "mx_tile128x128", "mx_tile64x128", "mx_tile64x64"};
  return names[tile_plan(a.T, a.n, a.R).kind];
}

hipError_t launch_mx(const MxArgs& args, hipStream_t s) {
  MxArgs a = args;
  const Plan plan = tile_plan(a.T, a.n, a.R);
  Copies all = {};
  int64_t at = partial_bytes(a);
  const int copies = lay_out(a, at, all);
  if (copies > 0) {
    mx_copy_kernel<<<dim3(1024, static_cast<unsigned>(copies)), 256, 0, s>>>(all);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  switch (plan.kind) {
    case 0: return run_tile<4, 2, 4, 8, 1>(a, plan.splits, s);
    case 1: return run_tile<2, 2, 4, 4, 2>(a, plan.splits, s);
    case 2: return run_tile<2, 2, 4, 2, 2>(a, plan.splits, s);
    default: return run_tile<1, 4, 4, 1, 2>(a, plan.splits, s);
  }
}

}  // namespace signrot
