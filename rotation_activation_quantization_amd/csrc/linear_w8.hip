// The products on 8-bit weights: per-token INT8 codes (W8A8), or the rotated
// INT4 codes with their zero-points (W8A4), times INT8 weights with one scale
// per output channel,
//
//   out[t][k] = scale[t] v[k] (sum_j q[t][j] w[k][j] - zero[t] wsum[k]) + b[k]
//
// (zero = 0 for W8A8).  The sum runs on v_mfma_i32_16x16x64_i8 and is exact.
// The weights are the MFMA's A operand and the tokens its B operand, so that a
// lane's four results are consecutive output channels of one token.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>
#include <string.h>

#include "internal.h"
#include "row_ops.h"
#include "wave_ops.h"

namespace signrot {
namespace {

typedef __attribute__((__vector_size__(4 * sizeof(int32_t)))) int32_t i32x4_t;

constexpr int kCus = 256;  // of an MI355X: the plans do not depend on the device asked

// Eight packed INT4 codes (code 2i in the low nibble of byte i) as eight
// bytes in channel order.
__device__ __forceinline__ void widen8(uint32_t c, uint32_t& r0, uint32_t& r1) {
  const uint32_t lo = c & 0x0F0F0F0Fu, hi = (c >> 4) & 0x0F0F0F0Fu;
  r0 = __builtin_amdgcn_perm(hi, lo, 0x05010400u);
  r1 = __builtin_amdgcn_perm(hi, lo, 0x07030602u);
}

__device__ __forceinline__ float finish(const W8Args& a, int t, int k, int32_t acc) {
  float v = static_cast<float>(acc);
  if (a.a4) v = fmaf(-a.zero[t], static_cast<float>(a.w_sum[k]), v);
  return fmaf(v * a.scale[t], a.w_scale[k], a.bias ? a.bias[k] : 0.f);
}

// Results of token t from channel k on: vectors at whatever address they have
// (the output's rows need not be aligned; 2048 x 4096 x 4094 took 58.7 us with
// single elements there, 40.0 so), single ones at the row's end.
template <int N>
__device__ __forceinline__ void store_results(const W8Args& a, int t, int k, const float (&o)[N], bool whole) {
  const int64_t at = static_cast<int64_t>(t) * a.ldo + k;
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
    for (int e = 0; e < N; e += 4)
      row::store_as<false>(out + e, wave::f32x4_t{o[e], o[e + 1], o[e + 2], o[e + 3]});
  } else {
#pragma unroll
    for (int e = 0; e < N; ++e)
      if (k + e < a.R) row::store_elem(a.out, at + e, o[e], a.out_bf16);
  }
}

// ---- large tiles ------------------------------------------------------------
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

constexpr int kDeep = 64;  // k of one MFMA

// WK x WT waves of FK x FT 16 x 16 results each, a ring of S steps of KU
// MFMAs' depth.
template <bool A4, int WK, int WT, int FK, int FT, int KU, int S>
struct Tile {
  static constexpr int kStep = KU * kDeep;                // k per step
  static constexpr int kWaves = WK * WT;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kBN = 16 * WK * FK;                // channels
  static constexpr int kBM = 16 * WT * FT;                // tokens
  static constexpr int kTokRow = A4 ? kDeep / 2 : kDeep;  // bytes of a token row and MFMA
  // LDS bytes of one MFMA's depth, its 1 KiB loads, and the loads per wave and step
  static constexpr int kWDeep = kBN * kDeep, kTDeep = kBM * kTokRow;
  static constexpr int kWBlocks = kWDeep / 1024, kTBlocks = kTDeep / 1024;
  static constexpr int kWLoads = KU * kWBlocks / kWaves, kTLoads = KU * kTBlocks / kWaves;
  static constexpr int kLoads = kWLoads + kTLoads;
  static constexpr int kWStage = KU * kWDeep, kTStage = KU * kTDeep;
  static constexpr int kPart = 256 * FK * FT * kWaves;  // int32 of a tile's partial sums
  // work-groups to a CU: as many as its LDS holds, at most eight waves
  static constexpr int kLds = S * (kWStage + kTStage);
  static constexpr int kFit = 160 * 1024 / kLds < 8 / kWaves ? 160 * 1024 / kLds : 8 / kWaves;
  static_assert(kWLoads * kWaves == KU * kWBlocks && kTLoads * kWaves == KU * kTBlocks, "whole loads per wave");
  static_assert(kWBlocks * 1024 == kWDeep && kTBlocks * 1024 == kTDeep, "whole loads");
  static_assert(FK % 4 == 0, "a lane's channels come in sixteens");
  static_assert(KU == 1 || KU % 2 == 0, "the token operands alternate");
  // The factors of a tile's results are there before its stores, since a load
  // after a store waits for the store: in registers where those are free (512 x
  // 4096 x 4096: 12.8 us, 13.9 loaded between the stores), else (64 x 128
  // results a wave, where registers would spill: 421 us at 8192 x 4096 x 14336)
  // in LDS, loaded with the tile's first step (395; 404 between the stores).
  // Two copies, since waves enter the next tile on their own.
  static constexpr bool kFactorsInLds = FK * FT >= 32;
  static constexpr int kFactors = kFactorsInLds ? 3 * kBN + 2 * kBM : 0;  // w_scale, scale, w_sum, zero, bias
  static_assert(!kFactorsInLds || (kBN == 256 && kBM == 256 && kWaves == 8 && kLds + 8 * kFactors <= 160 * 1024),
                "a wave loads 64 channels or 64 tokens");
  static_assert(S >= 4 && kFit > 0, "ring");
};

// Both operands stream global -> LDS (16 bytes a lane, no registers) through a
// ring of S k steps; one barrier a step.  Step s: the MFMAs of step s, the
// loads of step s + S - 1 into the buffers step s - 1 used, and towards its
// end the first operand reads of step s + 1 (which has landed: the barrier at
// the end of step s - 1 came after every wave's wait for it).
//
// A work-group takes the tiles p, p + stride, ... below `end`, and the ring
// runs on from tile to tile: the last steps of a tile load the first ones of
// the next, which arrive while its results are scaled and stored.
//
// Step 0 of a tile is the last, possibly short one of the row: its chunks
// beyond n are read as chunk 0 and the token operand is zeroed there.
//
// LDS rows of 64 bytes, four 16-byte chunks: logical chunk c of row r sits at
// physical chunk c ^ 2 ((r >> 3) & 1).  A 16-byte LDS read serves sixteen lanes
// at a time, among them lanes 0-3 and 12-15 of one group of sixteen with 4-11 of
// the next; rows 4 apart share banks, and this swizzle gives those lanes
// four chunks of their own (SQ_LDS_BANK_CONFLICT reads zero; c ^ ((r >> 2) & 3)
// cost 4 cycles a read).  A lane (g = lane / 16,
// i = lane % 16) reads row i, chunk g of a 16-row group: k = 16 g .. 16 g + 15
// of the step for both operands.  The packed codes (32 bytes a row) are kept
// per 16-row group as the first 16 bytes of every row, then the second; a lane
// reads its 8 bytes there and widens them in registers.
//
// 8192 x 14336 x 4096 runs 359 us, 2.7 POP/s (W8A4 379 us), with the MFMAs 68 %
// (61 %) busy.  The clock bounds it: the same instructions on zeros take 278 us
// (300).
//
// Slot 16 f + i of a 64-channel group holds channel 16 (i / 4) + 4 f + i % 4:
// the four 16 x 16 results f = 0 .. 3 then leave a lane sixteen consecutive
// channels of a token, stored as whole vectors.
template <bool A4, int WK, int WT, int FK, int FT, int KU, int S, bool SPLIT>
__device__ __forceinline__ void w8_tile(const W8Args& a, int tiles_m, int tiles_n, int splits) {
  using C = Tile<A4, WK, WT, FK, FT, KU, S>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[C::kLds + (SPLIT ? 0 : 8 * C::kFactors)];
  uint8_t* const lds_w = lds;
  uint8_t* const lds_t = lds + S * C::kWStage;
  float* const factors = reinterpret_cast<float*>(lds + C::kLds);
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
  const int steps = (a.n + C::kStep - 1) / C::kStep;
  const int tail = a.n - (steps - 1) * C::kStep;  // k of step 0
  // part j of a row: steps first(j) .. first(j + 1) - 1
  auto first = [&](int j) { return static_cast<int>(static_cast<int64_t>(steps) * j / splits); };

  // What is loaded next: step ik of item src_p.  Rows beyond the tensor are
  // clamped (their results are not stored).
  // Load l of a wave is block kLoads * wave + l of the step's, counted through
  // the depths: sixteen rows of weights or tokens (32 of packed codes).
  const int chunk_w = (lane & 3) ^ (2 * (lane >> 5));  // logical chunk of the lane's slot: row lane / 4 of 16
  const int chunk_t = A4 ? (g & 1) : chunk_w;
  auto depth_w = [&](int l) { return (C::kWLoads * wid + l) / C::kWBlocks; };
  auto depth_t = [&](int l) { return (C::kTLoads * wid + l) / C::kTBlocks; };
  // what a chunk beyond n is moved back by in the short step: to chunk 0
  auto cut_w = [&](int l) {
    const int k = kDeep * depth_w(l) + 16 * chunk_w;
    return k >= tail ? static_cast<uint32_t>(k) : 0u;
  };
  auto cut_t = [&](int l) {
    const int k = kDeep * depth_t(l) + (A4 ? 32 : 16) * chunk_t;
    return k >= tail ? static_cast<uint32_t>(A4 ? k / 2 : k) : 0u;
  };
  int src_p = p, ik, ik_end;
  const int8_t* base_w;
  const uint8_t* base_t;
  uint32_t size_w, size_t_, off_w[C::kWLoads], off_t[C::kTLoads];
  auto set_source = [&]() {
    const int part = SPLIT ? src_p / tiles : 0;
    ik = __builtin_amdgcn_readfirstlane(first(part));
    ik_end = __builtin_amdgcn_readfirstlane(first(part + 1));
    int tm, tn;
    tile_at(src_p - part * tiles, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * C::kBM, n0 = tn * C::kBN;
    const bool cut = ik == 0 && tail < C::kStep;
    const int rows_w = min(C::kBN, a.R - n0), rows_t = min(C::kBM, a.T - m0);
    base_w = a.w + static_cast<int64_t>(n0) * a.ldw;
    base_t = a.a + static_cast<int64_t>(m0) * a.lda;
    size_w = static_cast<uint32_t>(rows_w - 1) * static_cast<uint32_t>(a.ldw) + a.n;
    size_t_ = static_cast<uint32_t>(rows_t - 1) * static_cast<uint32_t>(a.lda) + a.row_bytes;
#pragma unroll
    for (int l = 0; l < C::kWLoads; ++l) {
      const int slot = 16 * ((C::kWLoads * wid + l) % C::kWBlocks) + (lane >> 2);
      const int at = slot & 15;
      const int ch = (slot & ~63) + 16 * (at >> 2) + 4 * ((slot >> 4) & 3) + (at & 3);
      off_w[l] = static_cast<uint32_t>(min(ch, rows_w - 1)) * static_cast<uint32_t>(a.ldw) + kDeep * depth_w(l) +
                 16 * chunk_w - (cut ? cut_w(l) : 0);
    }
#pragma unroll
    for (int l = 0; l < C::kTLoads; ++l) {
      const int block = (C::kTLoads * wid + l) % C::kTBlocks;
      const int r = A4 ? 32 * block + 16 * (lane >> 5) + i : 16 * block + (lane >> 2);
      off_t[l] = static_cast<uint32_t>(min(r, rows_t - 1)) * static_cast<uint32_t>(a.lda) + C::kTokRow * depth_t(l) +
                 16 * chunk_t - (cut ? cut_t(l) : 0);
    }
  };
  int wr_w = 0, wr_t = 0;  // ring position that is filled
  int ks;                  // k of step ik, in steps
  auto issue = [&](int l) {
    if (l < C::kWLoads) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          wave::buffer_rsrc(base_w, size_w),
          (__attribute__((address_space(3))) void*)(lds_w + wr_w + 1024 * (C::kWLoads * wid + l)), 16,
          off_w[l], C::kStep * ks, 0, 0);
    } else {
      const int j = l - C::kWLoads;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          wave::buffer_rsrc(base_t, size_t_),
          (__attribute__((address_space(3))) void*)(lds_t + wr_t + 1024 * (C::kTLoads * wid + j)), 16,
          off_t[j], KU * C::kTokRow * ks, 0, 0);
    }
  };
  auto block_of = [&](int step) { return __builtin_amdgcn_readfirstlane(step == 0 ? steps - 1 : step - 1); };
  // Past the last item the loads go on with that item's: every step issues the
  // same number, so the vmcnt threshold is exact.
  auto issued = [&]() {
    wr_w = wr_w == (S - 1) * C::kWStage ? 0 : wr_w + C::kWStage;
    wr_t = wr_t == (S - 1) * C::kTStage ? 0 : wr_t + C::kTStage;
    if (ik == 0 && tail < C::kStep) {
#pragma unroll
      for (int l = 0; l < C::kWLoads; ++l) off_w[l] += cut_w(l);
#pragma unroll
      for (int l = 0; l < C::kTLoads; ++l) off_t[l] += cut_t(l);
    }
    ik = __builtin_amdgcn_readfirstlane(ik + 1);
    if (ik == ik_end) {
      src_p = src_p + stride < end ? src_p + stride : src_p;
      set_source();
    }
    ks = block_of(ik);
  };

  const int read_w = (64 * wk * FK / 4) * kDeep + i * kDeep + 16 * (g ^ (2 * (i >> 3)));
  const int read_t = A4 ? 512 * (wt * FT) + 256 * (g >> 1) + 16 * i + 8 * (g & 1)
                        : 16 * wt * FT * kDeep + i * kDeep + 16 * (g ^ (2 * (i >> 3)));
  int rd_w = 0, rd_t = 0;  // ring position that is multiplied
  auto weight = [&](int at, int f) {
    return *reinterpret_cast<const i32x4_t*>(lds_w + at + read_w + 16 * kDeep * f);
  };

  i32x4_t acc[FK][FT];
  i32x4_t tok[2][FT];  // token operands of this and the next step
  wave::u32x2_t code[FT];
  auto read_token = [&](int at, int j, i32x4_t& dst) {
    const uint8_t* s = lds_t + at + read_t;
    if (A4)
      code[j] = *reinterpret_cast<const wave::u32x2_t*>(s + 512 * j);
    else
      dst = *reinterpret_cast<const i32x4_t*>(s + 16 * kDeep * j);
  };
  auto widen = [&](int j, i32x4_t& dst) {
    uint32_t w0, w1, w2, w3;
    widen8(code[j][0], w0, w1);
    widen8(code[j][1], w2, w3);
    dst = i32x4_t{static_cast<int>(w0), static_cast<int>(w1), static_cast<int>(w2), static_cast<int>(w3)};
    asm volatile("" : "+v"(dst));  // here, not where the next step uses it
  };

  set_source();
  ks = block_of(ik);
  for (int s = 0; s < S - 1; ++s) {
#pragma unroll
    for (int l = 0; l < C::kLoads; ++l) issue(l);
    issued();
  }
  wave::wait_vmcnt<(S - 3) * C::kLoads>();
  __builtin_amdgcn_s_barrier();
  i32x4_t wf[FK + 2];
  wf[0] = weight(0, 0);
  wf[1] = weight(0, 1);
#pragma unroll
  for (int j = 0; j < FT; ++j) {
    read_token(0, j, tok[0][j]);
    if (A4) widen(j, tok[0][j]);
  }

  // MFMA depth u of a step
  auto deep = [&](int u, int nx_w, int nx_t, i32x4_t (&now)[FT], i32x4_t (&next)[FT]) {
#pragma unroll
    for (int f = 0; f < FK; ++f) {
      // The reads follow the block's first MFMA: the wait before that one is
      // then for reads a whole block old.
      acc[f][0] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[f], now[0], acc[f][0], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      // two reads ahead, the last two from the next depth or step
      wf[f + 2] = f + 2 < FK ? weight(rd_w + u * C::kWDeep, f + 2) : weight(nx_w, f + 2 - FK);
      // the next depth's tokens: packed codes are read over the first half of
      // the blocks and widened, between the MFMAs, over the second
      constexpr int kOver = A4 ? FK / 2 : FK;
      if (f < kOver) {
#pragma unroll
        for (int j = f * FT / kOver; j < (f + 1) * FT / kOver; ++j) read_token(nx_t, j, next[j]);
      } else {
#pragma unroll
        for (int j = (f - kOver) * FT / kOver; j < (f - kOver + 1) * FT / kOver; ++j) widen(j, next[j]);
      }
      constexpr int kBlocks = KU * FK;
      const int b = u * FK + f;
#pragma unroll
      for (int l = 0; l < C::kLoads; ++l)
        if (l >= b * C::kLoads / kBlocks && l < (b + 1) * C::kLoads / kBlocks) issue(l);
#pragma unroll
      for (int j = 1; j < FT; ++j)
        acc[f][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[f], now[j], acc[f][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    wf[0] = wf[FK];
    wf[1] = wf[FK + 1];
  };
  // zeros in place of the k beyond n: depth u of the short step
  auto mask = [&](int u, i32x4_t (&t)[FT]) {
#pragma unroll
    for (int j = 0; j < FT; ++j)
      if (kDeep * u + 16 * g >= tail) t[j] = i32x4_t{0, 0, 0, 0};
  };
  // A step begins with tok[0] and, of odd depth, ends with the next one's in tok[1].
  auto step = [&](i32x4_t (&t0)[FT], i32x4_t (&t1)[FT], bool cut) {
    const int nx_w = rd_w == (S - 1) * C::kWStage ? 0 : rd_w + C::kWStage;
    const int nx_t = rd_t == (S - 1) * C::kTStage ? 0 : rd_t + C::kTStage;
#pragma unroll
    for (int u = 0; u < KU; ++u) {
      i32x4_t(&now)[FT] = u & 1 ? t1 : t0;
      i32x4_t(&next)[FT] = u & 1 ? t0 : t1;
      if (cut) mask(u, now);
      deep(u, u + 1 < KU ? rd_w + (u + 1) * C::kWDeep : nx_w, u + 1 < KU ? rd_t + (u + 1) * C::kTDeep : nx_t, now,
           next);
    }
    rd_w = nx_w;
    rd_t = nx_t;
    issued();
    wave::wait_vmcnt<(S - 3) * C::kLoads>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };

  int copy = 0;
  for (; p < end; p += stride) {
    int tm, tn;
    tile_at(SPLIT ? p % tiles : p, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * C::kBM, n0 = tn * C::kBN;
    if (C::kFactorsInLds && !SPLIT) {
      // Landed after the tile's first step: its wait leaves only later loads,
      // and its barrier comes after every wave's.
      copy ^= 1;
      const bool ch = wid < 4;
      const int rows = ch ? min(C::kBN, a.R - n0) : min(C::kBM, a.T - m0);
      const uint32_t at = 4 * min(64 * (wid & 3) + lane, rows - 1);
      auto fill = [&](const void* src, int to) {
        __builtin_amdgcn_raw_ptr_buffer_load_lds(
            wave::buffer_rsrc(static_cast<const uint32_t*>(src) + (ch ? n0 : m0), 4 * static_cast<uint32_t>(rows)),
            (__attribute__((address_space(3))) void*)(factors + copy * C::kFactors + to + 64 * wid), 4, at, 0, 0, 0);
      };
      fill(ch ? static_cast<const void*>(a.w_scale) : static_cast<const void*>(a.scale), 0);
      if (A4) fill(ch ? static_cast<const void*>(a.w_sum) : static_cast<const void*>(a.zero), C::kBN + C::kBM);
      if (a.bias && ch) fill(a.bias, 2 * (C::kBN + C::kBM));
    }
#pragma unroll
    for (int f = 0; f < FK; ++f)
#pragma unroll
      for (int j = 0; j < FT; ++j) acc[f][j] = i32x4_t{0, 0, 0, 0};
    const int part = SPLIT ? p / tiles : 0;
    const int count = first(part + 1) - first(part);
    bool cut = part == 0 && tail < C::kStep;  // the item begins with the short step
    if (KU % 2 == 0) {
      for (int kt = 0; kt < count; ++kt) {
        step(tok[0], tok[1], cut);
        cut = false;
      }
    } else {
      if (cut) mask(0, tok[0]);
      for (int kt = 1; kt < count; kt += 2) {
        step(tok[0], tok[1], false);
        step(tok[1], tok[0], false);
      }
      if (count & 1) {
        step(tok[0], tok[1], false);
#pragma unroll
        for (int j = 0; j < FT; ++j) tok[0][j] = tok[1][j];
      }
    }

    if (SPLIT) {
      // partial sums in operand order, [part][tile][wave][f][j][lane]
      i32x4_t* const out = reinterpret_cast<i32x4_t*>(a.partial) +
                           (static_cast<int64_t>(p) * C::kPart + 256 * FK * FT * wid) / 4 + lane;
#pragma unroll
      for (int f = 0; f < FK; ++f)
#pragma unroll
        for (int j = 0; j < FT; ++j) out[64 * (FT * f + j)] = acc[f][j];
      continue;
    }

    // Lane (g, i): token 16 j + i, channels 16 g .. 16 g + 15 of every 64.  The
    // factors come before the stores: a load after a store waits for the store.
    const float* const fac = factors + copy * C::kFactors;
    float sc[FT], z[FT];
    if (!C::kFactorsInLds) {
#pragma unroll
      for (int j = 0; j < FT; ++j) {
        const int t = min(m0 + 16 * (wt * FT + j) + i, a.T - 1);
        sc[j] = a.scale[t];
        z[j] = A4 ? a.zero[t] : 0.f;
      }
    }
#pragma unroll
    for (int q = 0; q < FK / 4; ++q) {
      const int k0 = n0 + 16 * wk * FK + 64 * q + 16 * g;
      if (k0 >= a.R) continue;
      const bool whole = k0 + 16 <= a.R;
      float v[16], b[16], ws[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int k = C::kFactorsInLds ? k0 - n0 + e : min(k0 + e, a.R - 1);
        v[e] = C::kFactorsInLds ? fac[k] : a.w_scale[k];
        ws[e] = 0.f;
        if (A4)
          ws[e] = static_cast<float>(C::kFactorsInLds ? __float_as_int(fac[C::kBN + C::kBM + k]) : a.w_sum[k]);
        b[e] = 0.f;
      }
      if (a.bias) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          b[e] = C::kFactorsInLds ? fac[2 * (C::kBN + C::kBM) + k0 - n0 + e] : a.bias[min(k0 + e, a.R - 1)];
      }
#pragma unroll
      for (int j = 0; j < FT; ++j) {
        const int t = m0 + 16 * (wt * FT + j) + i;
        if (t >= a.T) continue;
        const float scale = C::kFactorsInLds ? fac[C::kBN + t - m0] : sc[j];
        const float zero = !A4 ? 0.f : C::kFactorsInLds ? fac[2 * C::kBN + C::kBM + t - m0] : z[j];
        float o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float x = static_cast<float>(acc[4 * q + (e >> 2)][j][e & 3]);
          if (A4) x = fmaf(-zero, ws[e], x);
          o[e] = fmaf(x * scale, v[e], b[e]);
        }
        store_results(a, t, k0, o, whole);
      }
    }
  }
  wave::wait_vmcnt<0>();
}

template <bool A4, int WK, int WT, int FK, int FT, int KU, int S, bool SPLIT>
__global__ __launch_bounds__(64 * WK * WT) __attribute__((
    amdgpu_waves_per_eu(Tile<A4, WK, WT, FK, FT, KU, S>::kWaves * Tile<A4, WK, WT, FK, FT, KU, S>::kFit / 4)))
void w8_tile_kernel(W8Args a, int tiles_m, int tiles_n, int splits) {
  w8_tile<A4, WK, WT, FK, FT, KU, S, SPLIT>(a, tiles_m, tiles_n, SPLIT ? splits : 1);
}

// Sums the parts of a tile's results and finishes them: a thread takes one
// lane's four channels of a 16 x 16 result.
template <bool A4, int WK, int WT, int FK, int FT, int KU, int S>
__global__ __launch_bounds__(256) void w8_join_kernel(W8Args a, int tiles_m, int tiles_n, int splits) {
  using C = Tile<A4, WK, WT, FK, FT, KU, S>;
  const int tiles = tiles_m * tiles_n;
  const int64_t e = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;  // i32x4 of a part
  const int tile = static_cast<int>(e / (C::kPart / 4));
  const int at = static_cast<int>(e - static_cast<int64_t>(tile) * (C::kPart / 4));
  const int lane = at & 63, j = (at >> 6) % FT, f = (at >> 6) / FT % FK, wid = (at >> 6) / (FT * FK);
  int tm, tn;
  tile_at(tile, tiles_m, tiles_n, tm, tn);
  const int t = tm * C::kBM + 16 * ((wid / WK) * FT + j) + (lane & 15);
  const int k = tn * C::kBN + 16 * (wid % WK) * FK + 64 * (f >> 2) + 16 * (lane >> 4) + 4 * (f & 3);
  if (t >= a.T || k >= a.R) return;
  const i32x4_t* src = reinterpret_cast<const i32x4_t*>(a.partial) + e;
  const int64_t pitch = static_cast<int64_t>(tiles) * (C::kPart / 4);
  i32x4_t sum = src[0];
  for (int s = 1; s < splits; ++s) sum += src[s * pitch];
  float o[4];
#pragma unroll
  for (int c = 0; c < 4; ++c) o[c] = finish(a, t, min(k + c, a.R - 1), sum[c]);
  store_results(a, t, k, o, k + 4 <= a.R);
}

template <bool A4, int WK, int WT, int FK, int FT, int KU, int S>
hipError_t run_tile(const W8Args& a, int splits, hipStream_t s) {
  using C = Tile<A4, WK, WT, FK, FT, KU, S>;
  const int tiles_m = (a.T + C::kBM - 1) / C::kBM, tiles_n = (a.R + C::kBN - 1) / C::kBN;
  const int items = tiles_m * tiles_n * splits;
  const int most = (device_cu_count() & ~7) * C::kFit;
  const dim3 grid(static_cast<unsigned>(most > 0 && items > most ? most : items)), block(C::kThreads);
  if (splits == 1) {
    w8_tile_kernel<A4, WK, WT, FK, FT, KU, S, false><<<grid, block, 0, s>>>(a, tiles_m, tiles_n, 1);
    return hipGetLastError();
  }
  w8_tile_kernel<A4, WK, WT, FK, FT, KU, S, true><<<grid, block, 0, s>>>(a, tiles_m, tiles_n, splits);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  w8_join_kernel<A4, WK, WT, FK, FT, KU, S>
      <<<dim3(static_cast<unsigned>(tiles_m * tiles_n * (C::kPart / 1024))), dim3(256), 0, s>>>(a, tiles_m, tiles_n,
                                                                                              splits);
  return hipGetLastError();
}

// The tiles there are, and what they cost: microseconds for 128 of k with one
// work-group on a CU and with two side by side, and for a tile's start and
// stores, fitted to 714 timings of 25 shapes (40 x 4096 x 4096 to 8192 x 1024 x
// 1024; 10 % rms) beside the call's 4 us.  The least estimate picked the fastest
// of the timed choices or one within 3 % of it, 0.5 % off on average, but with
// weights that no cache holds it is further off at 64 x 14336 x 4096 (W8A8 20.6
// and 18.3 us) and 64 x 28672 x 8192 (53.4 and 49.3).  Both operands of
// the smaller tiles come a whole 128-byte line a row and step (KU = 2): 512 x
// 4096 x 4096 took 19.8 us with 64 bytes a step, 13.9 with 128 (12.8 now, see
// the factors above).
struct TileCost {
  int bm, bn, step, fit;
  double one, two, tile;
};
constexpr TileCost kTiles8[] = {{256, 256, 64, 1, 1.35, 0, 2.8},   // 4 x 2 waves of 64 channels x 128 tokens
                                {128, 128, 128, 1, 0.453, 0, 1.4},  // 2 x 2 waves of 64 x 64
                                {64, 128, 128, 1, 0.280, 0, 1.2},   // 2 x 2 waves of 64 x 32
                                {64, 64, 128, 2, 0.184, 0.341, 1.4},  // 1 x 4 waves of 64 x 16
                                {64, 64, 256, 1, 0.176, 0, 1.3}};   // the same, 256 of k a step
constexpr TileCost kTiles4[] = {{256, 256, 64, 1, 1.44, 0, 3.7},   // 2 x 4 waves of 128 x 64: codes are widened twice
                                {128, 128, 128, 1, 0.535, 0, 1.7},  // 2 x 4 waves of 64 x 32
                                {128, 64, 128, 1, 0.308, 0, 1.2},   // 1 x 4 waves of 64 x 32
                                {64, 64, 128, 2, 0.238, 0.363, 1.7},
                                {64, 64, 256, 1, 0.187, 0, 1.5}};

struct Plan {
  int kind, splits;
  double us;
};

// The least estimate over the tiles and over parts of the row joined by a
// second kernel (3.5 us, and 3.3 TB/s over the partial sums).  Where the bytes bound
// several of them their estimates are equal, and the first in the table stays
// unless another's own work is less by a tenth, the fit's error: W8A8 64 x 128 for
// 128 x 128 at 33 x 2048 x 28672 (14.5 us, 17.3) and 64 x 14336 x 28672 (78.7,
// 81.1), 64 x 64 for 64 x 128 in two parts at 64 x 28672 x 8192 (51.9, 70.7), W8A4
// 256 of k a step for 128 at 64 x 14336 x 14336 (41.2, 45.5).  Of W8A8 choices closer than
// that the first is the faster one as often as not (64 x 8192 x 5120 14.6 us, the other
// 16.0; 33 x 13824 x 11008 36.1 and 34.8).
Plan tile_plan(int64_t T, int64_t n, int64_t R, bool a4) {
  Plan best{0, 1, 1e30};
  double best_work = 1e30;
  const double bytes = static_cast<double>(R) * n + (a4 ? 0.5 : 1.0) * T * n + 2.0 * T * R;
  for (int c = 0; c < 5; ++c) {
    const TileCost& t = a4 ? kTiles4[c] : kTiles8[c];
    const double tiles = static_cast<double>((T + t.bm - 1) / t.bm) * static_cast<double>((R + t.bn - 1) / t.bn);
    for (const int splits : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (splits > 1 && (splits > (n + t.step - 1) / t.step || tiles * splits > 4 * kCus)) break;
      const double per_cu = ceil(tiles * splits / kCus);
      const double k = n / 128.0 / splits;
      double us = t.fit == 1 ? per_cu * (k * t.one + t.tile)
                             : floor(per_cu / 2) * (k * t.two + t.tile) + fmod(per_cu, 2) * (k * t.one + t.tile);
      const double join = splits > 1 ? 3.5 + tiles * splits * t.bm * t.bn * 4 / 3.3e6 : 0;
      const double work = us + join;
      us = fmax(us, bytes / 7e6) + join;
      if (us < best.us || (us == best.us && work < 0.9 * best_work)) {
        best = {c, splits, us};
        best_work = work;
      }
    }
  }
  return best;
}

// ---- few tokens ---------------------------------------------------------------
//
// The weights are read once and bound the time (16 x 28672 x 8192: 43 us, 5.4
// TB/s).  A work-group takes sixteen
// channels and all tokens (FT groups of sixteen); its waves share the row:
// wave w takes the 128-byte units w, w + waves, ... of k, so that the
// work-group reads sixteen rows side by side.  Each wave has a ring of D units
// of its own in LDS and waits for its own loads only; the partial sums meet in
// LDS at the end.
//
// The loads go through LDS, and not straight into the operand registers,
// because a lane (g, i) holds 16 bytes of row i: sixteen neighbouring lanes
// would read sixteen rows, 64 cache accesses an instruction instead of eight
// whole lines, and with many in flight a line's second half came back from L2
// again (1.3 M requests for 0.9 M lines at 16 x 14336 x 4096).
//
// LDS rows of 128 bytes: chunk c of row r sits at chunk c ^ h(r),
// h(r) = (r & 7) ^ ((r >> 3) & 1); of 64 bytes (packed codes): c ^ 2 ((r >> 3) & 1).
// Either way the sixteen lanes a 16-byte read serves at a time cover the 64
// banks once.
constexpr int kUnit = 128;

// The waves' partial sums [wave][FK][FT][64][4] joined and finished: result e is
// channel e % 4 + 4 (e / 64 % 4) of group e / 256 / FT, token e / 4 % 16 of
// group e / 256 % FT.
template <int FK, int FT>
__device__ __forceinline__ void few_finish(const W8Args& a, const int32_t* part, int n0, int waves) {
  for (int e = threadIdx.x; e < 256 * FK * FT; e += blockDim.x) {
    const int k = n0 + 16 * ((e >> 8) / FT) + (e & 3) + 4 * ((e >> 6) & 3);
    const int t = 16 * ((e >> 8) % FT) + ((e >> 2) & 15);
    if (k >= a.R || t >= a.T) continue;
    int32_t sum = part[e];
    for (int v = 1; v < waves; ++v) sum += part[256 * FK * FT * v + e];
    row::store_elem(a.out, static_cast<int64_t>(t) * a.ldo + k, finish(a, t, k, sum), a.out_bf16);
  }
}

template <bool A4, int FK, int FT, int D>
struct Few {
  static constexpr int kTokRow = A4 ? kUnit / 2 : kUnit;
  static constexpr int kWBytes = 16 * FK * kUnit;
  static constexpr int kTBytes = 16 * FT * kTokRow;
  static constexpr int kWLoads = kWBytes / 1024, kTLoads = kTBytes / 1024;
  static constexpr int kLoads = kWLoads + kTLoads;
  static constexpr int kRing = D * (kWBytes + kTBytes);  // bytes of a wave
  static constexpr int kPart = 1024 * FK * FT;                // bytes of a wave's partial sums
};

template <bool A4, int FK, int FT, int D>
__device__ __forceinline__ void w8_few(const W8Args& a, uint8_t* lds) {
  using C = Few<A4, FK, FT, D>;
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int g = lane >> 4, i = lane & 15;
  const int n0 = 16 * FK * blockIdx.x;
  const int units = (a.n + kUnit - 1) / kUnit;
  const int tail = a.n - (units - 1) * kUnit;  // k of the row's last unit
  const int count = units > wid ? (units - wid - 1) / waves + 1 : 0;
  uint8_t* const ring_w = lds + wid * C::kRing;
  uint8_t* const ring_t = ring_w + D * C::kWBytes;
  int32_t* const part = reinterpret_cast<int32_t*>(lds + waves * C::kRing);

  // rows and tokens beyond the tensors are clamped (their results are not stored)
  const int rows_w = min(16 * FK, a.R - n0);
  const __amdgpu_buffer_rsrc_t src_w =
      wave::buffer_rsrc(a.w + static_cast<int64_t>(n0) * a.ldw,
                        static_cast<uint32_t>(rows_w - 1) * static_cast<uint32_t>(a.ldw) + a.n);
  const __amdgpu_buffer_rsrc_t src_t = wave::buffer_rsrc(
      a.a, static_cast<uint32_t>(a.T - 1) * static_cast<uint32_t>(a.lda) + a.row_bytes);
  auto h = [](int r) { return (r & 7) ^ ((r >> 3) & 1); };
  // sources of the lane: load l of the weights fills rows 8 l .. 8 l + 7
  uint32_t off_w[C::kWLoads], off_t[C::kTLoads];
  int chunk_w[C::kWLoads], chunk_t[C::kTLoads];
#pragma unroll
  for (int l = 0; l < C::kWLoads; ++l) {
    const int r = 8 * l + (lane >> 3);
    chunk_w[l] = (lane & 7) ^ h(r & 15);
    off_w[l] = static_cast<uint32_t>(min(r, rows_w - 1)) * static_cast<uint32_t>(a.ldw);
  }
#pragma unroll
  for (int l = 0; l < C::kTLoads; ++l) {
    const int r = A4 ? 16 * l + (lane >> 2) : 8 * l + (lane >> 3);
    chunk_t[l] = A4 ? (lane & 3) ^ (2 * (lane >> 5)) : (lane & 7) ^ h(r & 15);
    off_t[l] = static_cast<uint32_t>(min(r, a.T - 1)) * static_cast<uint32_t>(a.lda);
  }
  // unit x of this wave into ring slot x % D; in the row's last unit the
  // chunks beyond n are read as chunk 0
  auto issue = [&](int x) {
    const int u = wid + x * waves;
    const int left = u == units - 1 ? tail : kUnit;
    const int slot = x % D;
#pragma unroll
    for (int l = 0; l < C::kWLoads; ++l)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          src_w, (__attribute__((address_space(3))) void*)(ring_w + slot * C::kWBytes + 1024 * l), 16,
          off_w[l] + (16 * chunk_w[l] < left ? 16 * chunk_w[l] : 0), kUnit * u, 0, 0);
#pragma unroll
    for (int l = 0; l < C::kTLoads; ++l)
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          src_t, (__attribute__((address_space(3))) void*)(ring_t + slot * C::kTBytes + 1024 * l), 16,
          off_t[l] + ((A4 ? 32 : 16) * chunk_t[l] < left ? 16 * chunk_t[l] : 0), C::kTokRow * u, 0, 0);
  };

  i32x4_t acc[FK][FT];
#pragma unroll
  for (int f = 0; f < FK; ++f)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[f][j] = i32x4_t{0, 0, 0, 0};
  for (int x = 0; x < min(D, count); ++x) issue(x);
  for (int x = 0; x < count; ++x) {
    if (x + D <= count)
      wave::wait_vmcnt<(D - 1) * C::kLoads>();
    else
      wave::wait_vmcnt<0>();
    __builtin_amdgcn_sched_barrier(0);
    const uint8_t* const sw = ring_w + (x % D) * C::kWBytes;
    const uint8_t* const st = ring_t + (x % D) * C::kTBytes;
    // lane (g, i): chunks 2 g and 2 g + 1 of row i
    i32x4_t w[2][FK], tok[2][FT];
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int f = 0; f < FK; ++f)
        w[s][f] = *reinterpret_cast<const i32x4_t*>(sw + 2048 * f + kUnit * i + 16 * ((2 * g + s) ^ h(i)));
#pragma unroll
    for (int j = 0; j < FT; ++j) {
      if (A4) {
        const i32x4_t c = *reinterpret_cast<const i32x4_t*>(st + 1024 * j + 64 * i + 16 * (g ^ (2 * (i >> 3))));
#pragma unroll
        for (int s = 0; s < 2; ++s) {
          uint32_t b[4];
          widen8(static_cast<uint32_t>(c[2 * s]), b[0], b[1]);
          widen8(static_cast<uint32_t>(c[2 * s + 1]), b[2], b[3]);
          tok[s][j] = i32x4_t{static_cast<int>(b[0]), static_cast<int>(b[1]), static_cast<int>(b[2]),
                              static_cast<int>(b[3])};
        }
      } else {
#pragma unroll
        for (int s = 0; s < 2; ++s)
          tok[s][j] = *reinterpret_cast<const i32x4_t*>(st + 2048 * j + kUnit * i + 16 * ((2 * g + s) ^ h(i)));
      }
    }
    if (wid + x * waves == units - 1 && tail < kUnit) {
#pragma unroll
      for (int s = 0; s < 2; ++s)
#pragma unroll
        for (int f = 0; f < FK; ++f)
          if (16 * (2 * g + s) >= tail) w[s][f] = i32x4_t{0, 0, 0, 0};
    }
#pragma unroll
    for (int s = 0; s < 2; ++s)
#pragma unroll
      for (int f = 0; f < FK; ++f)
#pragma unroll
        for (int j = 0; j < FT; ++j)
          acc[f][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(w[s][f], tok[s][j], acc[f][j], 0, 0, 0);
    // The slot is free once its reads are done; they are not ordered with the loads, and the
    // products that wait for them may be moved behind the barrier.
    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    if (x + D < count) issue(x + D);
  }
#pragma unroll
  for (int f = 0; f < FK; ++f)
#pragma unroll
    for (int j = 0; j < FT; ++j)
      *reinterpret_cast<i32x4_t*>(part + 4 * (((wid * FK + f) * FT + j) * 64 + lane)) = acc[f][j];
  __syncthreads();
  few_finish<FK, FT>(a, part, n0, waves);
}

template <bool A4, int FK, int FT, int D>
__global__ __launch_bounds__(512) void w8_few_kernel(W8Args a) {
  extern __shared__ __attribute__((aligned(16))) uint8_t few_lds[];
  w8_few<A4, FK, FT, D>(a, few_lds);
}

template <bool A4, int FK, int FT, int D>
hipError_t run_few_as(const W8Args& a, hipStream_t s) {
  using C = Few<A4, FK, FT, D>;
  const int groups = (a.R + 16 * FK - 1) / (16 * FK), units = (a.n + kUnit - 1) / kUnit;
  int waves = 8;
  while (waves > 2 && (groups * waves > 8 * kCus || units < waves)) waves /= 2;
  w8_few_kernel<A4, FK, FT, D><<<dim3(static_cast<unsigned>(groups)), dim3(static_cast<unsigned>(64 * waves)),
                             static_cast<unsigned>(waves * (C::kRing + C::kPart)), s>>>(a);
  return hipGetLastError();
}

// Thirty-two channels to a work-group where that leaves one to two of them a
// CU: 16 x 28672 x 8192 43.5 us and 1 x 4096 x 14336 13.8 us against 48.1 and
// 15.3 with sixteen; fewer channels need the work-groups (16 x 14336 x 4096 has
// 256 of sixteen), and 1 x 8192 x 28672 ran 45.0 us with sixteen, 48.9 with
// thirty-two.
template <bool A4>
hipError_t run_few(const W8Args& a, hipStream_t s) {
  if (a.R >= 8192 && a.R <= 16384)
    return a.T <= 16 ? run_few_as<A4, 2, 1, 3>(a, s) : run_few_as<A4, 2, 2, 2>(a, s);
  return a.T <= 16 ? run_few_as<A4, 1, 1, 3>(a, s) : run_few_as<A4, 1, 2, 2>(a, s);
}

constexpr int64_t kMaxPitch = 1 << 23;  // a tile's offsets stay below 2^32

// Rows that start on 16-byte boundaries and end on one.
bool aligned_rows(const W8Args& a) {
  return a.n % (a.a4 ? 32 : 16) == 0 && a.lda % 16 == 0 && a.ldw % 16 == 0 &&
         ((reinterpret_cast<uintptr_t>(a.a) | reinterpret_cast<uintptr_t>(a.w)) & 15u) == 0 && a.lda < kMaxPitch &&
         a.ldw < kMaxPitch;
}

// Up to 32 tokens: 32 x 14336 x 4096 16.9 us, 32 x 4096 x 4096 7.1 us, the best
// tile 17.3 and 10.5.
bool takes_few(int64_t T, int64_t R) { return T <= 32 && R <= (int64_t{1} << 24); }

// ---- any stride and alignment -------------------------------------------------
//
// Rows that are not made of whole, aligned 16-byte chunks cannot go straight to
// LDS.

// The 16 operand bytes (8 of packed codes) from channel j0 on of a row with n
// channels, in two halves so that loads stay in flight: the dwords that hold
// them, moved back where they would pass the row's end, and the shifts that
// take the bytes out and leave zeros beyond n.  (A load at an odd address costs
// several times an aligned one: 1 x 14338 x 4096 took 27 us with those, 17.6
// us so.)  No dword without a byte of the row is read, if the row has the chunk's
// bytes at least.  TINY: shorter rows, byte by byte.
template <bool A4, bool TINY>
struct AnyChunk {
  static constexpr int kBytes = A4 ? 8 : 16, kWords = kBytes / 4;
  uint32_t d[kWords + 1];

  static __device__ __forceinline__ int offset(int j0, int n) {
    return min(A4 ? j0 / 2 : j0, max((A4 ? n / 2 : n) - kBytes, 0));
  }
  __device__ __forceinline__ void load(const uint8_t* p, int j0, int n) {
    if (TINY) {
#pragma unroll
      for (int i = 0; i <= kWords; ++i) d[i] = 0;
      if (j0 == 0) {
#pragma unroll
        for (int i = 0; i < kBytes; ++i)
          if (i < (A4 ? n / 2 : n)) d[i >> 2] |= static_cast<uint32_t>(p[i]) << (8 * (i & 3));
      }
      return;
    }
    p += offset(j0, n);
    const int odd = static_cast<int>(reinterpret_cast<uintptr_t>(p) & 3u);
    const uint32_t* const q = reinterpret_cast<const uint32_t*>(p - odd);
#pragma unroll
    for (int i = 0; i < kWords; ++i) d[i] = q[i];
    d[kWords] = q[odd ? kWords : kWords - 1];
  }
  // The operand; `cut`: the chunk may pass the row's end.  Packed codes are widened.
  __device__ __forceinline__ i32x4_t take(const uint8_t* p, int j0, int n, bool cut) const {
    uint32_t w[4] = {0, 0, 0, 0};
    const uint32_t odd = TINY ? 0 : (reinterpret_cast<uintptr_t>(p) + offset(j0, n)) & 3u;
#pragma unroll
    for (int i = 0; i < kWords; ++i) w[i] = __builtin_amdgcn_alignbyte(d[i + 1], d[i], odd);
    if (cut && !TINY) {
      const int by = (A4 ? j0 / 2 : j0) - offset(j0, n);  // bytes moved back
      uint64_t lo = w[0] | static_cast<uint64_t>(w[1]) << 32, hi = w[2] | static_cast<uint64_t>(w[3]) << 32;
      if (by >= 16) {
        lo = hi = 0;
      } else if (by >= 8) {
        lo = hi >> (8 * (by - 8));
        hi = 0;
      } else if (by > 0) {
        lo = lo >> (8 * by) | hi << (64 - 8 * by);
        hi >>= 8 * by;
      }
      w[0] = static_cast<uint32_t>(lo);
      w[1] = static_cast<uint32_t>(lo >> 32);
      w[2] = static_cast<uint32_t>(hi);
      w[3] = static_cast<uint32_t>(hi >> 32);
    }
    if (A4) {
      const uint32_t c0 = w[0], c1 = w[1];
      widen8(c0, w[0], w[1]);
      widen8(c1, w[2], w[3]);
    }
    return i32x4_t{static_cast<int>(w[0]), static_cast<int>(w[1]), static_cast<int>(w[2]), static_cast<int>(w[3])};
  }
};

// Tile of WK x WT waves of FK x FT 16 x 16 results, steps of KU * 64 k.  Step s
// multiplies from one LDS buffer while the registers with step s + 1 are written
// to the other and filled with step s + 2 (three sets of registers were slower).
// LDS as in w8_tile: for each depth rows of 64 bytes, chunk c of row r at chunk
// c ^ 2 ((r >> 3) & 1).
template <bool A4, int WK, int WT, int FK, int FT, int KU>
struct AnyTile {
  static constexpr int kThreads = 64 * WK * WT;
  static constexpr int kBN = 16 * WK * FK, kBM = 16 * WT * FT;
  static constexpr int kStep = 64 * KU;
  static constexpr int kWSlots = kBN * 4 * KU, kTSlots = kBM * 4 * KU;  // 16-byte chunks of a step
  static constexpr int kWPer = kWSlots / kThreads, kTPer = kTSlots / kThreads;
  static_assert(kWPer * kThreads == kWSlots && kTPer * kThreads == kTSlots, "whole chunks per thread");
};

// The factors of a lane's results: channels k + 16 f + e (e < 4), tokens t + 16 j.
template <bool A4, int FK, int FT>
struct Factors {
  float v[FK][4], ws[FK][4], b[FK][4], sc[FT], z[FT];
  __device__ __forceinline__ Factors(const W8Args& a, int k, int t) {
#pragma unroll
    for (int f = 0; f < FK; ++f)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int c = min(k + 16 * f + e, a.R - 1);
        v[f][e] = a.w_scale[c];
        ws[f][e] = A4 ? static_cast<float>(a.w_sum[c]) : 0.f;
        b[f][e] = a.bias ? a.bias[c] : 0.f;
      }
#pragma unroll
    for (int j = 0; j < FT; ++j) {
      const int c = min(t + 16 * j, a.T - 1);
      sc[j] = a.scale[c];
      z[j] = A4 ? a.zero[c] : 0.f;
    }
  }
  __device__ __forceinline__ float finish(int f, int e, int j, int32_t acc) const {
    float x = static_cast<float>(acc);
    if (A4) x = fmaf(-z[j], ws[f][e], x);
    return fmaf(x * sc[j], v[f][e], b[f][e]);
  }
};

template <bool A4, int WK, int WT, int FK, int FT, int KU, bool TINY>
__global__ __launch_bounds__(64 * WK * WT) void w8_any_kernel(W8Args a, int first_m, int first_n, int tiles_n) {
  using C = AnyTile<A4, WK, WT, FK, FT, KU>;
  __shared__ i32x4_t lds[2][C::kWSlots + C::kTSlots];
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int m0 = (first_m + static_cast<int>(blockIdx.x / tiles_n)) * C::kBM;
  const int n0 = (first_n + static_cast<int>(blockIdx.x % tiles_n)) * C::kBN;
  const int wk = wid % WK, wt = wid / WK;
  const int steps = (a.n + C::kStep - 1) / C::kStep;

  // chunk x of a thread: KU * 4 neighbouring threads share a row; rows clamped (not stored)
  const uint8_t* pw[C::kWPer];
  const uint8_t* pt[C::kTPer];
  int kw[C::kWPer], kt[C::kTPer], sw[C::kWPer], st[C::kTPer];
  auto slot = [](int r, int c, int rows) { return ((c >> 2) * rows + r) * 4 + ((c & 3) ^ (2 * ((r >> 3) & 1))); };
  const int at = 4 * (lane & 15) + ((lane >> 4) ^ (2 * ((lane >> 3) & 1)));  // the lane's chunk of a 16-row group
#pragma unroll
  for (int x = 0; x < C::kWPer; ++x) {
    const int e = tid + x * C::kThreads, r = e / (4 * KU), c = e % (4 * KU);
    pw[x] = reinterpret_cast<const uint8_t*>(a.w) + static_cast<int64_t>(min(n0 + r, a.R - 1)) * a.ldw;
    kw[x] = 16 * c;
    sw[x] = slot(r, c, C::kBN);
  }
#pragma unroll
  for (int x = 0; x < C::kTPer; ++x) {
    const int e = tid + x * C::kThreads, r = e / (4 * KU), c = e % (4 * KU);
    pt[x] = a.a + static_cast<int64_t>(min(m0 + r, a.T - 1)) * a.lda;
    kt[x] = 16 * c;
    st[x] = C::kWSlots + slot(r, c, C::kBM);
  }
  AnyChunk<false, TINY> vw[C::kWPer];
  AnyChunk<A4, TINY> vt[C::kTPer];
  // step 0 is the row's last, possibly short one
  auto start = [&](int s) { return C::kStep * (s == 0 ? steps - 1 : s - 1); };
  auto load = [&](int s) {
    const int k0 = start(s);
#pragma unroll
    for (int x = 0; x < C::kWPer; ++x) vw[x].load(pw[x], k0 + kw[x], a.n);
#pragma unroll
    for (int x = 0; x < C::kTPer; ++x) vt[x].load(pt[x], k0 + kt[x], a.n);
  };
  auto store = [&](int s, bool cut) {
    const int k0 = start(s);
#pragma unroll
    for (int x = 0; x < C::kWPer; ++x) lds[s & 1][sw[x]] = vw[x].take(pw[x], k0 + kw[x], a.n, cut);
#pragma unroll
    for (int x = 0; x < C::kTPer; ++x) lds[s & 1][st[x]] = vt[x].take(pt[x], k0 + kt[x], a.n, cut);
  };
  i32x4_t acc[FK][FT];
#pragma unroll
  for (int f = 0; f < FK; ++f)
#pragma unroll
    for (int j = 0; j < FT; ++j) acc[f][j] = i32x4_t{0, 0, 0, 0};

  load(0);
  store(0, true);
  load(min(1, steps - 1));
  __syncthreads();
  for (int s = 0; s < steps; ++s) {
    const int buf = s & 1;
    i32x4_t fw[KU][FK], ft[KU][FT];
#pragma unroll
    for (int u = 0; u < KU; ++u) {
#pragma unroll
      for (int f = 0; f < FK; ++f) fw[u][f] = lds[buf][(u * C::kBN + 16 * (wk * FK + f)) * 4 + at];
#pragma unroll
      for (int j = 0; j < FT; ++j) ft[u][j] = lds[buf][C::kWSlots + (u * C::kBM + 16 * (wt * FT + j)) * 4 + at];
    }
    if (s + 1 < steps) store(s + 1, false);
    load(min(s + 2, steps - 1));
#pragma unroll
    for (int u = 0; u < KU; ++u)
#pragma unroll
      for (int f = 0; f < FK; ++f)
#pragma unroll
        for (int j = 0; j < FT; ++j)
          acc[f][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[u][f], ft[u][j], acc[f][j], 0, 0, 0);
    __syncthreads();
  }
  // All factors first: a load after a store waits for the store.
  Factors<A4, FK, FT> fac(a, n0 + 16 * wk * FK + 4 * (lane >> 4), m0 + 16 * wt * FT + (lane & 15));
#pragma unroll
  for (int j = 0; j < FT; ++j) {
    const int t = m0 + 16 * (wt * FT + j) + (lane & 15);
    if (t >= a.T) continue;
#pragma unroll
    for (int f = 0; f < FK; ++f) {
      float o[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[e] = fac.finish(f, e, j, acc[f][j][e]);
      const int k = n0 + 16 * (wk * FK + f) + 4 * (lane >> 4);
      store_results(a, t, k, o, k + 4 <= a.R);
    }
  }
}

constexpr double kAnyOne = 0.50, kAnyTwo = 0.74;  // as in TileCost, for its 64 x 64 tile

template <bool A4>
hipError_t run_any(const W8Args& a, hipStream_t s) {
  using C = AnyTile<A4, 2, 2, 2, 2, 2>;
  // A launch holds fewer than 2^32 threads, so rows too short to be laid out anew
  // may take several, each over some token tiles and channel tiles.
  constexpr int kMost = 1 << 23;
  const int tiles_m = (a.T + C::kBM - 1) / C::kBM, tiles_n = (a.R + C::kBN - 1) / C::kBN;
  const int step_n = tiles_n < kMost ? tiles_n : kMost, step_m = kMost / step_n;
  const dim3 block(static_cast<unsigned>(C::kThreads));
  for (int m = 0; m < tiles_m; m += step_m) {
    for (int n = 0; n < tiles_n; n += step_n) {
      const int rows = tiles_m - m < step_m ? tiles_m - m : step_m;
      const int columns = tiles_n - n < step_n ? tiles_n - n : step_n;
      const dim3 grid(static_cast<unsigned>(rows) * static_cast<unsigned>(columns));
      if (a.n < 16)
        w8_any_kernel<A4, 2, 2, 2, 2, 2, true><<<grid, block, 0, s>>>(a, m, n, columns);
      else
        w8_any_kernel<A4, 2, 2, 2, 2, 2, false><<<grid, block, 0, s>>>(a, m, n, columns);
      const hipError_t e = hipGetLastError();
      if (e != hipSuccess) return e;
    }
  }
  return hipSuccess;
}

// Few tokens: as w8_few, with both operands straight to registers, a lane (g, i)
// reading 16 bytes (g) of row i for each 64 k.
template <bool A4, int FT, bool TINY>
__global__ __launch_bounds__(1024) void w8_few_any_kernel(W8Args a) {
  extern __shared__ __attribute__((aligned(16))) int32_t few_part[];  // [wave][FT][64][4]
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int waves = blockDim.x >> 6;
  const int g = lane >> 4, i = lane & 15;
  const int n0 = 16 * blockIdx.x;
  const uint8_t* const pw =
      reinterpret_cast<const uint8_t*>(a.w) + static_cast<int64_t>(min(n0 + i, a.R - 1)) * a.ldw;
  const uint8_t* pt[FT];
#pragma unroll
  for (int j = 0; j < FT; ++j) pt[j] = a.a + static_cast<int64_t>(min(16 * j + i, a.T - 1)) * a.lda;
  i32x4_t acc[FT];
#pragma unroll
  for (int j = 0; j < FT; ++j) acc[j] = i32x4_t{0, 0, 0, 0};
  auto unit = [&](int k0, bool cut) {
    AnyChunk<false, TINY> w[2];
    AnyChunk<A4, TINY> tok[2][FT];
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = k0 + 64 * s + 16 * g;
      w[s].load(pw, k, a.n);
#pragma unroll
      for (int j = 0; j < FT; ++j) tok[s][j].load(pt[j], k, a.n);
    }
#pragma unroll
    for (int s = 0; s < 2; ++s) {
      const int k = k0 + 64 * s + 16 * g;
      const i32x4_t ws = w[s].take(pw, k, a.n, cut);
#pragma unroll
      for (int j = 0; j < FT; ++j)
        acc[j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(ws, tok[s][j].take(pt[j], k, a.n, cut), acc[j], 0, 0, 0);
    }
  };
  int k0 = kUnit * wid;
  for (; k0 + kUnit <= a.n; k0 += kUnit * waves) unit(k0, false);
  if (k0 < a.n) unit(k0, true);
#pragma unroll
  for (int j = 0; j < FT; ++j)
    *reinterpret_cast<i32x4_t*>(few_part + 4 * ((wid * FT + j) * 64 + lane)) = acc[j];
  __syncthreads();
  few_finish<1, FT>(a, few_part, n0, waves);
}

template <bool A4>
hipError_t run_few_any(const W8Args& a, hipStream_t s) {
  const int groups = (a.R + 15) / 16;
  int waves = 16;
  while (waves > 4 && (groups * waves > 32 * kCus || (a.n + kUnit - 1) / kUnit < waves)) waves /= 2;
  const dim3 grid(static_cast<unsigned>(groups)), block(static_cast<unsigned>(64 * waves));
  const unsigned lds = static_cast<unsigned>(1024 * waves);
  if (a.n < 16) {
    if (a.T <= 16)
      w8_few_any_kernel<A4, 1, true><<<grid, block, lds, s>>>(a);
    else
      w8_few_any_kernel<A4, 2, true><<<grid, block, 2 * lds, s>>>(a);
  } else if (a.T <= 16) {
    w8_few_any_kernel<A4, 1, false><<<grid, block, lds, s>>>(a);
  } else {
    w8_few_any_kernel<A4, 2, false><<<grid, block, 2 * lds, s>>>(a);
  }
  return hipGetLastError();
}

// Many tokens: the rows are laid out anew in the workspace, in whole chunks with
// zeros beyond n, and the tile kernels run on those.  One launch for both
// operands: rows 0 .. rows_w - 1 are the weights', the rest the codes'.
struct PackArgs {  // rows of at least sixteen bytes
  const uint8_t* src[2];
  uint8_t* dst[2];
  int64_t ld[2];
  int bytes[2], chunks[2];
  int64_t rows[2];
};
__global__ __launch_bounds__(256) void w8_pack_kernel(PackArgs a) {
  for (int64_t row = blockIdx.x; row < a.rows[0] + a.rows[1]; row += gridDim.x) {
    const int x = row < a.rows[0] ? 0 : 1;
    const int64_t r = x ? row - a.rows[0] : row;
    const uint8_t* const src = a.src[x] + r * a.ld[x];
    i32x4_t* const dst = reinterpret_cast<i32x4_t*>(a.dst[x]) + r * a.chunks[x];
    for (int c = threadIdx.x; c < a.chunks[x]; c += blockDim.x) {
      AnyChunk<false, false> v;
      v.load(src, 16 * c, a.bytes[x]);
      dst[c] = v.take(src, 16 * c, a.bytes[x], 16 * c + 16 > a.bytes[x]);
    }
  }
}

hipError_t run_pack(const PackArgs& a, hipStream_t s) {
  const int64_t rows = a.rows[0] + a.rows[1];
  const int waves = (a.chunks[0] + 63) / 64;
  w8_pack_kernel<<<dim3(static_cast<unsigned>(rows < 64 * kCus ? rows : 64 * kCus)),
                   dim3(static_cast<unsigned>(64 * (waves < 4 ? waves : 4))), 0, s>>>(a);
  return hipGetLastError();
}

// Where the operands of a product that packs lie in its workspace: the weights,
// the codes unless their rows are aligned already, then the partial sums.
struct Packed {
  int n;          // k of the packed rows
  bool codes;     // the codes are packed too
  int64_t w_bytes, t_bytes;
};
Packed packing(const W8Args& a) {
  Packed p;
  p.n = a.a4 ? (a.n + 31) / 32 * 32 : (a.n + 15) / 16 * 16;
  p.codes = a.lda % 16 != 0 || (reinterpret_cast<uintptr_t>(a.a) & 15u) != 0 || a.lda >= kMaxPitch;
  p.w_bytes = static_cast<int64_t>(a.R) * p.n;
  p.t_bytes = p.codes ? static_cast<int64_t>(a.T) * (a.a4 ? p.n / 2 : p.n) : 0;
  return p;
}

hipError_t run_tiles(const W8Args& a, const Plan& p, hipStream_t s) {
  if (a.a4) {
    switch (p.kind) {
      case 0: return run_tile<true, 2, 4, 8, 4, 1, 4>(a, p.splits, s);
      case 1: return run_tile<true, 2, 4, 4, 2, 2, 5>(a, p.splits, s);
      case 2: return run_tile<true, 1, 4, 4, 2, 2, 5>(a, p.splits, s);
      case 3: return run_tile<true, 1, 4, 4, 1, 2, 5>(a, p.splits, s);
      default: return run_tile<true, 1, 4, 4, 1, 4, 5>(a, p.splits, s);
    }
  }
  switch (p.kind) {
    case 0: return run_tile<false, 4, 2, 4, 8, 1, 4>(a, p.splits, s);
    case 1: return run_tile<false, 2, 2, 4, 4, 2, 5>(a, p.splits, s);
    case 2: return run_tile<false, 2, 2, 4, 2, 2, 5>(a, p.splits, s);
    case 3: return run_tile<false, 1, 4, 4, 1, 2, 5>(a, p.splits, s);
    default: return run_tile<false, 1, 4, 4, 1, 4, 5>(a, p.splits, s);
  }
}

// The way a product takes.
struct Way {
  enum { kFew, kFewAny, kAny, kTiles, kPackTiles } kind;
  Plan plan;  // kTiles, kPackTiles
};
Way way_of(const W8Args& a) {
  const bool aligned = aligned_rows(a);
  if (takes_few(a.T, a.R)) return {aligned ? Way::kFew : Way::kFewAny, {0, 1, 0}};
  if (aligned) return {Way::kTiles, tile_plan(a.T, a.n, a.R, a.a4 != 0)};
  const Packed k = packing(a);
  Plan p = tile_plan(a.T, k.n, a.R, a.a4 != 0);
  // packing: a launch and the workspace, and 5 TB/s over what it reads and writes
  p.us += 7.0 + 2.0 * (k.w_bytes + k.t_bytes) / 5e6;
  const double tiles = static_cast<double>((a.T + int64_t{63}) / 64) * static_cast<double>((a.R + int64_t{63}) / 64);
  const double per_cu = ceil(tiles / kCus), deep = a.n / 128.0;
  const double any =
      floor(per_cu / 2) * (deep * kAnyTwo + 2.0) + fmod(per_cu, 2) * (deep * kAnyOne + 1.8);
  // w8_any up to where packing both operands and the tiles are less: 1000 x 1111 x
  // 1000 8.0 us, packed 11.5; 64 x 4098 x 4096 18.0 and 23.7; 256 x 4098 x 14336
  // 51.8 and 45.3; 4000 x 300 x 4000 33.4 and 20.6.  (At 18 shapes the estimate
  // takes the slower one by 15 % at most.)  Packing reads whole 16-byte chunks, so
  // rows of fewer bytes stay here.
  if ((any < p.us && tiles < (1 << 22)) || (a.a4 ? a.n / 2 : a.n) < 16) return {Way::kAny, {0, 1, any}};
  return {Way::kPackTiles, p};
}

}  // namespace

int64_t w8_workspace(const W8Args& a) {
  if (a.T == 0 || a.R == 0) return 0;
  const Way way = way_of(a);
  int64_t bytes = 0;
  if (way.kind == Way::kPackTiles) {
    const Packed k = packing(a);
    bytes = k.w_bytes + k.t_bytes;
  }
  if (way.plan.splits > 1) {
    const TileCost& t = a.a4 ? kTiles4[way.plan.kind] : kTiles8[way.plan.kind];
    bytes += ((static_cast<int64_t>(a.T) + t.bm - 1) / t.bm) * ((static_cast<int64_t>(a.R) + t.bn - 1) / t.bn) *
             way.plan.splits * t.bm * t.bn * 4;
  }
  return bytes;
}

const char* w8_name(const W8Args& a) {
  if (a.T == 0 || a.R == 0) return "none";
  const Way way = way_of(a);
  static const char* const names[2][6] = {{"w8_tile_256x256", "w8_tile_128x128", "w8_tile_64x128", "w8_tile_64x64",
                                           "w8_tile_64x64_deep", "w8_tile_128x64"},
                                          {"w8_pack_tile_256x256", "w8_pack_tile_128x128", "w8_pack_tile_64x128",
                                           "w8_pack_tile_64x64", "w8_pack_tile_64x64_deep", "w8_pack_tile_128x64"}};
  switch (way.kind) {
    case Way::kFew: return "w8_few";
    case Way::kFewAny: return "w8_few_any";
    case Way::kAny: return "w8_any";
    default: return names[way.kind == Way::kPackTiles][a.a4 && way.plan.kind == 2 ? 5 : way.plan.kind];
  }
}

hipError_t launch_w8(const W8Args& all, hipStream_t s) {
  W8Args a = all;
  a.row_bytes = a.a4 ? a.n / 2 : a.n;
  const Way way = way_of(a);
  switch (way.kind) {
    case Way::kFew: return a.a4 ? run_few<true>(a, s) : run_few<false>(a, s);
    case Way::kFewAny: return a.a4 ? run_few_any<true>(a, s) : run_few_any<false>(a, s);
    case Way::kAny: return a.a4 ? run_any<true>(a, s) : run_any<false>(a, s);
    case Way::kTiles: return run_tiles(a, way.plan, s);
    case Way::kPackTiles: break;
  }
  const Packed k = packing(a);
  uint8_t* const at = reinterpret_cast<uint8_t*>(a.partial);
  const int pitch = a.a4 ? k.n / 2 : k.n;
  const PackArgs pack = {{reinterpret_cast<const uint8_t*>(a.w), a.a}, {at, at + k.w_bytes},   {a.ldw, a.lda},
                         {a.n, a.row_bytes},                           {k.n / 16, pitch / 16}, {a.R, k.codes ? a.T : 0}};
  const hipError_t e = run_pack(pack, s);
  if (e != hipSuccess) return e;
  a.w = reinterpret_cast<const int8_t*>(at);
  a.ldw = a.n = k.n;
  if (k.codes) {
    a.a = at + k.w_bytes;
    a.lda = pitch;
  }
  // aligned codes are read to the end of their last 16-byte chunk, up to 15 bytes
  // past the row (of the last row too) but in the page of the chunk's first byte;
  // whatever is there meets weights of zero
  a.row_bytes = pitch;
  a.partial = reinterpret_cast<int32_t*>(at + k.w_bytes + k.t_bytes);
  return run_tiles(a, way.plan, s);
}

}  // namespace signrot
