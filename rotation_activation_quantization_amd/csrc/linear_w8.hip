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
#include <stdint.h>
#include <string.h>

#include "internal.h"
#include "row_ops.h"
#include "wave_ops.h"

namespace signrot {
namespace {

typedef __attribute__((__vector_size__(4 * sizeof(int32_t)))) int32_t i32x4_t;

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
  v = v * a.scale[t] * a.w_scale[k];
  return a.bias ? v + a.bias[k] : v;
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

constexpr int kStep = 64;  // k per step, one MFMA deep

// WK x WT waves of FK x FT 16 x 16 results each, a ring of S steps.
template <bool A4, int WK, int WT, int FK, int FT, int S>
struct Tile {
  static constexpr int kWaves = WK * WT;
  static constexpr int kThreads = 64 * kWaves;
  static constexpr int kBN = 16 * WK * FK;                // channels
  static constexpr int kBM = 16 * WT * FT;                // tokens
  static constexpr int kTokRow = A4 ? kStep / 2 : kStep;  // bytes of a token row and step
  static constexpr int kWStage = kBN * kStep;
  static constexpr int kTStage = kBM * kTokRow;
  static constexpr int kWLoads = kWStage / 1024 / kWaves;  // LDS loads per wave and step
  static constexpr int kTLoads = kTStage / 1024 / kWaves;
  static constexpr int kLoads = kWLoads + kTLoads;
  static_assert(kWLoads * 1024 * kWaves == kWStage && kTLoads * 1024 * kWaves == kTStage, "whole loads per wave");
  static_assert(FK % 4 == 0, "a lane's channels come in sixteens");
  static_assert(S >= 4 && S * (kWStage + kTStage) <= 160 * 1024, "ring");
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
// Slot 16 f + i of a 64-channel group holds channel 16 (i / 4) + 4 f + i % 4:
// the four 16 x 16 results f = 0 .. 3 then leave a lane sixteen consecutive
// channels of a token, stored as whole vectors.
template <bool A4, int WK, int WT, int FK, int FT, int S>
__device__ __forceinline__ void w8_tile(const W8Args& a, int tiles_m, int tiles_n) {
  using C = Tile<A4, WK, WT, FK, FT, S>;
  __shared__ __attribute__((aligned(16))) uint8_t lds[S * (C::kWStage + C::kTStage)];
  uint8_t* const lds_w = lds;
  uint8_t* const lds_t = lds + S * C::kWStage;
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wid % WK, wt = wid / WK;
  const int g = lane >> 4, i = lane & 15;

  // Consecutive block ids go to different XCDs: each XCD takes one contiguous
  // range of the tiles, its work-groups (gridDim / 8 of them) the tiles of that
  // range in turn.  A grid that is not a multiple of eight is one tile each.
  int p, end, stride;
  {
    const int tiles = tiles_m * tiles_n;
    const int q = tiles >> 3, rem = tiles & 7;
    const int x = blockIdx.x & 7;
    const int start = x < rem ? x * (q + 1) : rem * (q + 1) + (x - rem) * q;
    p = start + (blockIdx.x >> 3);
    end = start + q + (x < rem ? 1 : 0);
    stride = (gridDim.x & 7) ? tiles : gridDim.x >> 3;
  }
  const int last = (a.n + kStep - 1) / kStep - 1;
  const int tail = a.n - last * kStep;  // k of step 0

  // What is loaded next: step ik of tile src_p.  Rows beyond the tensor are
  // clamped (their results are not stored).
  const int chunk_w = (lane & 3) ^ (2 * (lane >> 5));  // logical chunk of the lane's slot: row lane / 4 of 16
  const int chunk_t = A4 ? (g & 1) : chunk_w;
  const uint32_t cut_w = 16 * chunk_w >= tail ? -16 * chunk_w : 0;
  const uint32_t cut_t = (A4 ? 32 : 16) * chunk_t >= tail ? -16 * chunk_t : 0;
  int src_p = p, ik = 0;
  const int8_t* base_w;
  const uint8_t* base_t;
  uint32_t size_w, size_t_, off_w[C::kWLoads], off_t[C::kTLoads];
  auto set_source = [&]() {
    int tm, tn;
    tile_at(src_p, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * C::kBM, n0 = tn * C::kBN;
    const int rows_w = min(C::kBN, a.R - n0), rows_t = min(C::kBM, a.T - m0);
    base_w = a.w + static_cast<int64_t>(n0) * a.ldw;
    base_t = a.a + static_cast<int64_t>(m0) * a.lda;
    size_w = static_cast<uint32_t>(rows_w - 1) * static_cast<uint32_t>(a.ldw) + a.n;
    size_t_ = static_cast<uint32_t>(rows_t - 1) * static_cast<uint32_t>(a.lda) + (A4 ? a.n / 2 : a.n);
#pragma unroll
    for (int l = 0; l < C::kWLoads; ++l) {
      const int slot = 16 * (C::kWLoads * wid + l) + (lane >> 2);
      const int at = slot & 15;
      const int ch = (slot & ~63) + 16 * (at >> 2) + 4 * ((slot >> 4) & 3) + (at & 3);
      off_w[l] = static_cast<uint32_t>(min(ch, rows_w - 1)) * static_cast<uint32_t>(a.ldw) + 16 * chunk_w + cut_w;
    }
#pragma unroll
    for (int l = 0; l < C::kTLoads; ++l) {
      const int r =
          A4 ? 32 * (C::kTLoads * wid + l) + 16 * (lane >> 5) + i : 16 * (C::kTLoads * wid + l) + (lane >> 2);
      off_t[l] = static_cast<uint32_t>(min(r, rows_t - 1)) * static_cast<uint32_t>(a.lda) + 16 * chunk_t + cut_t;
    }
  };
  int wr_w = 0, wr_t = 0;  // ring position that is filled
  int ks = last;           // 64 k-block of step ik
  auto issue = [&](int l) {
    if (l < C::kWLoads) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          wave::buffer_rsrc(base_w, size_w),
          (__attribute__((address_space(3))) void*)(lds_w + wr_w + 1024 * (C::kWLoads * wid + l)), 16,
          off_w[l], kStep * ks, 0, 0);
    } else {
      const int j = l - C::kWLoads;
      __builtin_amdgcn_raw_ptr_buffer_load_lds(
          wave::buffer_rsrc(base_t, size_t_),
          (__attribute__((address_space(3))) void*)(lds_t + wr_t + 1024 * (C::kTLoads * wid + j)), 16,
          off_t[j], C::kTokRow * ks, 0, 0);
    }
  };
  // Past the last tile the loads go on with that tile's: every step issues the
  // same number, so the vmcnt threshold is exact.
  auto issued = [&]() {
    wr_w = wr_w == (S - 1) * C::kWStage ? 0 : wr_w + C::kWStage;
    wr_t = wr_t == (S - 1) * C::kTStage ? 0 : wr_t + C::kTStage;
    if (ik == 0 && tail < kStep) {
#pragma unroll
      for (int l = 0; l < C::kWLoads; ++l) off_w[l] -= cut_w;
#pragma unroll
      for (int l = 0; l < C::kTLoads; ++l) off_t[l] -= cut_t;
    }
    ik = __builtin_amdgcn_readfirstlane(ik == last ? 0 : ik + 1);
    if (ik == 0) {
      src_p = src_p + stride < end ? src_p + stride : src_p;
      set_source();
    }
    ks = __builtin_amdgcn_readfirstlane(ik == 0 ? last : ik - 1);
  };

  const int read_w = (64 * wk * FK / 4) * kStep + i * kStep + 16 * (g ^ (2 * (i >> 3)));
  const int read_t = A4 ? 512 * (wt * FT) + 256 * (g >> 1) + 16 * i + 8 * (g & 1)
                        : 16 * wt * FT * kStep + i * kStep + 16 * (g ^ (2 * (i >> 3)));
  int rd_w = 0, rd_t = 0;  // ring position that is multiplied
  auto weight = [&](int at, int f) {
    return *reinterpret_cast<const i32x4_t*>(lds_w + at + read_w + 16 * kStep * f);
  };

  i32x4_t acc[FK][FT];
  i32x4_t tok[2][FT];  // token operands of this and the next step
  wave::u32x2_t code[FT];
  auto read_token = [&](int at, int j, i32x4_t& dst) {
    const uint8_t* s = lds_t + at + read_t;
    if (A4)
      code[j] = *reinterpret_cast<const wave::u32x2_t*>(s + 512 * j);
    else
      dst = *reinterpret_cast<const i32x4_t*>(s + 16 * kStep * j);
  };
  auto widen = [&](int j, i32x4_t& dst) {
    uint32_t w0, w1, w2, w3;
    widen8(code[j][0], w0, w1);
    widen8(code[j][1], w2, w3);
    dst = i32x4_t{static_cast<int>(w0), static_cast<int>(w1), static_cast<int>(w2), static_cast<int>(w3)};
    asm volatile("" : "+v"(dst));  // here, not where the next step uses it
  };

  set_source();
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

  auto step = [&](i32x4_t (&now)[FT], i32x4_t (&next)[FT]) {
    const int nx_w = rd_w == (S - 1) * C::kWStage ? 0 : rd_w + C::kWStage;
    const int nx_t = rd_t == (S - 1) * C::kTStage ? 0 : rd_t + C::kTStage;
#pragma unroll
    for (int f = 0; f < FK; ++f) {
      // The reads follow the block's first MFMA: the wait before that one is
      // then for reads a whole block old.
      acc[f][0] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[f], now[0], acc[f][0], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
      // two reads ahead, the last two from the next step
      wf[f + 2] = f + 2 < FK ? weight(rd_w, f + 2) : weight(nx_w, f + 2 - FK);
      // the next step's tokens: packed codes are read over the first half of
      // the blocks and widened, between the MFMAs, over the second
      constexpr int kOver = A4 ? FK / 2 : FK;
      if (f < kOver) {
#pragma unroll
        for (int j = f * FT / kOver; j < (f + 1) * FT / kOver; ++j) read_token(nx_t, j, next[j]);
      } else {
#pragma unroll
        for (int j = (f - kOver) * FT / kOver; j < (f - kOver + 1) * FT / kOver; ++j) widen(j, next[j]);
      }
#pragma unroll
      for (int l = f * C::kLoads / FK; l < (f + 1) * C::kLoads / FK; ++l) issue(l);
#pragma unroll
      for (int j = 1; j < FT; ++j)
        acc[f][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(wf[f], now[j], acc[f][j], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    wf[0] = wf[FK];
    wf[1] = wf[FK + 1];
    rd_w = nx_w;
    rd_t = nx_t;
    issued();
    wave::wait_vmcnt<(S - 3) * C::kLoads>();
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };

  const bool wide = (a.ldo % 8 == 0) && (reinterpret_cast<uintptr_t>(a.out) & 15u) == 0;
  for (; p < end; p += stride) {
#pragma unroll
    for (int f = 0; f < FK; ++f)
#pragma unroll
      for (int j = 0; j < FT; ++j) acc[f][j] = i32x4_t{0, 0, 0, 0};
    if (tail < kStep) {
#pragma unroll
      for (int j = 0; j < FT; ++j)
        if (16 * g >= tail) tok[0][j] = i32x4_t{0, 0, 0, 0};
    }
    for (int kt = 0; kt < last; kt += 2) {
      step(tok[0], tok[1]);
      step(tok[1], tok[0]);
    }
    if ((last & 1) == 0) {
      step(tok[0], tok[1]);
#pragma unroll
      for (int j = 0; j < FT; ++j) tok[0][j] = tok[1][j];
    }

    // Lane (g, i): token 16 j + i, channels 16 g .. 16 g + 15 of every 64.
    int tm, tn;
    tile_at(p, tiles_m, tiles_n, tm, tn);
    const int m0 = tm * C::kBM, n0 = tn * C::kBN;
#pragma unroll
    for (int q = 0; q < FK / 4; ++q) {
      const int k0 = n0 + 16 * wk * FK + 64 * q + 16 * g;
      if (k0 >= a.R) continue;
      const bool whole = wide && k0 + 16 <= a.R;
      float v[16], b[16], ws[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        const int k = min(k0 + e, a.R - 1);
        v[e] = a.w_scale[k];
        ws[e] = A4 ? static_cast<float>(a.w_sum[k]) : 0.f;
        b[e] = 0.f;
      }
      if (a.bias) {
#pragma unroll
        for (int e = 0; e < 16; ++e) b[e] = a.bias[min(k0 + e, a.R - 1)];
      }
#pragma unroll
      for (int j = 0; j < FT; ++j) {
        const int t = m0 + 16 * (wt * FT + j) + i;
        if (t >= a.T) continue;
        const float sc = a.scale[t], z = A4 ? a.zero[t] : 0.f;
        float o[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float x = static_cast<float>(acc[4 * q + (e >> 2)][j][e & 3]);
          if (A4) x = fmaf(-z, ws[e], x);
          o[e] = fmaf(x * sc, v[e], b[e]);
        }
        const int64_t at = static_cast<int64_t>(t) * a.ldo + k0;
        if (whole && a.out_bf16) {
          uint32_t h[8];
#pragma unroll
          for (int e = 0; e < 8; ++e)
            h[e] = row::f32_bf16(o[2 * e]) | static_cast<uint32_t>(row::f32_bf16(o[2 * e + 1])) << 16;
          wave::u32x4_t* out = reinterpret_cast<wave::u32x4_t*>(static_cast<uint16_t*>(a.out) + at);
          out[0] = wave::u32x4_t{h[0], h[1], h[2], h[3]};
          out[1] = wave::u32x4_t{h[4], h[5], h[6], h[7]};
        } else if (whole) {
          wave::f32x4_t* out = reinterpret_cast<wave::f32x4_t*>(static_cast<float*>(a.out) + at);
#pragma unroll
          for (int e = 0; e < 4; ++e) out[e] = wave::f32x4_t{o[4 * e], o[4 * e + 1], o[4 * e + 2], o[4 * e + 3]};
        } else {
#pragma unroll
          for (int e = 0; e < 16; ++e)
            if (k0 + e < a.R) row::store_elem(a.out, at + e, o[e], a.out_bf16);
        }
      }
    }
  }
  wave::wait_vmcnt<0>();
}

template <bool A4, int WK, int WT, int FK, int FT, int S>
__global__ __launch_bounds__(64 * WK * WT) __attribute__((amdgpu_waves_per_eu(WK * WT / 4)))
void w8_tile_kernel(W8Args a, int tiles_m, int tiles_n) {
  w8_tile<A4, WK, WT, FK, FT, S>(a, tiles_m, tiles_n);
}

template <bool A4, int WK, int WT, int FK, int FT, int S>
void run_tile(const W8Args& a, hipStream_t s) {
  using C = Tile<A4, WK, WT, FK, FT, S>;
  const int tiles_m = (a.T + C::kBM - 1) / C::kBM, tiles_n = (a.R + C::kBN - 1) / C::kBN;
  const int tiles = tiles_m * tiles_n;
  const int cus = device_cu_count() & ~7;
  w8_tile_kernel<A4, WK, WT, FK, FT, S><<<dim3(static_cast<unsigned>(cus > 0 && tiles > cus ? cus : tiles)),
                                          dim3(C::kThreads), 0, s>>>(a, tiles_m, tiles_n);
}

// Rows that start on 16-byte boundaries and end on one.
bool aligned_rows(const W8Args& a) {
  return a.n % (a.a4 ? 32 : 16) == 0 && a.lda % 16 == 0 && a.ldw % 16 == 0 &&
         ((reinterpret_cast<uintptr_t>(a.a) | reinterpret_cast<uintptr_t>(a.w)) & 15u) == 0 &&
         a.lda < (int64_t{1} << 23) && a.ldw < (int64_t{1} << 23);
}

// ---- any shape, stride and alignment ----------------------------------------
//
// Tile 64 tokens x 64 channels, four waves of 32 x 32, k steps of 64.  Both
// operands go through registers (16 bytes a thread, loads of any alignment,
// the row's last bytes one at a time) into a double-buffered LDS tile kept in
// operand order: 16-row group, 16-byte chunk, row.
constexpr int kAnyTile = 64;

// 16 operand bytes from channel j0 on of a row with n channels, zeros beyond.
template <bool A4>
__device__ __forceinline__ i32x4_t any_load(const uint8_t* p, int j0, int n) {
  uint32_t w[4] = {0, 0, 0, 0};
  if (A4) {
    uint32_t c[2] = {0, 0};
    const int left = (n - j0) / 2;
    if (left >= 8) {
      memcpy(c, p + j0 / 2, 8);
    } else {
      for (int i = 0; i < left; ++i) c[i >> 2] |= static_cast<uint32_t>(p[j0 / 2 + i]) << (8 * (i & 3));
    }
    widen8(c[0], w[0], w[1]);
    widen8(c[1], w[2], w[3]);
  } else {
    const int left = n - j0;
    if (left >= 16) {
      memcpy(w, p + j0, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (i < left) w[i >> 2] |= static_cast<uint32_t>(p[j0 + i]) << (8 * (i & 3));
    }
  }
  return i32x4_t{static_cast<int>(w[0]), static_cast<int>(w[1]), static_cast<int>(w[2]), static_cast<int>(w[3])};
}

template <bool A4>
__global__ __launch_bounds__(256) void w8_any_kernel(W8Args a) {
  __shared__ i32x4_t lds[2][2][kAnyTile * 4];  // [buffer][weights, tokens]
  const int tid = threadIdx.x, lane = tid & 63, wid = tid >> 6;
  const int tiles_n = (a.R + kAnyTile - 1) / kAnyTile;
  const int m0 = static_cast<int>(blockIdx.x / tiles_n) * kAnyTile;
  const int n0 = static_cast<int>(blockIdx.x % tiles_n) * kAnyTile;
  // thread -> tile row tid / 4, chunk tid % 4; rows clamped (not stored)
  const int r = tid >> 2, c = tid & 3;
  const uint8_t* pw = reinterpret_cast<const uint8_t*>(a.w) + static_cast<int64_t>(min(n0 + r, a.R - 1)) * a.ldw;
  const uint8_t* pt = a.a + static_cast<int64_t>(min(m0 + r, a.T - 1)) * a.lda;
  const int slot = (r >> 4) * 64 + c * 16 + (r & 15);
  const int steps = (a.n + 63) / 64;
  const int wk = 2 * (wid & 1), wt = 2 * (wid >> 1);  // first 16-row group of channels and of tokens
  i32x4_t acc[2][2] = {};
  i32x4_t vw = any_load<false>(pw, 16 * c, a.n), vt = any_load<A4>(pt, 16 * c, a.n);
  for (int s = 0; s < steps; ++s) {
    const int b = s & 1;
    lds[b][0][slot] = vw;
    lds[b][1][slot] = vt;
    __syncthreads();
    if (s + 1 < steps) {
      vw = any_load<false>(pw, 64 * (s + 1) + 16 * c, a.n);
      vt = any_load<A4>(pt, 64 * (s + 1) + 16 * c, a.n);
    }
    i32x4_t fw[2], ft[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      fw[i] = lds[b][0][(wk + i) * 64 + lane];
      ft[i] = lds[b][1][(wt + i) * 64 + lane];
    }
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(fw[i], ft[j], acc[i][j], 0, 0, 0);
  }
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    const int t = m0 + 16 * (wt + j) + (lane & 15);
    if (t >= a.T) continue;
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int k = n0 + 16 * (wk + i) + 4 * (lane >> 4) + e;
        if (k < a.R) row::store_elem(a.out, static_cast<int64_t>(t) * a.ldo + k, finish(a, t, k, acc[i][j][e]), a.out_bf16);
      }
  }
}

}  // namespace

int64_t w8_workspace(int64_t, int64_t, int64_t, bool) { return 0; }

const char* w8_name(const W8Args& a) { return aligned_rows(a) && a.T > 64 ? "w8_tile" : "w8_any"; }

hipError_t launch_w8(const W8Args& all, hipStream_t s) {
  // a launch holds fewer than 2^32 threads in one dimension: token ranges of at most 2^22 tiles
  const int64_t tiles_n = (static_cast<int64_t>(all.R) + kAnyTile - 1) / kAnyTile;
  if (tiles_n > (int64_t{1} << 22)) return hipErrorInvalidConfiguration;
  const int64_t step = ((int64_t{1} << 22) / tiles_n) * kAnyTile;
  for (int64_t t = 0; t < all.T; t += step) {
    W8Args a = all;
    a.T = static_cast<int>(step < all.T - t ? step : all.T - t);
    a.a += t * a.lda;
    a.scale += t;
    if (a.a4) a.zero += t;
    a.out = static_cast<uint8_t*>(a.out) + t * a.ldo * (a.out_bf16 ? 2 : 4);
    if (aligned_rows(a) && a.T > 64) {
      if (a.a4)
        run_tile<true, 2, 4, 8, 4, 4>(a, s);
      else
        run_tile<false, 4, 2, 4, 8, 4>(a, s);
      continue;
    }
    const dim3 grid(static_cast<unsigned>(((a.T + kAnyTile - 1) / kAnyTile) * tiles_n)), block(256);
    if (a.a4)
      w8_any_kernel<true><<<grid, block, 0, s>>>(a);
    else
      w8_any_kernel<false><<<grid, block, 0, s>>>(a);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

}  // namespace signrot
