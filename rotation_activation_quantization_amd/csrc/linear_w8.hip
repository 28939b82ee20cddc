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

const char* w8_name(const W8Args&) { return "w8_any"; }

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
