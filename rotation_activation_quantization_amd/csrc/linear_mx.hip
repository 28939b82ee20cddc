// The product of MXFP4 operands,
//
//   out[t][k] = sum_j x[t][j] w[k][j] + b[k],
//
// on v_mfma_scale_f32_16x16x128_f8f6f4, which multiplies the codes and applies
// both blocks' scales; the sum is binary32.  The weights are the MFMA's A
// operand and the tokens its B operand, so that a lane's four results are
// consecutive output channels of one token.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "mx_ops.h"
#include "row_ops.h"
#include "wave_ops.h"

namespace signrot {
namespace {

typedef __attribute__((__vector_size__(8 * sizeof(int32_t)))) int32_t i32x8_t;
typedef __attribute__((__vector_size__(4 * sizeof(int32_t)))) int32_t i32x4_t;
using wave::f32x4_t;

constexpr int kFp4 = 4;  // format number of E2M1 in the MFMA

__device__ __forceinline__ f32x4_t mfma(const i32x4_t& a, const i32x4_t& b, const f32x4_t& c, int sa, int sb) {
  const i32x8_t wa = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, wb = {b[0], b[1], b[2], b[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wa, wb, c, kFp4, kFp4, 0, sa, 0, sb);
}

// 64 channels x 64 tokens, a wave sixteen channels; lane (g, i) holds block g
// of a step of four, of row i.
__global__ __launch_bounds__(256) void mx_any_kernel(MxArgs a) {
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6, g = lane >> 4, i = lane & 15;
  const int tiles_n = (a.R + 63) / 64;
  const int m0 = 64 * static_cast<int>(blockIdx.x / tiles_n), n0 = 64 * static_cast<int>(blockIdx.x % tiles_n) + 16 * wid;
  const int blocks = a.n / mx::kBlock;
  const int64_t kr = min(n0 + i, a.R - 1);
  const uint8_t* const w = a.w + kr * a.ldw;
  const uint8_t* const ws = a.w_scale + kr * a.ldws;
  f32x4_t acc[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) acc[j] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int kb = g; kb < blocks + g; kb += 4) {
    const bool in = kb < blocks;
    i32x4_t x = {0, 0, 0, 0};
    int s = 127;
    if (in) {
      x = row::load_as<false, i32x4_t>(w + mx::kBlockBytes * static_cast<int64_t>(kb));
      s = ws[kb];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t t = min(m0 + 16 * j + i, a.T - 1);
      i32x4_t y = {0, 0, 0, 0};
      int st = 127;
      if (in) {
        y = row::load_as<false, i32x4_t>(a.a + t * a.lda + mx::kBlockBytes * static_cast<int64_t>(kb));
        st = a.scale[t * a.lds + kb];
      }
      acc[j] = mfma(x, y, acc[j], s, st);
    }
  }
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int t = m0 + 16 * j + i;
    if (t >= a.T) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int k = n0 + 4 * g + e;
      if (k < a.R)
        row::store_elem(a.out, static_cast<int64_t>(t) * a.ldo + k, acc[j][e] + (a.bias ? a.bias[k] : 0.f), a.out_bf16);
    }
  }
}

}  // namespace

int64_t mx_workspace(const MxArgs& a) {
  (void)a;
  return 0;
}

const char* mx_name(const MxArgs& a) {
  (void)a;
  return "mx_any";
}

hipError_t launch_mx(const MxArgs& a, hipStream_t s) {
  const int64_t tiles = static_cast<int64_t>((a.T + 63) / 64) * ((a.R + 63) / 64);
  mx_any_kernel<<<dim3(static_cast<unsigned>(tiles)), dim3(256), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace signrot
