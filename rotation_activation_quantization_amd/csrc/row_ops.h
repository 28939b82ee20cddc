// Helpers of the kernels that reduce rows of activations (the INT8 quantizer
// and the residual norms): element access by type, work-group reductions and
// the INT8 code of a value.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace signrot {
namespace row {

// Work-groups of a launch over rows: a launch holds fewer than 2^32 threads,
// so the kernels stride over the rows beyond.
constexpr int64_t kMaxBlocks = 1 << 20;

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

// Round to nearest even through the hardware conversion (NaN stays NaN).
__device__ __forceinline__ uint16_t f32_bf16(float f) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f)); }

// Element j of a row of binary32 (bf16 == 0) or bf16 values.
__device__ __forceinline__ float load_elem(const void* p, int64_t j, int bf16) {
  return bf16 ? bf16_f32(static_cast<const uint16_t*>(p)[j]) : static_cast<const float*>(p)[j];
}
__device__ __forceinline__ void store_elem(void* p, int64_t j, float v, int bf16) {
  if (bf16)
    static_cast<uint16_t*>(p)[j] = f32_bf16(v);
  else
    static_cast<float*>(p)[j] = v;
}

// |x| as ordered bits: for finite values the order of the magnitudes, with
// infinity above them and NaN above infinity, so a maximum over a row keeps
// whatever is not finite.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ float add(float a, float b) { return a + b; }
__device__ __forceinline__ int32_t add(int32_t a, int32_t b) { return a + b; }
__device__ __forceinline__ uint32_t add(uint32_t a, uint32_t b) { return a > b ? a : b; }  // the maximum of abs_bits

// Reduction over the work-group (float and int32 sums, uint32 maximum); every
// thread gets the result.  Called by all threads; `sh` holds one word per
// wave and is free again when the call returns in every thread.
template <typename T>
__device__ __forceinline__ T block_reduce(T v, T* sh) {
#pragma unroll
  for (int m = 32; m > 0; m >>= 1) v = add(v, __shfl_xor(v, m));
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  T r = sh[0];
  for (int i = 1; i < waves; ++i) r = add(r, sh[i]);
  __syncthreads();
  return r;
}

// The code of u in a row whose largest magnitude is a: rint(127 u / a), with
// 0 for an all-zero row.  127 u / a is the binary32 quotient correctly
// rounded; where u and a are bf16 numbers 127 u is exact and no quotient
// other than an exact tie rounds onto one, so the code is exact.
__device__ __forceinline__ int code_of(float u, float a) {
  if (!(a > 0.f)) return 0;
  const float q = rintf(127.f * u / a);
  return static_cast<int>(fminf(fmaxf(q, -127.f), 127.f));
}
__device__ __forceinline__ float scale_of(float a) { return a == 0.f ? 1.f : a / 127.f; }

}  // namespace row
}  // namespace signrot
