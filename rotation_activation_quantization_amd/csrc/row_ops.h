// Helpers of the kernels that reduce rows of activations (the INT8 quantizer
// and the residual norms): element access by type, wave and work-group
// reductions and the INT8 codes of a row.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace signrot {
namespace row {

typedef __attribute__((__vector_size__(4 * sizeof(uint32_t)))) uint32_t u32x4_t;
typedef __attribute__((__vector_size__(2 * sizeof(uint32_t)))) uint32_t u32x2_t;

// Work-groups of a launch over rows: a launch holds fewer than 2^32 threads,
// so the kernels stride over the rows beyond.
constexpr int64_t kMaxBlocks = 1 << 20;

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float(static_cast<uint32_t>(b) << 16); }

// Round to nearest even through the hardware conversion (NaN stays NaN).
__device__ __forceinline__ uint16_t f32_bf16(float f) { return __builtin_bit_cast(uint16_t, static_cast<__bf16>(f)); }
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef float f32x2_t __attribute__((ext_vector_type(2)));
  typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{lo, hi}, bf16x2_t));
}

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

// Eight values of a 16-byte chunk of bf16.
__device__ __forceinline__ void widen_bf16(const u32x4_t& w, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
// Sixteen or eight bytes at an aligned address, or at any (the hardware takes
// those; the compiler has to be told).
template <bool ALIGNED, typename T>
__device__ __forceinline__ T load_as(const void* p) {
  if (ALIGNED) return *static_cast<const T*>(p);
  T v;
  __builtin_memcpy(&v, p, sizeof(T));
  return v;
}
template <bool ALIGNED, typename T>
__device__ __forceinline__ void store_as(void* p, const T& v) {
  if (ALIGNED)
    *static_cast<T*>(p) = v;
  else
    __builtin_memcpy(p, &v, sizeof(T));
}

// Eight consecutive elements from j on.
template <bool ALIGNED>
__device__ __forceinline__ void load8(const void* p, int64_t j, int bf16, float (&v)[8]) {
  if (bf16) {
    widen_bf16(load_as<ALIGNED, u32x4_t>(static_cast<const uint16_t*>(p) + j), v);
  } else {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const u32x4_t w = load_as<ALIGNED, u32x4_t>(static_cast<const float*>(p) + j + 4 * i);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[4 * i + e] = __uint_as_float(w[e]);
    }
  }
}

// The rows kernels hold a row as chunks of eight elements.  Rows of whole,
// aligned chunks (WHOLE) are read and written as vectors.  In other rows (n >= 8)
// the vectors lie at any address, and the last chunk is moved back to the row's
// last eight elements: the first `dup` of them belong to the chunk before, are
// left out of every sum and maximum, and are not stored again (the other
// thread may have stored them already, over an input that is the output).
template <bool WHOLE>
struct Chunk {
  int at;   // first element
  int dup;  // elements of the chunk before
  __device__ __forceinline__ Chunk(int c, int n) : at(WHOLE ? 8 * c : min(8 * c, n - 8)), dup(8 * c - at) {}
  __device__ __forceinline__ bool own(int e) const { return WHOLE || e >= dup; }
};

// |x| as ordered bits: for finite values the order of the magnitudes, with
// infinity above them and NaN above infinity, so a maximum over a row keeps
// whatever is not finite.
__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7fffffffu; }

__device__ __forceinline__ float join(float a, float b) { return a + b; }
__device__ __forceinline__ int32_t join(int32_t a, int32_t b) { return a + b; }
__device__ __forceinline__ uint32_t join(uint32_t a, uint32_t b) { return a > b ? a : b; }  // maximum of abs_bits

template <int CTRL, typename T>
__device__ __forceinline__ T dpp(T v) {
  return __builtin_bit_cast(T, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xf, 0xf, true));
}
template <typename T>
__device__ __forceinline__ T lane_of(T v, int lane) {
  return __builtin_bit_cast(T, __builtin_amdgcn_readlane(__builtin_bit_cast(int, v), lane));
}

// Reduction over the wave, the same value in every lane: lane ^ 1, lane ^ 2,
// mirror in 8 and in 16 by DPP, then the four rows of sixteen.
template <typename T>
__device__ __forceinline__ T wave_reduce(T v) {
  v = join(v, dpp<0xB1>(v));   // quad_perm 1, 0, 3, 2
  v = join(v, dpp<0x4E>(v));   // quad_perm 2, 3, 0, 1
  v = join(v, dpp<0x141>(v));  // row_half_mirror
  v = join(v, dpp<0x140>(v));  // row_mirror
  return join(join(lane_of(v, 0), lane_of(v, 16)), join(lane_of(v, 32), lane_of(v, 48)));
}

// Reduction over the work-group (float and int32 sums, uint32 maximum); every
// thread gets the result.  Called by all threads.  `sh` holds one word for
// each of up to sixteen waves; one barrier: the caller passes other words the
// next time, or has a barrier in between.
template <typename T>
__device__ __forceinline__ T block_reduce(T v, T* sh) {
  v = wave_reduce(v);
  const int waves = blockDim.x >> 6;
  if (waves == 1) return v;
  if ((threadIdx.x & 63) == 0) sh[threadIdx.x >> 6] = v;
  __syncthreads();
  T r = sh[0];
  for (int i = 1; i < waves; ++i) r = join(r, sh[i]);
  return r;
}

// The INT8 codes of a row whose largest magnitude is a: rint(127 x / a), 0 in
// an all-zero row.  The quotient is one Newton step on x' r, x' = 127 s x and
// r = 1 / (a s): with the remainder x' - q (a s) exact in a fused
// multiply-add, the step rounds the true quotient to nearest (Markstein 1990).
// Where x and a are bf16 numbers x' is exact, a representable quotient (among
// them the ties k + 1/2) comes out exactly, and any other one is further than
// 2^-9 relative from a tie: the code is the exact rint.  The power of two s
// keeps r and x' clear of overflow and of subnormals.
struct Codes {
  float mul, a, r;
  __device__ __forceinline__ explicit Codes(float top) {
    const float s = top < 0x1p-60f ? 0x1p100f : (top > 0x1p60f ? 0x1p-100f : 1.f);
    mul = 127.f * s;
    a = top * s;
    r = top > 0.f ? 1.f / a : 0.f;
  }
  // The code in the low byte (two's complement): 1.5 * 2^23 is added, which
  // rounds to a whole number, ties to even.
  __device__ __forceinline__ uint32_t bits(float x) const {
    const float v = x * mul;
    const float q = v * r;
    return __float_as_uint(fmaf(fmaf(-q, a, v), r, q) + 12582912.f);
  }
};
// Four codes in one word.
__device__ __forceinline__ uint32_t pack_codes(uint32_t b0, uint32_t b1, uint32_t b2, uint32_t b3) {
  const uint32_t lo = __builtin_amdgcn_perm(b1, b0, 0x0c0c0400u), hi = __builtin_amdgcn_perm(b3, b2, 0x0c0c0400u);
  return __builtin_amdgcn_perm(hi, lo, 0x05040100u);
}
__device__ __forceinline__ float scale_of(float top) { return top == 0.f ? 1.f : top / 127.f; }

// How many 16-byte chunks of a row a thread holds, and the threads of the
// row's work-group (whole waves, at most 1024).  With up to 512 rows (two
// work-groups a CU) one chunk: the norms take 3.8 us on 1 x 4096 and 5.4 us on
// 256 x 4096, with two chunks 4.4 and 6.0.  With more rows two chunks: 12.7 us
// on 1237 x 5120, 46.4 on 8192 x 4096, 99.8 on 8192 x 8192, with one 17.0, 55.3
// and 142.2 (twice the waves to pass the reductions' barriers), with four 15.0,
// 52.0 and 109.4 (half the waves in flight).  More where the work-group would
// not hold the row.
inline int chunks_per_thread(int chunks, int64_t tokens) {
  int v = tokens <= 512 ? 1 : 2;
  while ((chunks + v - 1) / v > 1024) v *= 2;
  return v;
}
inline int threads_for(int chunks, int v) { return ((chunks + v - 1) / v + 63) / 64 * 64; }

}  // namespace row
}  // namespace signrot
