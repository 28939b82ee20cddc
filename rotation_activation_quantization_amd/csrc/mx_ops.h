// Microscaled 4-bit floating point (MXFP4): blocks of 32 values, each a sign
// and a magnitude of 0, 0.5, 1, 1.5, 2, 3, 4, 6 (E2M1), times the power of two
// 2^(b - 127) of the block's scale byte b (E8M0; 255 is NaN).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace signrot {
namespace mx {

constexpr int kBlock = 32;        // values of a block
constexpr int kBlockBytes = 16;   // of its codes
constexpr uint32_t kNan = 255;    // scale byte of a block that holds an infinity or NaN

// Scale byte of a block whose largest magnitude has the binary32 bits `top`:
// the exponent of top less that of 4, so that top / 2^e lies in [4, 8) and
// what is over 6 saturates ("floor"); with `noclip` one more where it is over
// 6.  Blocks below 2^-125 take the least scale, 2^-127.
__device__ __forceinline__ uint32_t scale_byte(uint32_t top, int noclip) {
  if (top >= 0x7f800000u) return kNan;
  const int e = static_cast<int>(top >> 23) - 2 + ((noclip && (top & 0x7fffffu) > 0x400000u) ? 1 : 0);
  return static_cast<uint32_t>(max(e, 0));
}

// 2^(b - 127) for b < 255.
__device__ __forceinline__ float scale_of(uint32_t b) { return __uint_as_float(b ? b << 23 : 0x00400000u); }

typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

// Eight codes of a block with scale byte b in one word, value j in bits
// 4 j .. 4 j + 3: v / 2^e rounded to the nearest level, the even code at a tie,
// 6 for what is larger (the hardware conversion).  All zero in a NaN block.
__device__ __forceinline__ uint32_t codes_f32(const float* v, uint32_t b) {
  if (b == kNan) return 0;
  const float s = scale_of(b);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[0], v[1], s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[2], v[3], s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[4], v[5], s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, v[6], v[7], s, 3);
}
__device__ __forceinline__ uint32_t codes_bf16(const uint32_t (&w)[4], uint32_t b) {
  if (b == kNan) return 0;
  const float s = scale_of(b);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w[0]), s, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w[1]), s, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w[2]), s, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2_t, w[3]), s, 3);
}

// Maximum over the lanes that hold one block after the 16-point lane transform
// of the rotate kernels, the same in each.  There lane nl holds output number
// lane_perm(nl), so neighbouring outputs are lanes 6 apart (in the exclusive
// or), the next 5 and 7, then 8; the steps below generate the same groups from
// what DPP offers: 1, 2, 3, 7 and 8.
template <int CTRL>
__device__ __forceinline__ uint32_t from_lane(uint32_t v) {
  return static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), CTRL, 0xf, 0xf, true));
}
template <int LANES>
__device__ __forceinline__ uint32_t lanes_top(uint32_t v) {
  static_assert(LANES == 1 || LANES == 2 || LANES == 4 || LANES == 8 || LANES == 16, "lanes of a block");
  if (LANES == 4) v = max(v, from_lane<0x1B>(v));                      // quad_perm 3, 2, 1, 0
  if (LANES == 2 || LANES == 4) v = max(v, from_lane<0xB1>(from_lane<0x141>(v)));  // 7, then 1: 6
  if (LANES >= 8) {
    v = max(v, from_lane<0xB1>(v));   // quad_perm 1, 0, 3, 2
    v = max(v, from_lane<0x4E>(v));   // quad_perm 2, 3, 0, 1
    v = max(v, from_lane<0x141>(v));  // row_half_mirror
  }
  if (LANES == 16) v = max(v, from_lane<0x128>(v));  // row_ror:8
  return v;
}

}  // namespace mx
}  // namespace signrot
