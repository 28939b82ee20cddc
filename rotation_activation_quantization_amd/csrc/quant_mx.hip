// The MXFP4 quantizer and its inverse.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "mx_ops.h"
#include "row_ops.h"

namespace signrot {
namespace {

constexpr int kThreads = 256;

// Sixteen-byte chunk c of a launch -> row and chunk of the row, `per` chunks a
// row.  The launchers keep a launch below 2^31 chunks.
struct At {
  uint32_t row, chunk;
  __device__ __forceinline__ At(uint32_t c, uint32_t per) : row(c / per), chunk(c - row * per) {}
};

// Bound by memory: 8192 x 14336 bf16 55.6 us (5.35 TB/s), binary32 91.6 (5.8).
//
// A lane takes eight values and four neighbouring lanes a block, so that a
// wave reads 1 KiB (bf16) of one row side by side and writes 256 bytes of codes.
// The block's maximum is two DPP steps over the four lanes' bits.
// WHOLE: rows of whole, aligned chunks; else vectors at any address, and the
// chunk at the row's end value by value, zeros beyond it.
template <bool BF16, bool WHOLE>
__global__ __launch_bounds__(kThreads) void quant_mx_kernel(const void* __restrict__ x, int n, int64_t ld,
                                                            uint8_t* __restrict__ codes, int64_t ldc,
                                                            uint8_t* __restrict__ scale, int64_t lds, int noclip,
                                                            uint32_t chunks, uint32_t per) {
  const uint32_t c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= chunks) return;  // whole blocks: `per` is a multiple of four
  const At at(c, per);
  const int j = 8 * static_cast<int>(at.chunk);
  const int64_t first = at.row * ld + j;
  float v[8];
  uint32_t w[4] = {0, 0, 0, 0};
  uint32_t top = 0;
  if (BF16) {
    if (WHOLE ? j < n : j + 8 <= n) {
      const row::u32x4_t q = row::load_as<WHOLE, row::u32x4_t>(static_cast<const uint16_t*>(x) + first);
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = q[i];
    } else if (!WHOLE) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e < n) w[e >> 1] |= static_cast<uint32_t>(static_cast<const uint16_t*>(x)[first + e]) << (16 * (e & 1));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) top = row::join(top, row::join((w[i] << 16) & 0x7fffffffu, w[i] & 0x7fff0000u));
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = 0.f;
    if (WHOLE ? j < n : j + 8 <= n) {
      row::load8<WHOLE>(x, first, 0, v);
    } else if (!WHOLE) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (j + e < n) v[e] = static_cast<const float*>(x)[first + e];
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) top = row::join(top, row::abs_bits(v[e]));
  }
  top = row::join(top, row::dpp<0xB1>(top));  // quad_perm 1, 0, 3, 2
  top = row::join(top, row::dpp<0x4E>(top));  // quad_perm 2, 3, 0, 1
  const uint32_t b = mx::scale_byte(top, noclip);
  row::store_as<WHOLE>(codes + at.row * ldc + 4 * static_cast<int64_t>(at.chunk),
                       BF16 ? mx::codes_bf16(w, b) : mx::codes_f32(v, b));
  if ((threadIdx.x & 3) == 0) scale[at.row * lds + (at.chunk >> 2)] = static_cast<uint8_t>(b);
}

// A lane takes eight values: four bytes of codes, the block's scale, and 16 or
// 32 bytes out.
template <bool BF16, bool WHOLE>
__global__ __launch_bounds__(kThreads) void dequant_mx_kernel(const uint8_t* __restrict__ codes, int64_t ldc,
                                                              const uint8_t* __restrict__ scale, int64_t lds, int n,
                                                              void* __restrict__ y, int64_t ldy, uint32_t chunks,
                                                              uint32_t per, int stream) {
  const uint32_t c = blockIdx.x * kThreads + threadIdx.x;
  if (c >= chunks) return;
  const At at(c, per);
  const int j = 8 * static_cast<int>(at.chunk);
  const uint32_t b = scale[at.row * lds + (at.chunk >> 2)];
  const uint32_t q = row::load_as<WHOLE, uint32_t>(codes + at.row * ldc + 4 * static_cast<int64_t>(at.chunk));
  const float s = b == mx::kNan ? __uint_as_float(0x7fc00000u) : mx::scale_of(b);
  float v[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    // magnitudes 0, 1, 2, 3, 4, 6, 8, 12 halves
    const uint32_t m = (q >> (4 * e)) & 7u;
    const uint32_t h = (0xC8643210u >> (4 * m)) & 15u;
    const float a = 0.5f * static_cast<float>(h) * s;
    v[e] = (q >> (4 * e + 3)) & 1u ? -a : a;
  }
  const int64_t out = at.row * ldy + j;
  if (j + 8 <= n) {
    if (BF16) {
      row::store_chunk<WHOLE>(static_cast<uint16_t*>(y) + out,
                              row::u32x4_t{row::pack_bf16(v[0], v[1]), row::pack_bf16(v[2], v[3]),
                                           row::pack_bf16(v[4], v[5]), row::pack_bf16(v[6], v[7])},
                              stream);
    } else {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        row::store_as<WHOLE>(static_cast<float*>(y) + out + 4 * h,
                             row::u32x4_t{__float_as_uint(v[4 * h]), __float_as_uint(v[4 * h + 1]),
                                          __float_as_uint(v[4 * h + 2]), __float_as_uint(v[4 * h + 3])});
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (j + e < n) row::store_elem(y, out + e, v[e], BF16);
  }
}

// Launches over slices of rows with fewer than 2^31 chunks.
template <class Launch>
hipError_t over_rows(int64_t tokens, uint32_t per, Launch launch) {
  const int64_t most = ((int64_t{1} << 31) - kThreads) / per;
  for (int64_t t = 0; t < tokens; t += most) {
    const uint32_t chunks = static_cast<uint32_t>((tokens - t < most ? tokens - t : most) * per);
    launch(t, chunks, dim3((chunks + kThreads - 1) / kThreads));
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

bool aligned_to(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

}  // namespace

hipError_t launch_quant_mx(const void* x, int bf16, int64_t tokens, int n, int64_t ld, uint8_t* codes, int64_t ldc,
                           uint8_t* scale, int64_t lds, int noclip, hipStream_t s) {
  const uint32_t per = static_cast<uint32_t>((n + mx::kBlock - 1) / mx::kBlock) * 4;
  const int size = bf16 ? 2 : 4;
  const bool whole = n % 8 == 0 && ld % (16 / size) == 0 && aligned_to(x, 16) && ldc % 4 == 0 && aligned_to(codes, 4);
  return over_rows(tokens, per, [&](int64_t t, uint32_t chunks, dim3 grid) {
    const auto run = [&](auto kernel) {
      kernel<<<grid, kThreads, 0, s>>>(static_cast<const uint8_t*>(x) + t * ld * size, n, ld, codes + t * ldc, ldc,
                                       scale + t * lds, lds, noclip, chunks, per);
    };
    if (bf16)
      whole ? run(quant_mx_kernel<true, true>) : run(quant_mx_kernel<true, false>);
    else
      whole ? run(quant_mx_kernel<false, true>) : run(quant_mx_kernel<false, false>);
  });
}

hipError_t launch_dequant_mx(const uint8_t* codes, int64_t ldc, const uint8_t* scale, int64_t lds, int64_t tokens,
                             int n, void* y, int64_t ldy, int bf16, hipStream_t s) {
  const uint32_t per = static_cast<uint32_t>(n + 7) / 8;
  const int size = bf16 ? 2 : 4;
  const bool whole = n % 8 == 0 && ldy % (16 / size) == 0 && aligned_to(y, 16) && ldc % 4 == 0 && aligned_to(codes, 4);
  const int stream = row::past_caches(tokens * n, bf16);
  return over_rows(tokens, per, [&](int64_t t, uint32_t chunks, dim3 grid) {
    const auto run = [&](auto kernel) {
      kernel<<<grid, kThreads, 0, s>>>(codes + t * ldc, ldc, scale + t * lds, lds, n,
                                       static_cast<uint8_t*>(y) + t * ldy * size, ldy, chunks, per, stream);
    };
    if (bf16)
      whole ? run(dequant_mx_kernel<true, true>) : run(dequant_mx_kernel<true, false>);
    else
      whole ? run(dequant_mx_kernel<false, true>) : run(dequant_mx_kernel<false, false>);
  });
}

}  // namespace signrot
