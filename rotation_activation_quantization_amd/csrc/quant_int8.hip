// The symmetric per-token INT8 quantizer: scale = max |x| / 127 and
// q = rint(127 x / max |x|).
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "row_ops.h"

namespace signrot {
namespace {

// One work-group per row, the row in registers (V chunks of eight values a
// thread), so it is read once.  Bound by memory: 8192 x 4096 23 us between two
// large products (4.4 TB/s), and by latency for one row (2.5 us at 4096).
template <int V, bool WHOLE>
__global__ __launch_bounds__(1024) void quant_int8_rows_kernel(const uint16_t* __restrict__ x, int n, int64_t ld,
                                                              int8_t* __restrict__ codes, int64_t ldc,
                                                              float* __restrict__ scale, int32_t* __restrict__ sum,
                                                              int64_t tokens) {
  __shared__ uint32_t sh_top[16];
  __shared__ int32_t sh_sum[16];
  const int chunks = (n + 7) >> 3, step = blockDim.x;
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    const uint16_t* const xr = x + t * ld;
    row::u32x4_t w[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = static_cast<int>(threadIdx.x) + v * step;
      w[v] = row::u32x4_t{0, 0, 0, 0};
      if (c < chunks) w[v] = row::load_as<WHOLE, row::u32x4_t>(xr + row::Chunk<WHOLE>(c, n).at);
    }
    uint32_t top = 0;
#pragma unroll
    for (int v = 0; v < V; ++v)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        top = row::join(top, row::join((w[v][i] << 16) & 0x7fffffffu, w[v][i] & 0x7fff0000u));
    const float a = __uint_as_float(row::block_reduce(top, sh_top));
    const row::Codes code(a);
    int32_t total = 0;
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = static_cast<int>(threadIdx.x) + v * step;
      float f[8];
      row::widen_bf16(w[v], f);
      row::u32x2_t q;
#pragma unroll
      for (int h = 0; h < 2; ++h)
        q[h] = row::pack_codes(code.bits(f[4 * h]), code.bits(f[4 * h + 1]), code.bits(f[4 * h + 2]),
                               code.bits(f[4 * h + 3]));
      const row::Chunk<WHOLE> k(c, n);
      if (sum) {
        if (WHOLE || k.dup == 0) {
#pragma unroll
          for (int h = 0; h < 2; ++h)
            total = __builtin_amdgcn_sdot4(static_cast<int>(q[h]), 0x01010101, total, false);
        } else if (c < chunks) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (k.own(e)) total += static_cast<int8_t>(q[e >> 2] >> (8 * (e & 3)));
        }
      }
      int8_t* const out = codes + t * ldc + k.at;
      if (c < chunks) {
        if (WHOLE || k.dup == 0) {
          row::store_as<WHOLE>(out, q);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (k.own(e)) out[e] = static_cast<int8_t>(q[e >> 2] >> (8 * (e & 3)));
        }
      }
    }
    if (threadIdx.x == 0) scale[t] = row::scale_of(a);
    if (sum) {
      total = row::block_reduce(total, sh_sum);
      if (threadIdx.x == 0) sum[t] = total;
    }
    if (t + gridDim.x < tokens) __syncthreads();  // sh_top and sh_sum are used again
  }
}

// Rows of fewer than eight values or more than 65536: read twice, element by
// element.
constexpr int kAnyThreads = 256;
__global__ __launch_bounds__(kAnyThreads) void quant_int8_any_kernel(const uint16_t* __restrict__ x, int n, int64_t ld,
                                                                    int8_t* __restrict__ codes, int64_t ldc,
                                                                    float* __restrict__ scale,
                                                                    int32_t* __restrict__ sum, int64_t tokens) {
  __shared__ uint32_t sh_top[16];
  __shared__ int32_t sh_sum[16];
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    const uint16_t* xr = x + t * ld;
    uint32_t top = 0;
    for (int j = threadIdx.x; j < n; j += kAnyThreads) top = row::join(top, xr[j] & 0x7fffu);
    const float a = __uint_as_float(row::block_reduce(top, sh_top) << 16);
    const row::Codes code(a);
    int32_t total = 0;
    for (int j = threadIdx.x; j < n; j += kAnyThreads) {
      const int8_t q = static_cast<int8_t>(code.bits(row::bf16_f32(xr[j])));
      codes[t * ldc + j] = q;
      total += q;
    }
    if (threadIdx.x == 0) scale[t] = row::scale_of(a);
    if (sum) {
      total = row::block_reduce(total, sh_sum);
      if (threadIdx.x == 0) sum[t] = total;
    }
    if (t + gridDim.x < tokens) __syncthreads();
  }
}

template <bool WHOLE>
void run_rows(const uint16_t* x, int64_t tokens, int n, int64_t ld, int8_t* codes, int64_t ldc, float* scale,
              int32_t* sum, dim3 grid, hipStream_t s) {
  const int chunks = (n + 7) / 8;
  const int v = row::chunks_per_thread(chunks, tokens);
  const dim3 block(static_cast<unsigned>(row::threads_for(chunks, v)));
  switch (v) {
    case 1: quant_int8_rows_kernel<1, WHOLE><<<grid, block, 0, s>>>(x, n, ld, codes, ldc, scale, sum, tokens); break;
    case 2: quant_int8_rows_kernel<2, WHOLE><<<grid, block, 0, s>>>(x, n, ld, codes, ldc, scale, sum, tokens); break;
    case 4: quant_int8_rows_kernel<4, WHOLE><<<grid, block, 0, s>>>(x, n, ld, codes, ldc, scale, sum, tokens); break;
    default: quant_int8_rows_kernel<8, WHOLE><<<grid, block, 0, s>>>(x, n, ld, codes, ldc, scale, sum, tokens); break;
  }
}

}  // namespace

hipError_t launch_quant_int8(const uint16_t* x, int64_t tokens, int n, int64_t ld, int8_t* codes, int64_t ldc,
                             float* scale, int32_t* sum, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(tokens < row::kMaxBlocks ? tokens : row::kMaxBlocks));
  const bool whole = n % 8 == 0 && ld % 8 == 0 && ldc % 8 == 0 && (reinterpret_cast<uintptr_t>(x) & 15u) == 0 &&
                     (reinterpret_cast<uintptr_t>(codes) & 7u) == 0;
  if (n < 8 || n > 8 * 8 * 1024)
    quant_int8_any_kernel<<<grid, dim3(kAnyThreads), 0, s>>>(x, n, ld, codes, ldc, scale, sum, tokens);
  else if (whole)
    run_rows<true>(x, tokens, n, ld, codes, ldc, scale, sum, grid, s);
  else
    run_rows<false>(x, tokens, n, ld, codes, ldc, scale, sum, grid, s);
  return hipGetLastError();
}

}  // namespace signrot
