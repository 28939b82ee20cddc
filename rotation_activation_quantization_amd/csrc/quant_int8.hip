// The symmetric per-token INT8 quantizer: scale = max |x| / 127 and
// q = rint(127 x / max |x|), one work-group per row.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "row_ops.h"

namespace signrot {
namespace {

constexpr int kThreads = 256;

__global__ __launch_bounds__(kThreads) void quant_int8_any_kernel(const uint16_t* __restrict__ x, int n, int64_t ld,
                                                                 int8_t* __restrict__ codes, int64_t ldc,
                                                                 float* __restrict__ scale, int32_t* __restrict__ sum,
                                                                 int64_t tokens) {
  __shared__ uint32_t sh[kThreads / 64];
  __shared__ int32_t shi[kThreads / 64];
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
  const uint16_t* xr = x + t * ld;
  uint32_t top = 0;
  for (int j = threadIdx.x; j < n; j += kThreads) top = row::add(top, row::abs_bits(row::bf16_f32(xr[j])));
  const float a = __uint_as_float(row::block_reduce(top, sh));
  int32_t total = 0;
  for (int j = threadIdx.x; j < n; j += kThreads) {
    const int q = row::code_of(row::bf16_f32(xr[j]), a);
    codes[t * ldc + j] = static_cast<int8_t>(q);
    total += q;
  }
  if (threadIdx.x == 0) scale[t] = row::scale_of(a);
  if (sum) {
    total = row::block_reduce(total, shi);
    if (threadIdx.x == 0) sum[t] = total;
  }
  }
}

}  // namespace

hipError_t launch_quant_int8(const uint16_t* x, int64_t tokens, int n, int64_t ld, int8_t* codes, int64_t ldc,
                             float* scale, int32_t* sum, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>(tokens < row::kMaxBlocks ? tokens : row::kMaxBlocks);
  quant_int8_any_kernel<<<dim3(blocks), dim3(kThreads), 0, s>>>(x, n, ld, codes, ldc, scale, sum, tokens);
  return hipGetLastError();
}

}  // namespace signrot
