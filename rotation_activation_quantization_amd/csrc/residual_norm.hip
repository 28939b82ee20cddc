// The norm after a block, its gate and residual scale, the residual sum and
// the norm before the next block in one launch:
//
//   h' = beta h + alpha g Norm_post(y),  u = Norm_pre(h') (1 + m) + c,
//
// u stored as bf16 and/or as symmetric per-token INT8 codes.
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "row_ops.h"

namespace signrot {
namespace {

using NormArgs = signrot_residual_norm_args;

constexpr int kThreads = 256;

// Any width, stride and alignment: one work-group per row, every pass
// recomputes the row's values from memory (the row is in cache after the
// first).  Thread i owns the elements i, i + 256, ... in every pass, so h_out
// may be h.
__global__ __launch_bounds__(kThreads) void residual_norm_any_kernel(NormArgs a) {
  __shared__ float sh[kThreads / 64];
  __shared__ uint32_t shm[kThreads / 64];
  const int n = static_cast<int>(a.n);
  const float inv_n = 1.f / static_cast<float>(n);
  const int hb = a.h_type == SIGNROT_BF16, pb = a.param_type == SIGNROT_BF16;
  const int tid = threadIdx.x;
  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
  int64_t r = t;
  if (a.mod_index) {
    const int64_t i = a.mod_index[t];
    r = i < 0 ? 0 : (i >= a.mod_rows ? a.mod_rows - 1 : i);
  }
  const int64_t gate_at = a.ldg ? r * a.ldg : 0, mod_at = a.ldm ? r * a.ldm : 0;
  const int64_t h_at = t * a.ldh, y_at = t * a.ldy;

  // mean and 1 / sqrt(var + eps) of the n values of f
  auto stats = [&](auto f, int kind, float eps, float& mean, float& inv) {
    mean = 0.f;
    inv = 1.f;
    if (kind == SIGNROT_NORM_NONE) return;
    if (kind == SIGNROT_NORM_LAYER) {
      float s = 0.f;
      for (int j = tid; j < n; j += kThreads) s += f(j);
      mean = row::block_reduce(s, sh) * inv_n;
    }
    float q = 0.f;
    for (int j = tid; j < n; j += kThreads) {
      const float d = f(j) - mean;
      q = fmaf(d, d, q);
    }
    inv = 1.f / sqrtf(row::block_reduce(q, sh) * inv_n + eps);
  };
  auto affine = [&](float v, int kind, float mean, float inv, const void* w, const void* b, int j) {
    if (kind == SIGNROT_NORM_NONE) return v;
    v = (v - mean) * inv;
    if (w) v *= row::load_elem(w, j, pb);
    if (b) v += row::load_elem(b, j, pb);
    return v;
  };

  float mean_y = 0.f, inv_y = 1.f, mean_h, inv_h;
  if (a.y)
    stats([&](int j) { return row::load_elem(a.y, y_at + j, 1); }, a.post_norm, a.eps_post, mean_y, inv_y);
  auto stream = [&](int j) {
    float v = a.beta * row::load_elem(a.h, h_at + j, hb);
    if (a.y) {
      float b = affine(row::load_elem(a.y, y_at + j, 1), a.post_norm, mean_y, inv_y, a.post_weight, a.post_bias, j);
      if (a.gate) b *= row::load_elem(a.gate, gate_at + j, pb);
      v = fmaf(a.alpha, b, v);
    }
    return v;
  };
  stats(stream, a.pre_norm, a.eps_pre, mean_h, inv_h);
  auto out = [&](float v, int j) {
    v = affine(v, a.pre_norm, mean_h, inv_h, a.pre_weight, a.pre_bias, j);
    if (a.mod_scale) v *= 1.f + row::load_elem(a.mod_scale, mod_at + j, pb);
    if (a.mod_shift) v += row::load_elem(a.mod_shift, mod_at + j, pb);
    return v;
  };
  float top = 0.f;
  if (a.codes) {
    uint32_t m = 0;
    for (int j = tid; j < n; j += kThreads) m = row::add(m, row::abs_bits(out(stream(j), j)));
    top = __uint_as_float(row::block_reduce(m, shm));
    if (tid == 0) a.code_scale[t] = row::scale_of(top);
  }
  for (int j = tid; j < n; j += kThreads) {
    const float v = stream(j);
    const float u = out(v, j);
    if (a.h_out) row::store_elem(a.h_out, t * a.ldho + j, v, hb);
    if (a.u) row::store_elem(a.u, t * a.ldu + j, u, 1);
    if (a.codes) a.codes[t * a.ldc + j] = static_cast<int8_t>(row::code_of(u, top));
  }
  }
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs& a, hipStream_t s) {
  const unsigned blocks = static_cast<unsigned>(a.tokens < row::kMaxBlocks ? a.tokens : row::kMaxBlocks);
  residual_norm_any_kernel<<<dim3(blocks), dim3(kThreads), 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace signrot
