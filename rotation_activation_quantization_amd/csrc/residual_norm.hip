// The norm after a block, its gate and residual scale, the residual sum and
// the norm before the next block in one launch:
//
//   h' = beta h + alpha g Norm_post(y),  u = Norm_pre(h') (1 + m) + c,
//
// u stored as bf16 and/or as symmetric per-token INT8 codes.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "row_ops.h"

namespace signrot {
namespace {

using NormArgs = signrot_residual_norm_args;

// Row of the modulations that token t takes.
__device__ __forceinline__ int64_t modulation_row(const NormArgs& a, int64_t t) {
  if (!a.mod_index) return t;
  const int64_t i = a.mod_index[t];
  return i < 0 ? 0 : (i >= a.mod_rows ? a.mod_rows - 1 : i);
}

// s / n for the sum s that every thread holds, inv_n = 1 / n rounded: one Newton
// step from s inv_n, which leaves a representable quotient exact.  So a row of n
// equal bf16 values, whose sum is exact, has that value as its mean and centres
// to zeros (s inv_n alone was a rounding off for two of three values at n = 1000
// or 28672, which the norm blew up to 0.1).  The mean is held in a scalar
// register: as a vector one it cost rows of two chunks a place on the CU (8192 x
// 1111 23.4 us, 22.0 so).
__device__ __forceinline__ float mean_of(float s, int n, float inv_n) {
  const float q = s * inv_n;
  return row::lane_of(fmaf(fmaf(-q, static_cast<float>(n), s), inv_n, q), 0);
}

// Squares of values around 2^64 and more pass binary32's range, and an infinite
// sum of them would make every result of a finite row zero.  Such a row's squares
// are summed again, scaled by this, which keeps the sum below 2^17 (2^129
// 2^-80)^2; eps (unless it is 2^86 or more) is below a rounding of their mean.
constexpr float kSmall = 0x1p-80f;

// One work-group per row, the row in registers (V chunks of eight values a
// thread).  y and h are read once, h' and u written once; the statistics are one
// or two reductions each (a LayerNorm's centred sum of squares follows its mean,
// so that it cannot cancel).  Many rows are bound by memory: 8192 x 8192 in bf16,
// RMS, 99 to 106 us, 5.1 to 5.4 TB/s, where a copy reaches 5.2; LayerNorms with
// modulations take 144, for four reductions and seven rows of parameters from L2.
// One row is bound by its latency: 3.7 us at 4096.  Registers decide how many
// rows a CU holds: a single reduction for mean and variance took twelve more
// and was slower (106 us at 8192 x 8192).
template <int V, bool HB, bool WHOLE>
__global__ __launch_bounds__(1024) void residual_norm_rows_kernel(NormArgs a) {
  __shared__ float sh[4][16];
  __shared__ uint32_t sh_top[16];
  const int n = static_cast<int>(a.n);
  const float inv_n = 1.f / static_cast<float>(n);
  const int pb = a.param_type == SIGNROT_BF16;
  const int chunks = (n + 7) >> 3, step = blockDim.x;
  const int tid = threadIdx.x;

  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const int64_t r = modulation_row(a, t);
    const int64_t gate_at = a.ldg ? r * a.ldg : 0, mod_at = a.ldm ? r * a.ldm : 0;
    // the rows as they are stored; zeros beyond the last chunk
    row::u32x4_t hw[V][HB ? 1 : 2], yw[V];
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = tid + v * step;
      yw[v] = row::u32x4_t{0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < (HB ? 1 : 2); ++i) hw[v][i] = row::u32x4_t{0, 0, 0, 0};
      if (c < chunks) {
        const int at = row::Chunk<WHOLE>(c, n).at;
        if (a.y) yw[v] = row::load_as<WHOLE, row::u32x4_t>(static_cast<const uint16_t*>(a.y) + t * a.ldy + at);
        const uint8_t* const hr = static_cast<const uint8_t*>(a.h) + (t * a.ldh + at) * (HB ? 2 : 4);
#pragma unroll
        for (int i = 0; i < (HB ? 1 : 2); ++i) hw[v][i] = row::load_as<WHOLE, row::u32x4_t>(hr + 16 * i);
      }
    }
    // mean and 1 / sqrt(var + eps) of the row whose chunk v is get(v)
    auto stats = [&](auto get, int kind, float eps, float* sh1, float* sh2, float& mean, float& inv) {
      mean = 0.f;
      inv = 1.f;
      if (kind == SIGNROT_NORM_NONE) return;
      if (kind == SIGNROT_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          float x[8];
          get(v, x);
          const row::Chunk<WHOLE> k(tid + v * step, n);
#pragma unroll
          for (int e = 0; e < 8; ++e) s += WHOLE || k.own(e) ? x[e] : 0.f;
        }
        mean = mean_of(row::block_reduce(s, sh1), n, inv_n);
      }
      float q = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = tid + v * step;
        if (c >= chunks) continue;
        float x[8];
        get(v, x);
        const row::Chunk<WHOLE> k(c, n);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float d = WHOLE || k.own(e) ? x[e] - mean : 0.f;
          q = fmaf(d, d, q);
        }
      }
      q = row::block_reduce(q, sh2);
      inv = 1.f / sqrtf(q * inv_n + eps);
      if (__builtin_expect(q == INFINITY, 0)) {  // every thread's q
        __syncthreads();
        q = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int c = tid + v * step;
          if (c >= chunks) continue;
          float x[8];
          get(v, x);
          const row::Chunk<WHOLE> k(c, n);
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const float d = WHOLE || k.own(e) ? (x[e] - mean) * kSmall : 0.f;
            q = fmaf(d, d, q);
          }
        }
        inv = kSmall / sqrtf(row::block_reduce(q, sh2) * inv_n);
      }
    };
    // x = (x - mean) inv w + b on the chunk from element j on
    auto affine = [&](float (&x)[8], int kind, float mean, float inv, const void* w, const void* b, int j) {
      if (kind == SIGNROT_NORM_NONE) return;
      float p[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = (x[e] - mean) * inv;
      if (w) {
        row::load8<WHOLE>(w, j, pb, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] *= p[e];
      }
      if (b) {
        row::load8<WHOLE>(b, j, pb, p);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] += p[e];
      }
    };

    float mean, inv, h[V][8];
    if (a.y)
      stats([&](int v, float (&x)[8]) { row::widen_bf16(yw[v], x); }, a.post_norm, a.eps_post, sh[0], sh[1], mean, inv);
#pragma unroll
    for (int v = 0; v < V; ++v) {
      const int c = tid + v * step;
      if (HB) {
        row::widen_bf16(hw[v][0], h[v]);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] = __uint_as_float(hw[v][HB ? 0 : e >> 2][e & 3]);
      }
      if (c >= chunks) continue;
      const row::Chunk<WHOLE> k(c, n);
#pragma unroll
      for (int e = 0; e < 8; ++e) h[v][e] *= a.beta;
      if (a.y) {
        float y[8];
        row::widen_bf16(yw[v], y);
        affine(y, a.post_norm, mean, inv, a.post_weight, a.post_bias, k.at);
        if (a.gate) {
          float p[8];
          row::load8<WHOLE>(a.gate, gate_at + k.at, pb, p);
#pragma unroll
          for (int e = 0; e < 8; ++e) y[e] *= p[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e) h[v][e] = fmaf(a.alpha, y[e], h[v][e]);
      }
      if (a.h_out) {
        uint8_t* const out = static_cast<uint8_t*>(a.h_out) + (t * a.ldho + k.at) * (HB ? 2 : 4);
        if (!WHOLE && k.dup > 0) {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            if (k.own(e)) row::store_elem(out, e, h[v][e], HB);
        } else if (HB) {
          row::u32x4_t w;
#pragma unroll
          for (int e = 0; e < 4; ++e) w[e] = row::pack_bf16(h[v][2 * e], h[v][2 * e + 1]);
          row::store_as<WHOLE>(out, w);
        } else {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            row::u32x4_t w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = __float_as_uint(h[v][4 * i + e]);
            row::store_as<WHOLE>(out + 16 * i, w);
          }
        }
      }
    }
    if (a.u || a.codes) {
      stats(
          [&](int v, float (&x)[8]) {
#pragma unroll
            for (int e = 0; e < 8; ++e) x[e] = h[v][e];
          },
          a.pre_norm, a.eps_pre, sh[2], sh[3], mean, inv);
      uint32_t top = 0;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = tid + v * step;
        if (c >= chunks) continue;
        const row::Chunk<WHOLE> k(c, n);
        affine(h[v], a.pre_norm, mean, inv, a.pre_weight, a.pre_bias, k.at);
        float p[8];
        if (a.mod_scale) {
          row::load8<WHOLE>(a.mod_scale, mod_at + k.at, pb, p);
#pragma unroll
          for (int e = 0; e < 8; ++e) h[v][e] = fmaf(h[v][e], p[e], h[v][e]);
        }
        if (a.mod_shift) {
          row::load8<WHOLE>(a.mod_shift, mod_at + k.at, pb, p);
#pragma unroll
          for (int e = 0; e < 8; ++e) h[v][e] += p[e];
        }
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (WHOLE || k.own(e)) top = row::join(top, row::abs_bits(h[v][e]));
        if (a.u) {
          uint16_t* const out = static_cast<uint16_t*>(a.u) + t * a.ldu + k.at;
          if (!WHOLE && k.dup > 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (k.own(e)) out[e] = row::f32_bf16(h[v][e]);
          } else {
            row::u32x4_t w;
#pragma unroll
            for (int e = 0; e < 4; ++e) w[e] = row::pack_bf16(h[v][2 * e], h[v][2 * e + 1]);
            row::store_as<WHOLE>(out, w);
          }
        }
      }
      if (a.codes) {
        const float m = __uint_as_float(row::block_reduce(top, sh_top));
        const row::Codes code(m);
        if (tid == 0) a.code_scale[t] = row::scale_of(m);
#pragma unroll
        for (int v = 0; v < V; ++v) {
          const int c = tid + v * step;
          if (c >= chunks) continue;
          row::u32x2_t q;
#pragma unroll
          for (int e = 0; e < 2; ++e)
            q[e] = row::pack_codes(code.bits(h[v][4 * e]), code.bits(h[v][4 * e + 1]), code.bits(h[v][4 * e + 2]),
                                   code.bits(h[v][4 * e + 3]));
          const row::Chunk<WHOLE> k(c, n);
          int8_t* const out = a.codes + t * a.ldc + k.at;
          if (!WHOLE && k.dup > 0) {
#pragma unroll
            for (int e = 0; e < 8; ++e)
              if (k.own(e)) out[e] = static_cast<int8_t>(q[e >> 2] >> (8 * (e & 3)));
          } else {
            row::store_as<WHOLE>(out, q);
          }
        }
      }
    }
    if (t + gridDim.x < a.tokens) __syncthreads();  // the reductions' words are used again
  }
}

// Rows of fewer than eight values or more than 32768: one work-group per row,
// every pass recomputes the row's values from memory (the row is in cache after
// the first).  Thread i owns the elements i, i + 256, ... in every pass, so h_out
// may be h.
constexpr int kAnyThreads = 256;
__global__ __launch_bounds__(kAnyThreads) void residual_norm_any_kernel(NormArgs a) {
  __shared__ float sh[4][16];
  __shared__ uint32_t sh_top[16];
  const int n = static_cast<int>(a.n);
  const float inv_n = 1.f / static_cast<float>(n);
  const int hb = a.h_type == SIGNROT_BF16, pb = a.param_type == SIGNROT_BF16;
  const int tid = threadIdx.x;

  for (int64_t t = blockIdx.x; t < a.tokens; t += gridDim.x) {
    const int64_t r = modulation_row(a, t);
    const int64_t gate_at = a.ldg ? r * a.ldg : 0, mod_at = a.ldm ? r * a.ldm : 0;
    const int64_t h_at = t * a.ldh, y_at = t * a.ldy;

    // mean and 1 / sqrt(var + eps) of the n values of f
    auto stats = [&](auto f, int kind, float eps, float* sh1, float* sh2, float& mean, float& inv) {
      mean = 0.f;
      inv = 1.f;
      if (kind == SIGNROT_NORM_NONE) return;
      if (kind == SIGNROT_NORM_LAYER) {
        float s = 0.f;
        for (int j = tid; j < n; j += kAnyThreads) s += f(j);
        mean = mean_of(row::block_reduce(s, sh1), n, inv_n);
      }
      float q = 0.f;
      for (int j = tid; j < n; j += kAnyThreads) {
        const float d = f(j) - mean;
        q = fmaf(d, d, q);
      }
      q = row::block_reduce(q, sh2);
      inv = 1.f / sqrtf(q * inv_n + eps);
      if (__builtin_expect(q == INFINITY, 0)) {
        __syncthreads();
        q = 0.f;
        for (int j = tid; j < n; j += kAnyThreads) {
          const float d = (f(j) - mean) * kSmall;
          q = fmaf(d, d, q);
        }
        inv = kSmall / sqrtf(row::block_reduce(q, sh2) * inv_n);
      }
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
      stats([&](int j) { return row::load_elem(a.y, y_at + j, 1); }, a.post_norm, a.eps_post, sh[0], sh[1], mean_y,
            inv_y);
    auto stream = [&](int j) {
      float v = a.beta * row::load_elem(a.h, h_at + j, hb);
      if (a.y) {
        float b = affine(row::load_elem(a.y, y_at + j, 1), a.post_norm, mean_y, inv_y, a.post_weight, a.post_bias, j);
        if (a.gate) b *= row::load_elem(a.gate, gate_at + j, pb);
        v = fmaf(a.alpha, b, v);
      }
      return v;
    };
    stats(stream, a.pre_norm, a.eps_pre, sh[2], sh[3], mean_h, inv_h);
    auto out = [&](float v, int j) {
      v = affine(v, a.pre_norm, mean_h, inv_h, a.pre_weight, a.pre_bias, j);
      if (a.mod_scale) v *= 1.f + row::load_elem(a.mod_scale, mod_at + j, pb);
      if (a.mod_shift) v += row::load_elem(a.mod_shift, mod_at + j, pb);
      return v;
    };
    float top = 0.f;
    if (a.codes) {
      uint32_t m = 0;
      for (int j = tid; j < n; j += kAnyThreads) m = row::join(m, row::abs_bits(out(stream(j), j)));
      top = __uint_as_float(row::block_reduce(m, sh_top));
      if (tid == 0) a.code_scale[t] = row::scale_of(top);
    }
    const row::Codes code(top);
    for (int j = tid; j < n; j += kAnyThreads) {
      const float v = stream(j);
      const float u = out(v, j);
      if (a.h_out) row::store_elem(a.h_out, t * a.ldho + j, v, hb);
      if (a.u) row::store_elem(a.u, t * a.ldu + j, u, 1);
      if (a.codes) a.codes[t * a.ldc + j] = static_cast<int8_t>(code.bits(u));
    }
    if (t + gridDim.x < a.tokens) __syncthreads();  // the reductions' words are used again
  }
}

// Every row of every tensor starts on a 16-byte boundary (8 for the codes)
// and n is a multiple of eight.
bool aligned_rows(const NormArgs& a) {
  const int64_t hs = a.h_type == SIGNROT_BF16 ? 2 : 4, ps = a.param_type == SIGNROT_BF16 ? 2 : 4;
  uintptr_t at = 0;
  for (const void* p : {a.h, a.y, static_cast<const void*>(a.h_out), static_cast<const void*>(a.u), a.post_weight,
                        a.post_bias, a.gate, a.pre_weight, a.pre_bias, a.mod_scale, a.mod_shift})
    at |= reinterpret_cast<uintptr_t>(p);
  int64_t ld = a.ldh * hs;
  if (a.y) ld |= a.ldy * 2;
  if (a.h_out) ld |= a.ldho * hs;
  if (a.u) ld |= a.ldu * 2;
  if (a.gate) ld |= a.ldg * ps;
  if (a.mod_scale || a.mod_shift) ld |= a.ldm * ps;
  const bool codes = !a.codes || ((reinterpret_cast<uintptr_t>(a.codes) | static_cast<uintptr_t>(a.ldc)) & 7u) == 0;
  return a.n % 8 == 0 && (at & 15u) == 0 && (ld & 15) == 0 && codes;
}

template <int V, bool WHOLE>
void run_rows_as(const NormArgs& a, dim3 grid, dim3 block, hipStream_t s) {
  if (a.h_type == SIGNROT_BF16)
    residual_norm_rows_kernel<V, true, WHOLE><<<grid, block, 0, s>>>(a);
  else
    residual_norm_rows_kernel<V, false, WHOLE><<<grid, block, 0, s>>>(a);
}

template <bool WHOLE>
void run_rows(const NormArgs& a, dim3 grid, hipStream_t s) {
  const int chunks = static_cast<int>((a.n + 7) / 8);
  int v = row::chunks_per_thread(chunks, a.tokens);
  // A CU holds 24 waves of the bf16 kernel with two chunks a thread and 16 of the one
  // with four, each of which does twice as much: where only the latter takes
  // all rows in one round (2048 x 4096: 15.7 us, 17.9 with two; 1024 x 8192 16.1 and
  // 19.1; 1237 x 5120 14.8 and 15.7; but 1024 x 5120, one round of either, 13.1 and
  // 12.1).  The binary32 kernel loses (1237 x 5120 with modulations 25.5 us with
  // four, 23.9 with two; RMS without 19.8 and 18.0).
  if (WHOLE && a.h_type == SIGNROT_BF16 && v == 2) {
    auto places = [&](int chunks_each, int waves) {
      return device_cu_count() * (waves / (row::threads_for(chunks, chunks_each) / 64));
    };
    if (a.tokens > places(2, 24) && a.tokens <= places(4, 16)) v = 4;
  }
  const dim3 block(static_cast<unsigned>(row::threads_for(chunks, v)));
  switch (v) {
    case 1: run_rows_as<1, WHOLE>(a, grid, block, s); break;
    case 2: run_rows_as<2, WHOLE>(a, grid, block, s); break;
    default: run_rows_as<4, WHOLE>(a, grid, block, s); break;
  }
}

}  // namespace

hipError_t launch_residual_norm(const NormArgs& a, hipStream_t s) {
  const dim3 grid(static_cast<unsigned>(a.tokens < row::kMaxBlocks ? a.tokens : row::kMaxBlocks));
  if (a.n < 8 || a.n > 4 * 8 * 1024)
    residual_norm_any_kernel<<<grid, dim3(kAnyThreads), 0, s>>>(a);
  else if (aligned_rows(a))
    run_rows<true>(a, grid, s);
  else
    run_rows<false>(a, grid, s);
  return hipGetLastError();
}

}  // namespace signrot
