// The norm of each head of the queries and keys and their rotation by the
// token's position, in one pass:
//
//   v = Norm(x) over the head's channels (with weight and bias),
//   pair (a, b) of the first `rotary` channels, number p:
//     a' = a cos[pos][p] - b sin[pos][p],  b' = b cos[pos][p] + a sin[pos][p].
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include "internal.h"
#include "row_ops.h"

namespace signrot {
namespace {

using Args = signrot_qk_norm_rope_args;

constexpr int kWaves = 4;

// Sum over the G lanes of a head (a power of two), the same value in each.
template <int G>
__device__ __forceinline__ float head_sum(float v) {
  if (G > 1) v += row::dpp<0xB1>(v);   // quad_perm 1, 0, 3, 2
  if (G > 2) v += row::dpp<0x4E>(v);   // quad_perm 2, 3, 0, 1
  if (G > 4) v += row::dpp<0x141>(v);  // row_half_mirror
  if (G > 8) v += row::dpp<0x140>(v);  // row_mirror
  if (G > 16) v += __shfl_xor(v, 16);
  if (G > 32) v += __shfl_xor(v, 32);
  return v;
}

__device__ __forceinline__ int64_t place_of(const Args& a, int64_t t) {
  if (!a.positions) return t;
  const int64_t p = a.positions_64 ? static_cast<const int64_t*>(a.positions)[t]
                                   : static_cast<int64_t>(static_cast<const int32_t*>(a.positions)[t]);
  return p < 0 ? 0 : (p >= a.places ? a.places - 1 : p);
}

// Squares of values around 2^64 and more pass binary32's range; such a head is
// summed again, scaled by this (eps is then below a rounding of the mean).
constexpr float kSmall = 0x1p-80f;

// A lane holds eight channels of a head, G lanes a head, so that a wave takes
// 64 / G heads of a token at a time, read and written once.  The channels'
// partners come from the lane itself (interleaved pairs) or through 2 KiB of
// LDS (halves).  A wave keeps its token's angles and goes over the token's
// heads, every parts-th group of them.
template <int G, bool WHOLE>
__global__ __launch_bounds__(64 * kWaves) void qk_norm_rope_kernel(Args a, int parts) {
  __shared__ float sh[kWaves][64 * 8];
  const int lane = threadIdx.x & 63, wid = threadIdx.x >> 6;
  const int64_t item = static_cast<int64_t>(blockIdx.x) * kWaves + wid;
  const int64_t t = item / parts;
  const int part = static_cast<int>(item - t * parts);
  if (t >= a.tokens) return;
  constexpr int kHeads = 64 / G;
  const int head = static_cast<int>(a.head), rotary = static_cast<int>(a.rotary), half = rotary / 2;
  const int c = lane % G;
  const bool live = 8 * c < head;
  const row::Chunk<WHOLE> ch(live ? c : 0, head);
  const float inv_n = 1.f / static_cast<float>(head);

  // the angles of the lane's channels: number p(e)
  float cs[8], sn[8];
  {
    const int64_t at = place_of(a, t) * a.ldt;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int j = ch.at + e;
      const int p = a.interleaved ? j >> 1 : (j < half ? j : j - half);
      const bool turn = live && j < rotary;
      cs[e] = turn ? a.cos[at + p] : 1.f;
      sn[e] = turn ? a.sin[at + p] : 0.f;
      if (a.interleaved ? !(j & 1) : j < half) sn[e] = -sn[e];  // the first of a pair
    }
  }
  const int heads = a.q_heads + a.k_heads;
  const int groups = (heads + kHeads - 1) / kHeads;
  for (int gr = part; gr < groups; gr += parts) {
    const int h0 = gr * kHeads + lane / G;
    const bool on = live && h0 < heads;
    const bool key = h0 >= a.q_heads;
    const int h = key ? h0 - a.q_heads : h0;
    float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    if (on) {
      const void* const src = key ? a.k : a.q;
      row::load8<WHOLE>(src, t * (key ? a.ldk : a.ldq) + h * (key ? a.hsk : a.hsq) + ch.at, a.in_type == SIGNROT_BF16, v);
    }
    if (a.norm != SIGNROT_NORM_NONE) {
      float m[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) m[e] = ch.own(e) ? 1.f : 0.f;
      float mean = 0.f;
      if (a.norm == SIGNROT_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) s += ch.own(e) ? v[e] : 0.f;
        s = head_sum<G>(s);
        const float q = s * inv_n;
        mean = fmaf(fmaf(-q, static_cast<float>(head), s), inv_n, q);
      }
      float ss = 0.f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[e] = on ? v[e] - mean : 0.f;
        if (ch.own(e)) ss = fmaf(v[e], v[e], ss);
      }
      ss = head_sum<G>(ss);
      float r = 1.f / sqrtf(fmaf(ss, inv_n, a.eps));
      if (!(ss < INFINITY)) {  // the same in all lanes of a head
        float sm = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (ch.own(e)) sm = fmaf(v[e] * kSmall, v[e] * kSmall, sm);
        sm = head_sum<G>(sm);
        r = kSmall / sqrtf(fmaf(sm, inv_n, a.eps * kSmall * kSmall));
      }
      const void* const w = key ? a.k_weight : a.q_weight;
      const void* const b = key ? a.k_bias : a.q_bias;
      float f[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= r;
      if (w && on) {
        row::load8<WHOLE>(w, ch.at, a.param_type == SIGNROT_BF16, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= f[e];
      }
      if (b && on) {
        row::load8<WHOLE>(b, ch.at, a.param_type == SIGNROT_BF16, f);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] += f[e];
      }
    }
    float o[8];
    if (a.interleaved) {
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(v[e ^ 1], sn[e], v[e] * cs[e]);
    } else {
      float* const mine = &sh[wid][(lane / G) * 8 * G];
      if (live) {
#pragma unroll
        for (int e = 0; e < 8; ++e) mine[ch.at + e] = v[e];
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int j = ch.at + e;
        const float other = j < rotary ? mine[j < half ? j + half : j - half] : 0.f;
        o[e] = fmaf(other, sn[e], v[e] * cs[e]);
      }
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
    }
    if (!on) continue;
    const bool bf16 = a.out_type == SIGNROT_BF16;
    void* const dst = key ? a.k_out : a.q_out;
    const int64_t to = t * (key ? a.ldko : a.ldqo) + h * (key ? a.hsko : a.hsqo) + ch.at;
    if (WHOLE || ch.dup == 0) {
      if (bf16) {
        row::store_as<WHOLE>(static_cast<uint16_t*>(dst) + to,
                             row::u32x4_t{row::pack_bf16(o[0], o[1]), row::pack_bf16(o[2], o[3]),
                                          row::pack_bf16(o[4], o[5]), row::pack_bf16(o[6], o[7])});
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q)
          row::store_as<WHOLE>(static_cast<float*>(dst) + to + 4 * q,
                               row::u32x4_t{__float_as_uint(o[4 * q]), __float_as_uint(o[4 * q + 1]),
                                            __float_as_uint(o[4 * q + 2]), __float_as_uint(o[4 * q + 3])});
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (ch.own(e)) row::store_elem(dst, to + e, o[e], bf16);
    }
  }
}

template <int G>
void run(const Args& a, bool whole, hipStream_t s) {
  const int groups = (a.q_heads + a.k_heads + 64 / G - 1) / (64 / G);
  int parts = 1;
  while (parts < groups && a.tokens * parts < 4096) parts *= 2;
  if (parts > groups) parts = groups;
  // a launch holds fewer than 2^32 threads
  const int64_t most = (int64_t{1} << 25) / parts;
  for (int64_t t = 0; t < a.tokens; t += most) {
    Args b = a;
    b.tokens = a.tokens - t < most ? a.tokens - t : most;
    const int in = a.in_type == SIGNROT_BF16 ? 2 : 4, out = a.out_type == SIGNROT_BF16 ? 2 : 4;
    b.q = static_cast<const uint8_t*>(a.q) + t * a.ldq * in;
    b.q_out = static_cast<uint8_t*>(a.q_out) + t * a.ldqo * out;
    if (a.k) b.k = static_cast<const uint8_t*>(a.k) + t * a.ldk * in;
    if (a.k) b.k_out = static_cast<uint8_t*>(a.k_out) + t * a.ldko * out;
    if (a.positions) {
      b.positions = static_cast<const uint8_t*>(a.positions) + t * (a.positions_64 ? 8 : 4);
    } else {
      b.cos = a.cos + t * a.ldt;
      b.sin = a.sin + t * a.ldt;
    }
    const dim3 grid(static_cast<unsigned>((b.tokens * parts + kWaves - 1) / kWaves));
    if (whole)
      qk_norm_rope_kernel<G, true><<<grid, 64 * kWaves, 0, s>>>(b, parts);
    else
      qk_norm_rope_kernel<G, false><<<grid, 64 * kWaves, 0, s>>>(b, parts);
  }
}

}  // namespace

hipError_t launch_qk_norm_rope(const Args& a, hipStream_t s) {
  auto fits = [](const void* p, int64_t stride, int64_t stride2, int size) {
    return (reinterpret_cast<uintptr_t>(p) & 15u) == 0 && (stride * size) % 16 == 0 && (stride2 * size) % 16 == 0;
  };
  const int in = a.in_type == SIGNROT_BF16 ? 2 : 4, out = a.out_type == SIGNROT_BF16 ? 2 : 4;
  const int param = a.param_type == SIGNROT_BF16 ? 2 : 4;
  const bool whole = a.head % 8 == 0 && fits(a.q, a.ldq, a.hsq, in) && fits(a.q_out, a.ldqo, a.hsqo, out) &&
                     (!a.k || (fits(a.k, a.ldk, a.hsk, in) && fits(a.k_out, a.ldko, a.hsko, out))) &&
                     fits(a.q_weight, 0, 0, param) && fits(a.k_weight, 0, 0, param) && fits(a.q_bias, 0, 0, param) &&
                     fits(a.k_bias, 0, 0, param);
  const int chunks = static_cast<int>((a.head + 7) / 8);
  if (chunks <= 1) run<1>(a, whole, s);
  else if (chunks <= 2) run<2>(a, whole, s);
  else if (chunks <= 4) run<4>(a, whole, s);
  else if (chunks <= 8) run<8>(a, whole, s);
  else if (chunks <= 16) run<16>(a, whole, s);
  else if (chunks <= 32) run<32>(a, whole, s);
  else run<64>(a, whole, s);
  return hipGetLastError();
}

}  // namespace signrot
