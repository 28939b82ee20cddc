// The norm of each head of the queries and keys and their rotation by the
// token's position, in one pass:
//
//   v = Norm(x) over the head's channels (with weight and bias),
//   pair (a, b) of the first `rotary` channels, number p:
//     a' = a cos[pos][p] - b sin[pos][p],  b' = b cos[pos][p] + a sin[pos][p].
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdint.h>

#include <type_traits>

#include "internal.h"
#include "row_ops.h"

namespace signrot {
namespace {

using Args = signrot_qk_norm_rope_args;

constexpr int kWaves = 4;

// v of the two rows of sixteen (or the two halves of the wave) that pair up, the
// first in .x and the second in .y of both.
__device__ __forceinline__ uint2 both_rows(uint32_t v) {
  const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return make_uint2(r[0], r[1]);
}
__device__ __forceinline__ uint2 both_halves(uint32_t v) {
  const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  return make_uint2(r[0], r[1]);
}

// Sum over the G lanes of a head (a power of two), the same value in each.
template <int G>
__device__ __forceinline__ float head_sum(float v) {
  if (G > 1) v += row::dpp<0xB1>(v);   // quad_perm 1, 0, 3, 2
  if (G > 2) v += row::dpp<0x4E>(v);   // quad_perm 2, 3, 0, 1
  if (G > 4) v += row::dpp<0x141>(v);  // row_half_mirror
  if (G > 8) v += row::dpp<0x140>(v);  // row_mirror
  if (G > 16) {
    const uint2 r = both_rows(__float_as_uint(v));
    v = __uint_as_float(r.x) + __uint_as_float(r.y);
  }
  if (G > 32) {
    const uint2 r = both_halves(__float_as_uint(v));
    v = __uint_as_float(r.x) + __uint_as_float(r.y);
  }
  return v;
}

// The value of the lane G / 2 away in the head (exclusive or).
template <int G>
__device__ __forceinline__ uint32_t across(uint32_t v) {
  if (G == 2) return row::dpp<0xB1>(v);
  if (G == 4) return row::dpp<0x4E>(v);
  if (G == 8) return row::dpp<0x1B>(row::dpp<0x141>(v));  // 7, then 3
  if (G == 16) return row::dpp<0x128>(v);                 // row_ror:8
  const uint2 r = G == 32 ? both_rows(v) : both_halves(v);
  return (threadIdx.x & (G / 2)) ? r.x : r.y;
}

__device__ __forceinline__ int64_t place_of(const Args& a, int64_t t) {
  if (!a.positions) return t;
  const int64_t p = a.positions_64 ? static_cast<const int64_t*>(a.positions)[t]
                                   : static_cast<int64_t>(static_cast<const int32_t*>(a.positions)[t]);
  return p < 0 ? 0 : (p >= a.places ? a.places - 1 : p);
}

// 1 / sqrt(x): the hardware's estimate (1 ulp) and a Newton step, below 2^-100
// (where the estimate may not take its argument) the library's root.
__device__ __forceinline__ float inverse_root(float x) {
  if (x < 0x1p-100f) return 1.f / sqrtf(x);
  const float r = __builtin_amdgcn_rsqf(x);
  return fmaf(r, fmaf(-0.5f * x * r, r, 0.5f), r);  // NaN where x is not finite
}

// Squares of values around 2^64 and more pass binary32's range, those of values below
// 2^-63 lose bits or vanish.  A head whose mean square and eps are together not finite
// (r is NaN), or below 2^-100 (r over kMost), is normed again, its values scaled down or up:
// an eps of 2^-100 or more hides what squares below it lose.  A small head's values lie
// below 2^-45 and its mean below kMean, so that scaled up they stay below 2^80 and their
// sum of squares finite; where a mean is larger, such a small deviation can only be zero.
constexpr float kDown = 0x1p-80f, kUp = 0x1p100f;
constexpr float kMost = 0x1p50f, kMean = 0x1p-20f;

// Eight values as they lie in memory.
struct Raw {
  row::u32x4_t w[2];
};
template <bool BF16, bool WHOLE>
__device__ __forceinline__ Raw load_raw(const void* p, int64_t j) {
  Raw r = {};
  if (BF16) {
    r.w[0] = row::load_as<WHOLE, row::u32x4_t>(static_cast<const uint16_t*>(p) + j);
  } else {
    r.w[0] = row::load_as<WHOLE, row::u32x4_t>(static_cast<const float*>(p) + j);
    r.w[1] = row::load_as<WHOLE, row::u32x4_t>(static_cast<const float*>(p) + j + 4);
  }
  return r;
}
template <bool BF16>
__device__ __forceinline__ void widen(const Raw& r, float (&v)[8]) {
  if (BF16) {
    row::widen_bf16(r.w[0], v);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = __uint_as_float(r.w[e >> 2][e & 3]);
  }
}

// Where a channel's partner is: in the lane (interleaved pairs), in the lane G / 2
// away (halves of a head of 8 G channels, all of them rotated), or elsewhere in the
// head, reached through LDS: in whole chunks, or one by one.
enum Pairs { kOwn, kAcross, kChunks, kAnywhere };

// A lane holds eight channels of a head, G lanes a head, so that a wave takes
// 64 / G heads of a token at a time, read and written once.  A wave goes over its
// token's queries, every parts-th group of heads, then over the keys; the next
// group's loads are on their way while one is computed.  With weight w, bias b and
// angles of the token, channel j with partner p and the sign of p's part in the sine,
//   out_j = r (x_j - mean) w_j cos_j + r (x_p - mean) w_p sin_j + (b_j cos_j + b_p sin_j):
// the factors w_j cos_j, w_p sin_j and the last sum are formed once a token and kept
// for all its heads (8192 tokens of 64 + 8 heads of 128, bf16: 106 us with angles and
// weights read for each head, 77 so).
//
// Bound by memory where tokens are many: that shape now 61 us on inputs from HBM
// (5.0 TB/s), and in a loop over the same ones, which the caches hold in part, 52; with
// interleaved pairs 57; through LDS, half of the channels rotated, 52; 80 channels,
// where six of a head's sixteen lanes idle, 40; binary32 (4096 tokens of 64 heads) 55.
// That takes eight waves a SIMD, 64 registers (67: 58 us for the 52).
template <int G, bool BF16, bool WHOLE, int PAIRS>
__global__ __launch_bounds__(64 * kWaves) void qk_norm_rope_kernel(Args a, int parts, int stream) {
  __shared__ __attribute__((aligned(16))) float sh[PAIRS >= kChunks ? kWaves : 1][64 * 8];
  const int lane = threadIdx.x & 63, wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
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
  const int64_t angles = place_of(a, t) * a.ldt;
  float* const mine = &sh[PAIRS >= kChunks ? wid : 0][(lane / G) * 8 * G];

  // channel j's partner, itself where it is not rotated
  auto partner = [&](int j) { return j >= rotary ? j : PAIRS == kOwn ? j ^ 1 : j < half ? j + half : j - half; };

  auto side = [&](const void* src, int64_t ld, int64_t hs, void* dst, int64_t ldo, int64_t hso, int heads,
                  const void* weight, const void* bias, int gr) {
    const int groups = (heads + kHeads - 1) / kHeads;
    if (gr >= groups) return;
    const int bf16_out = a.out_type == SIGNROT_BF16, bf16_param = a.param_type == SIGNROT_BF16;
    const bool normed = a.norm != SIGNROT_NORM_NONE;
    src = static_cast<const uint8_t*>(src) + t * ld * (BF16 ? 2 : 4);
    dst = static_cast<uint8_t*>(dst) + t * ldo * (bf16_out ? 2 : 4);
    auto load = [&](int g) {
      const int h = g * kHeads + lane / G;
      Raw r = {};
      if (live && h < heads) r = load_raw<BF16, WHOLE>(src, h * hs + ch.at);
      return r;
    };
    Raw next = load(gr);
    // (ws and the sum of the biases negated: what a channel that is not rotated or has no bias
    // adds is then -0, which leaves a zero's sign)
    float wc[8], ws[8], sub[8];
    {
      // angles, weights and biases of the lane's channels and of their partners
      float cs[8], sn[8], w[8], wp[8], b[8], bp[8];
      const bool weighted = normed && weight, biased = normed && bias;
      if (PAIRS == kOwn) {
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const bool turn = live && ch.at + 2 * k < rotary;
          cs[2 * k] = cs[2 * k + 1] = turn ? a.cos[angles + ch.at / 2 + k] : 1.f;
          sn[2 * k] = sn[2 * k + 1] = turn ? a.sin[angles + ch.at / 2 + k] : 0.f;
        }
      } else if (PAIRS == kChunks && ch.at >= rotary) {
#pragma unroll
        for (int e = 0; e < 8; ++e) cs[e] = 1.f, sn[e] = 0.f;
      } else if (PAIRS == kAcross || PAIRS == kChunks) {
        const int64_t at = angles + (ch.at < half ? ch.at : ch.at - half);
        row::load8<false>(a.cos, at, 0, cs);
        row::load8<false>(a.sin, at, 0, sn);
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int j = ch.at + e;
          const bool turn = live && j < rotary;
          cs[e] = turn ? a.cos[angles + (j < half ? j : j - half)] : 1.f;
          sn[e] = turn ? a.sin[angles + (j < half ? j : j - half)] : 0.f;
        }
      }
      auto both = [&](const void* of, bool given, float none, float(&own)[8], float(&far)[8]) {
#pragma unroll
        for (int e = 0; e < 8; ++e) own[e] = far[e] = none;
        if (!given) return;
        row::load8<WHOLE>(of, ch.at, bf16_param, own);
        if (PAIRS == kAcross || PAIRS == kChunks) {
          row::load8<WHOLE>(of, partner(ch.at), bf16_param, far);
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e)
            far[e] = PAIRS == kOwn ? (ch.at + e < rotary ? own[e ^ 1] : own[e])
                                   : row::load_elem(of, partner(ch.at + e), bf16_param);
        }
      };
      both(weight, weighted, 1.f, w, wp);
      both(bias, biased, 0.f, b, bp);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (PAIRS == kOwn ? e & 1 : ch.at + e >= half) sn[e] = -sn[e];  // the second of a pair
        if (PAIRS != kAcross && ch.at + e >= rotary) {
          wp[e] = PAIRS == kOwn && !(e & 1) ? 0.f : -0.f;  // (times sn, +-0: +0)
          bp[e] = 0.f;
        }
        wc[e] = w[e] * cs[e];
        ws[e] = wp[e] * sn[e];
        sub[e] = biased ? fmaf(bp[e], sn[e], -(b[e] * cs[e])) : 0.f;
      }
    }
    for (; gr < groups; gr += parts) {
      const Raw raw = next;
      if (gr + parts < groups) next = load(gr + parts);
      const int h = gr * kHeads + lane / G;
      const bool on = live && h < heads;
      float v[8], o[8];
      widen<BF16>(raw, v);
      float mean = 0.f, r = 1.f, scale = 1.f;
      // A second time if a head is large or small, which is the same in all lanes of it.  (With
      // the first turn apart, as the compiler has it otherwise, half of the channels rotated
      // took 72.8 us, and 61.9 so.)
#pragma clang loop unroll(disable)
      for (bool again = false; normed; again = true) {
        if (a.norm == SIGNROT_NORM_LAYER) {
          float s = 0.f;
#pragma unroll
          for (int e = 0; e < 8; ++e) s += ch.own(e) ? v[e] : 0.f;
          s = head_sum<G>(s);
          const float q = s * inv_n;
          mean = fmaf(fmaf(-q, static_cast<float>(head), s), inv_n, q);
#pragma unroll
          for (int e = 0; e < 8; ++e) v[e] -= mean;
        }
        float ss = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (ch.own(e)) ss = fmaf(v[e], v[e], ss);
        ss = head_sum<G>(live ? ss : 0.f);
        r = inverse_root(fmaf(ss, inv_n, a.eps * scale * scale));
        if (again || __builtin_amdgcn_ballot_w64(!(r <= kMost)) == 0) break;
        scale = r <= kMost ? 1.f : r > kMost ? (fabsf(mean) < kMean ? kUp : 1.f) : kDown;
        widen<BF16>(load(gr), v);  // read again: raw does not have to stay
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] *= scale;
      }
      float other[8];
      if (PAIRS == kOwn) {
#pragma unroll
        for (int e = 0; e < 8; ++e) other[e] = v[e ^ 1];
      } else if (PAIRS == kAcross) {
        Raw far;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          far.w[0][i] = across<G>(raw.w[0][i]);
          if (!BF16) far.w[1][i] = across<G>(raw.w[1][i]);
        }
        widen<BF16>(far, other);
#pragma unroll
        for (int e = 0; e < 8; ++e) other[e] = fmaf(other[e], scale, -mean);
      } else {
        if (live) {
#pragma unroll
          for (int e = 0; e < 8; ++e) mine[ch.at + e] = v[e];
        }
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int e = 0; e < 8; ++e) other[e] = mine[PAIRS == kChunks ? partner(ch.at) + e : partner(ch.at + e)];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
      }
      if (PAIRS != kAcross && rotary < head) {
        // (a channel that is not rotated takes nothing of another one, not even of an infinity)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const int at = ch.at + (PAIRS == kChunks ? 0 : PAIRS == kOwn ? e & 6 : e);
          other[e] = at < rotary ? other[e] : 0.f;
        }
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] = fmaf(fmaf(other[e], -ws[e], v[e] * wc[e]), r, -sub[e]);
      if (!on) continue;
      const int64_t to = h * hso + ch.at;
      if (WHOLE || ch.dup == 0) {
        if (bf16_out) {
          row::store_chunk<WHOLE>(static_cast<uint16_t*>(dst) + to,
                             row::u32x4_t{row::pack_bf16(o[0], o[1]), row::pack_bf16(o[2], o[3]),
                                          row::pack_bf16(o[4], o[5]), row::pack_bf16(o[6], o[7])},
                             stream);
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
          if (ch.own(e)) row::store_elem(dst, to + e, o[e], bf16_out);
      }
    }
  };
  side(a.q, a.ldq, a.hsq, a.q_out, a.ldqo, a.hsqo, a.q_heads, a.q_weight, a.q_bias, part);
  // the keys' groups follow the queries': every parts-th of them all
  const int queries = (a.q_heads + kHeads - 1) / kHeads;
  if (a.k_heads > 0)
    side(a.k, a.ldk, a.hsk, a.k_out, a.ldko, a.hsko, a.k_heads, a.k_weight, a.k_bias,
         (part + parts - queries % parts) % parts);
}

template <int G>
void run(const Args& a, bool whole, hipStream_t s) {
  constexpr int kHeads = 64 / G;
  const int groups = (a.q_heads + kHeads - 1) / kHeads + (a.k_heads + kHeads - 1) / kHeads;
  // Fewer than 4096 tokens: several waves a token, up to one a group of heads, to have
  // waves for 1024 SIMDs (16 tokens 8.5 us, 13.7 with one; 1024 13.0 and 18.1; 2048 20.8
  // and 23.4).
  int parts = 1;
  while (parts < groups && a.tokens * parts < 4096) parts *= 2;
  if (parts > groups) parts = groups;
  const bool bf16 = a.in_type == SIGNROT_BF16;
  const int stream = row::past_caches(a.tokens * (a.q_heads + a.k_heads) * a.head, a.out_type == SIGNROT_BF16);
  const int pairs = a.interleaved || a.rotary == 0 ? kOwn
                    : whole && G > 1 && a.rotary == a.head && a.head == 8 * G ? kAcross
                    : whole && a.rotary % 16 == 0                             ? kChunks
                                                                              : kAnywhere;
  // A launch holds fewer than 2^32 threads.
  const int64_t most = (int64_t{1} << 25) / parts;
  for (int64_t t = 0; t < a.tokens; t += most) {
    Args b = a;
    b.tokens = a.tokens - t < most ? a.tokens - t : most;
    const int in = bf16 ? 2 : 4, out = a.out_type == SIGNROT_BF16 ? 2 : 4;
    b.q = static_cast<const uint8_t*>(a.q) + t * a.ldq * in;
    b.q_out = static_cast<uint8_t*>(a.q_out) + t * a.ldqo * out;
    if (a.k) b.k = static_cast<const uint8_t*>(a.k) + t * a.ldk * in;
    if (a.k) b.k_out = static_cast<uint8_t*>(a.k_out) + t * a.ldko * out;
    if (a.positions) {
      b.positions = static_cast<const uint8_t*>(a.positions) + t * (a.positions_64 ? 8 : 4);
    } else if (a.rotary > 0) {
      b.cos = a.cos + t * a.ldt;
      b.sin = a.sin + t * a.ldt;
    }
    const dim3 grid(static_cast<unsigned>((b.tokens * parts + kWaves - 1) / kWaves));
    const auto go = [&](auto kernel) { kernel<<<grid, 64 * kWaves, 0, s>>>(b, parts, stream); };
    const auto pick = [&](auto BF16) {
      constexpr bool kBf16 = decltype(BF16)::value;
      // (whole chunks in heads of one lane are the lane's own; of the sixteen channels of two
      // lanes none or all are rotated so)
      if constexpr (G > 1)
        if (pairs == kAcross) return go(qk_norm_rope_kernel<G, kBf16, true, kAcross>);
      if constexpr (G > 2)
        if (pairs == kChunks) return go(qk_norm_rope_kernel<G, kBf16, true, kChunks>);
      if (pairs == kOwn)
        whole ? go(qk_norm_rope_kernel<G, kBf16, true, kOwn>) : go(qk_norm_rope_kernel<G, kBf16, false, kOwn>);
      else
        whole ? go(qk_norm_rope_kernel<G, kBf16, true, kAnywhere>) : go(qk_norm_rope_kernel<G, kBf16, false, kAnywhere>);
    };
    bf16 ? pick(std::true_type{}) : pick(std::false_type{});
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
