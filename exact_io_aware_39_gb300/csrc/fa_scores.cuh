// Scores that are capped by a tanh or lowered with distance
// (flash_attn_scored.h): the host's reading of fa_scores and the arithmetic
// that the kernels share. In log2 units, with k = scale / softcap, c2 = softcap
// log2(e) and s the raw product Q . K,
//   t2 = c2 tanh(k s),  u2 = t2 - slope log2(e) |i - j|.
#pragma once

#include "flash_attn_scored.h"
#include "fa_ptx.cuh"

#include <cmath>
#include <cstddef>

namespace fa {

// What a packed kernel does to its scores: nothing; cap (and perhaps bias and
// prefix); bias or prefix without a cap; cap (and perhaps prefix) without a bias
// (the forward, whose registers the bias's code cost: 24 prompts of 16-2048 tokens, 32 / 8
// heads, d = 128, 171 us with it and 154 without).
constexpr int kScorePlain = 0, kScoreCap = 1, kScoreBias = 2, kScoreCapOnly = 3;
constexpr __host__ __device__ bool score_capped(int score) { return score == kScoreCap || score == kScoreCapOnly; }

struct ScoreParams {
  const float* slopes;       // [Hq] or null
  const int32_t* prefix;     // [B] or null
  float limit;               // |s| up to which the polynomial holds (kCapSmall / k), or -1: nowhere
  float a0, a1, a2, a3;      // there t2 = s (a0 + s^2 (a1 + s^2 (a2 + s^2 a3)))
  float b0, b1, b2, b3;      // and tanh(k s) the same with these, a / c2
  float k, e2, c2;           // k; 2 k log2(e): exp(2 k s) = 2^(e2 s); c2
  int cap;
  float head;                // how far above the first tile's largest score a row's reference starts (bf16, no bias)
};

// How far a row's reference may lie below its largest score, in log2 units, in the packed
// forward: P reaches 2^kRefMove there (fp16 ends at 2^16; in bf16 P, V and the number of
// keys share the 2^127 of an fp32 sum).
constexpr float kRefMove = 14.f;

// tanh(y) = y (C0 + C1 y^2 + C2 y^4 + C3 y^6) for |y| <= 0.4, to 9.8e-8 of the
// value: the polynomial of least relative error (Remez exchange, in 64 bits).
constexpr float kCapSmall = 0.4f;
constexpr float kTanh0 = 0.999999902f, kTanh1 = -0.333313625f, kTanh2 = 0.132709768f, kTanh3 = -0.0475536036f;

// Reads a caller's fa_scores (may be null). Returns FA_OK or the refusal.
inline fa_status read_scores(const fa_scores* scores, float scale, int causal, bool cached, ScoreParams* out) {
  *out = ScoreParams{};
  out->limit = -1.f;
  if (scores == nullptr) return FA_OK;
  fa_scores s{};
  if (scores->size < offsetof(fa_scores, softcap) + sizeof(float)) return FA_ERR_INVALID_ARG;
  s.softcap = scores->softcap;
  if (scores->size >= offsetof(fa_scores, slopes) + sizeof(void*)) s.slopes = scores->slopes;
  if (scores->size >= offsetof(fa_scores, prefix_lens) + sizeof(void*)) s.prefix_lens = scores->prefix_lens;
  if (!std::isfinite(s.softcap) || s.softcap < 0.f) return FA_ERR_INVALID_ARG;
  if ((reinterpret_cast<uintptr_t>(s.slopes) | reinterpret_cast<uintptr_t>(s.prefix_lens)) & 3) return FA_ERR_INVALID_ARG;
  if (s.prefix_lens != nullptr && cached) return FA_ERR_UNSUPPORTED;
  if (s.prefix_lens != nullptr && !causal) return FA_ERR_INVALID_ARG;
  out->slopes = s.slopes;
  out->prefix = s.prefix_lens;
  if (s.softcap == 0.f) return FA_OK;
  if (s.softcap < 0x1p-10f || s.softcap > 0x1p10f) return FA_ERR_UNSUPPORTED;
  const double k = (double)scale / s.softcap, c2 = s.softcap * 1.4426950408889634;
  if (k > 0x1p60 || k < 0x1p-60) return FA_ERR_UNSUPPORTED;   // (its square stays an fp32 number)
  out->cap = 1;
  out->k = (float)k;
  out->e2 = (float)(2. * 1.4426950408889634 * k);
  out->c2 = (float)c2;
  // (by how much more than the threshold a score can pass the first tile's largest, 2 c2 at
  // most; whole, and at most 16, whose rounding in the arguments is within the cap's 2^-20)
  const double head = std::floor(2. * c2 - kRefMove);
  out->head = head < 0. ? 0.f : head > 16. ? 16.f : (float)head;
  // (past these k, k^7 leaves the fp32 range)
  if (k < 0x1p15 && k > 0x1p-15) {
    out->limit = (float)(kCapSmall / k);
    out->a0 = (float)(c2 * k * kTanh0);
    out->a1 = (float)(c2 * k * k * k * kTanh1);
    out->a2 = (float)(c2 * k * k * k * k * k * kTanh2);
    out->a3 = (float)(c2 * k * k * k * k * k * k * k * kTanh3);
    out->b0 = (float)(k * kTanh0);
    out->b1 = (float)(k * k * k * kTanh1);
    out->b2 = (float)(k * k * k * k * k * kTanh2);
    out->b3 = (float)(k * k * k * k * k * k * k * kTanh3);
  }
  return FA_OK;
}

#ifdef __CUDACC__
__device__ __forceinline__ float rcp_approx(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// tanh(k s) = 1 - 2 / (1 + exp(2 k s)), to about 2^-22 absolutely (one
// exponential and a reciprocal of 2^-22 each); exp = inf and 0 give 1 and -1.
__device__ __forceinline__ float tanh_exp(float s, const ScoreParams& p) {
  return fmaf(-2.f, rcp_approx(1.f + ex2(s * p.e2)), 1.f);
}
// the same for a pair of one row, whose denominators share a reciprocal: 1 / a =
// b / (a b). The exponents are held to 60, where tanh is 1 in fp32, so that a b is
// finite (a NaN stays one, and makes its neighbour one, in a row that has a NaN then
// in any case).
__device__ __forceinline__ float min_nan(float a, float b) {
  float y;
  asm("min.NaN.f32 %0, %1, %2;" : "=f"(y) : "f"(a), "f"(b));
  return y;
}
__device__ __forceinline__ float2 tanh_exp2(float2 s, const ScoreParams& p) {
  const float2 a = make_float2(ex2(min_nan(s.x * p.e2, 60.f)), ex2(min_nan(s.y * p.e2, 60.f)));
  const float2 b = __fadd2_rn(a, make_float2(1.f, 1.f));
  const float r = -2.f * rcp_approx(b.x * b.y);
  return make_float2(fmaf(r, b.y, 1.f), fmaf(r, b.x, 1.f));
}
// tanh(k s) and its slope 1 - tanh^2 of a pair that belongs to two rows: with e =
// exp(2 k s) and q = 1 / (1 + e), tanh is 1 - 2 q and the slope 4 e q^2, which keeps its
// relative precision (2^-21, and 2^-23 of the exponent's argument) where 1 - tanh^2
// would be nothing but tanh's rounding. Exponents are held to 62, scores of 21 caps,
// where the slope is 2^-60 and the reciprocal of a pair's 2^124 still a normal number. A
// NaN counts as 62 here: it stays out of its neighbour.
__device__ __forceinline__ float2 tanh_slope2(float2 s, const ScoreParams& p, float2& slope) {
  const float2 e = make_float2(ex2(fminf(s.x * p.e2, 62.f)), ex2(fminf(s.y * p.e2, 62.f)));
  const float2 b = __fadd2_rn(e, make_float2(1.f, 1.f));
  const float r = 2.f * rcp_approx(b.x * b.y);
  const float2 q2 = __fmul2_rn(make_float2(b.y, b.x), make_float2(r, r));
  slope = __fmul2_rn(__fmul2_rn(e, q2), q2);
  return __fadd2_rn(make_float2(1.f, 1.f), make_float2(-q2.x, -q2.y));
}
// t2 = s times this, of a pair of small scores (|s| <= limit)
__device__ __forceinline__ float2 cap_small_factor2(float2 s, const ScoreParams& p) {
  const float2 z = __fmul2_rn(s, s);
  float2 r = __ffma2_rn(z, make_float2(p.a3, p.a3), make_float2(p.a2, p.a2));
  r = __ffma2_rn(z, r, make_float2(p.a1, p.a1));
  return __ffma2_rn(z, r, make_float2(p.a0, p.a0));
}
// tanh(k s) of a pair of small scores
__device__ __forceinline__ float2 tanh_small2(float2 s, const ScoreParams& p) {
  const float2 z = __fmul2_rn(s, s);
  float2 r = __ffma2_rn(z, make_float2(p.b3, p.b3), make_float2(p.b2, p.b2));
  r = __ffma2_rn(z, r, make_float2(p.b1, p.b1));
  return __fmul2_rn(s, __ffma2_rn(z, r, make_float2(p.b0, p.b0)));
}
// t2 of one score of any size: the polynomial where it holds
__device__ __forceinline__ float cap_any(float s, const ScoreParams& p) {
  const float z = s * s;
  const float small = s * fmaf(z, fmaf(z, fmaf(z, p.a3, p.a2), p.a1), p.a0);
  return fabsf(s) <= p.limit ? small : p.c2 * tanh_exp(s, p);
}
#endif

}  // namespace fa
