// What the packed kernels whose threads are query rows share: their work items
// and the scores of a row.
#pragma once

#include "fa_packed.cuh"

namespace fa {

namespace {

constexpr int kFwdThreads = 384;
constexpr int kSoftmaxRegs = 216;   // 2 x 128 x 216 + 128 x 72 = 384 x 168 registers
constexpr int kRowOtherRegs = 72;

// An item as the roles see it: its two query tiles, and the key tiles 0 .. n - 1
// live for either. SPLIT: one query tile, whose even key tiles are the first
// softmax group's and whose odd ones the second's.
// With scores of their own (PRE), every query sees the first `pre` keys.
template <bool SPLIT, bool PRE>
struct Pair {
  int start, len, c, head;      // c < 0: no item
  int nT, n;
  int pre, pre_last;            // PRE: the prefix, and its last key tile (-1: none)
  bool pair_heads, causal;
  // c: as the ring has it
  __device__ __forceinline__ void finish(bool pair_of_heads, bool is_causal) {
    pair_heads = pair_of_heads;
    causal = is_causal;
    nT = (len + kTile - 1) / kTile;
    pre = 0;
    pre_last = -1;
    if constexpr (PRE)
      if (c >= 0) {
        pre = prefix_of(c);
        pre_last = (pre + kTile - 1) / kTile - 1;
        c = tile_of(c);
      }
    if constexpr (SPLIT) n = causal ? max(c, pre_last) + 1 : nT;
    else n = causal ? last(has(1) ? 1 : 0) + 1 : nT;
  }
  __device__ __forceinline__ bool has(int t) const {
    if constexpr (SPLIT) return t < n;
    return t == 0 || pair_heads || 2 * c + 1 < nT;
  }
  __device__ __forceinline__ int qi(int t) const { return SPLIT || pair_heads ? c : 2 * c + t; }
  __device__ __forceinline__ int hq(int t) const { return SPLIT ? head : pair_heads ? 2 * head + t : head; }
  // first and last key tile of t, which has every one (SPLIT: every second) between them
  __device__ __forceinline__ int first(int t) const { return SPLIT ? t : 0; }
  __device__ __forceinline__ int last(int t) const {
    if constexpr (SPLIT) return n - 1 - ((n - 1 - t) & 1);
    if constexpr (PRE) return causal ? max(qi(t), pre_last) : nT - 1;
    return causal ? qi(t) : nT - 1;
  }
  __device__ __forceinline__ bool partial(int e, int q) const {
    if constexpr (PRE) return (causal && e >= q && (e + 1) * kTile > pre) || (e + 1) * kTile > len;
    return (causal && e == q) || (e + 1) * kTile > len;
  }
  // valid rows of the last key tile when it is not full, else 0
  __device__ __forceinline__ int tail() const { return len & (kTile - 1); }
};

// Brings a row of scores (raw products of query `row` with the keys from `key0`
// on) to log2 units, capped and lowered with the distance; key0 - row = far.
// side: -1 where all of these keys lie before the query's tile, 1 behind it, 0 in
// it. masked: columns from `lim` on are no keys of the row (what lies there may
// be NaN, which must not meet its neighbour).
template <int SCORE>
__device__ __forceinline__ void score_row(float (&x)[128], const ScoreParams& sp, float sl2, float slope2, float far,
                                          int side, bool masked, int lim) {
  if constexpr (SCORE == kScoreCap) {
    if (masked)
#pragma unroll
      for (int i = 0; i < 128; ++i)
        if (i >= lim) x[i] = 0.f;
    float top[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) top[k] = fmaxf(fabsf(x[k]), fabsf(x[4 + k]));
#pragma unroll
    for (int i = 8; i < 128; i += 8)
#pragma unroll
      for (int k = 0; k < 4; ++k) top[k] = fmax3(top[k], fabsf(x[i + k]), fabsf(x[i + 4 + k]));
    const float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
    if (__all_sync(0xFFFFFFFFu, most <= sp.limit)) {
#pragma unroll
      for (int i = 0; i < 128; i += 2) {
        const float2 t = cap_small2(make_float2(x[i], x[i + 1]), sp);
        x[i] = t.x;
        x[i + 1] = t.y;
      }
    } else {
#pragma unroll
      for (int i = 0; i < 128; i += 2) {
        const float2 t = tanh_exp2(make_float2(x[i], x[i + 1]), sp);
        x[i] = t.x * sp.c2;
        x[i + 1] = t.y * sp.c2;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < 128; i += 2) {
      const float2 t = __fmul2_rn(make_float2(x[i], x[i + 1]), make_float2(sl2, sl2));
      x[i] = t.x;
      x[i + 1] = t.y;
    }
  }
  if (sp.slopes != nullptr) {
    // the distances count up beside the scores (as constants they would take a
    // register each)
    float2 d[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) d[k] = make_float2(far + (float)(2 * k), far + (float)(2 * k + 1));
    const float2 step = make_float2(8.f, 8.f);
    if (side == 0) {
#pragma unroll
      for (int i = 0; i < 128; i += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          x[i + 2 * k] = fmaf(-slope2, fabsf(d[k].x), x[i + 2 * k]);
          x[i + 2 * k + 1] = fmaf(-slope2, fabsf(d[k].y), x[i + 2 * k + 1]);
          d[k] = __fadd2_rn(d[k], step);
        }
    } else {
      const float sl = side < 0 ? slope2 : -slope2;
#pragma unroll
      for (int i = 0; i < 128; i += 8)
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 t = __ffma2_rn(make_float2(sl, sl), d[k], make_float2(x[i + 2 * k], x[i + 2 * k + 1]));
          x[i + 2 * k] = t.x;
          x[i + 2 * k + 1] = t.y;
          d[k] = __fadd2_rn(d[k], step);
        }
    }
  }
}

}  // namespace

}  // namespace fa
