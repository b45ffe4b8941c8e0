// What the packed kernels whose threads are query rows share: their work items
// and the scores of a row.
#pragma once

#include "fa_packed.cuh"

namespace fa {

namespace {

constexpr int kFwdThreads = 384;
constexpr int kSoftmaxRegs = 216;   // 2 x 128 x 216 + 128 x 72 = 384 x 168 registers
constexpr int kRowOtherRegs = 72;
// with two warpgroups to a row: 4 x 128 x 104 + 128 x 64 = 640 x 96 registers
constexpr int kHalfThreads = 640, kHalfRegs = 104, kHalfOtherRegs = 64;

// An item as the roles see it: its two query tiles, and the key tiles 0 .. n - 1
// live for either. SPLIT: one query tile, whose even key tiles are the first
// softmax group's and whose odd ones the second's.
// With scores of their own (PRE), every query sees the first `pre` keys.
template <bool SPLIT, bool PRE>
struct Pair {
  int start, len, c, head;      // c < 0: no item
  int nT, n;
  int pre, pre_last;            // PRE: the prefix, and its last key tile (-1: none)
  int own;                      // PRE: the first query tile where entries go outward from it, else -1
  bool pair_heads, causal;
  // c: as the ring has it
  __device__ __forceinline__ void finish(bool pair_of_heads, bool is_causal, bool outward = false) {
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
    own = PRE && outward && c >= 0 ? qi(0) : -1;
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
  // The key tile of the forward's entry e: the tiles in order, or (with slopes) the
  // first query tile's own, those before it down to the first, those behind it, so that
  // a bias that falls with distance falls from entry to entry and a row's reference
  // stays. (11 prompts of 64-4096 tokens, 16 heads, d = 64, slopes 0.7 to 0.004: 145 us
  // in the tiles' order, 126 so; with prefixes 181 and 169.)
  __device__ __forceinline__ int tile(int e) const { return PRE && e <= own ? own - e : e; }
  __device__ __forceinline__ bool partial(int e, int q) const {
    if constexpr (PRE) return (causal && e >= q && (e + 1) * kTile > pre) || (e + 1) * kTile > len;
    return (causal && e == q) || (e + 1) * kTile > len;
  }
  // valid rows of the last key tile when it is not full, else 0
  __device__ __forceinline__ int tail() const { return len & (kTile - 1); }
};

// Scores of their own, of one row against half of a tile's keys: 64 columns in
// registers of one thread.
//
// (A thread for a whole row, as for plain scores, took 440 us for two sequences of
// 4547 and 5127 tokens, 32 / 8 heads, d = 128, with a cap: seven more operations a
// score in two warps of an SM's quarter. Two threads to a row 411, 64 KB of code
// less than 93; P in columns of its own, so that the next S is computed meanwhile, no
// maximum where the raw scores bound it, and a kernel without the bias 332; plain scores
// take 242. Weights against a reference of 0, which need no bound and no agreement of a
// row's two threads, took 320, but rounded the heaviest weight and ended at 2^30.)
//
// What is uniform for a row and a tile: the bias of key j is +-slope (j - i) where
// all keys lie on one side (linear), counted up beside the scores; else, in the
// query's own tile, -slope |j - i|. far = first key - query.
struct ScoreTile {
  float slope, far;          // slope: signed, in log2 units
  bool bias, linear, partial;
  bool live;                 // a row of the sequence
  int lim;                   // columns from here on are no keys of the row (partial)
};

template <int SCORE>
__device__ __forceinline__ ScoreTile score_tile(const ScoreParams& sp, float slope2, int key0, int row, int side,
                                                bool both_sides, bool partial, int lim, bool live) {
  ScoreTile s;
  s.bias = sp.slopes != nullptr;
  s.linear = !both_sides;
  s.slope = side > 0 ? -slope2 : slope2;
  s.far = (float)(key0 - row);
  s.partial = partial;
  s.lim = lim;
  s.live = live;
  return s;
}

// The largest bias of a row's keys in the tile from key0 on (about: masked keys
// count); -inf without a bias.
__device__ __forceinline__ float score_base(const ScoreParams& sp, float slope2, int key0, int row, int side) {
  if (sp.slopes == nullptr) return -INFINITY;
  const int first = key0 - row, last = first + kTile - 1;
  const int nearest = side < 0 ? -last : side > 0 ? first : 0, farthest = side < 0 ? -first : side > 0 ? last : kTile - 1;
  return -slope2 * (float)(slope2 >= 0.f ? nearest : farthest);
}

// The bias of columns c, c + 1, ... + 31 (and nref) by step: four chains of four
// steps, each rounded once.
struct BiasSteps {
  float2 d[4], step;
  __device__ __forceinline__ BiasSteps(const ScoreTile& s, int c, float nref) {
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float j = s.far + (float)(c + 2 * k);
      d[k] = make_float2(fmaf(s.slope, j, nref), fmaf(s.slope, j + 1.f, nref));
    }
    step = make_float2(8.f * s.slope, 8.f * s.slope);
  }
  __device__ __forceinline__ float2 next(int k) {
    const float2 b = d[k];
    d[k] = __fadd2_rn(d[k], step);
    return b;
  }
};

__device__ __forceinline__ float2 pair_of(const uint32_t (&u)[32], int i) {
  return make_float2(__uint_as_float(u[i]), __uint_as_float(u[i + 1]));
}
__device__ __forceinline__ void put_pair(uint32_t (&u)[32], int i, float2 x) {
  u[i] = __float_as_uint(x.x);
  u[i + 1] = __float_as_uint(x.y);
}
__device__ __forceinline__ void mask_columns(uint32_t (&u)[32], int lim, float with) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if (i >= lim) u[i] = __float_as_uint(with);
}

__device__ __forceinline__ float row_max(const uint32_t (&u)[2][32]) {
  float hi[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) hi[k] = -INFINITY;
#pragma unroll
  for (int i = 0; i < 64; i += 2)
    hi[(i >> 1) & 3] = fmax3(hi[(i >> 1) & 3], __uint_as_float(u[i >> 5][i & 31]), __uint_as_float(u[i >> 5][(i & 31) + 1]));
  return fmaxf(fmaxf(hi[0], hi[1]), fmaxf(hi[2], hi[3]));
}

// A cap's first step on a row's 64 raw scores: whether all of them, of all rows of
// the warp, are within the polynomial's limit; `most`, the row's largest magnitude. Rows past the sequence (not `live`)
// have no say: a sequence's bits are its own. What lies in masked columns may be
// NaN, which must not meet its neighbour in tanh_exp2: it becomes zeros.
__device__ __forceinline__ bool cap_vote(uint32_t (&u)[2][32], const ScoreParams& sp, bool partial, int lim, bool live,
                                         float& most) {
  if (partial) {
    mask_columns(u[0], lim, 0.f);
    mask_columns(u[1], lim - 32, 0.f);
  }
  float top[4];
#pragma unroll
  for (int k = 0; k < 4; ++k) top[k] = 0.f;
#pragma unroll
  for (int i = 0; i < 64; i += 2)
    top[(i >> 1) & 3] = fmax3(top[(i >> 1) & 3], fabsf(__uint_as_float(u[i >> 5][i & 31])),
                              fabsf(__uint_as_float(u[i >> 5][(i & 31) + 1])));
  most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
  return __all_sync(0xFFFFFFFFu, !live || most <= sp.limit);
}

// The cap of 32 scores, and nref; -inf where masked (partial: from column lim on).
__device__ __forceinline__ void cap_args(uint32_t (&u)[32], const ScoreParams& sp, bool partial, int lim, bool small,
                                         float nref) {
  const float2 n2 = make_float2(nref, nref);
  if (small) {
#pragma unroll
    for (int i = 0; i < 32; i += 2) {
      const float2 x = pair_of(u, i);
      put_pair(u, i, __ffma2_rn(x, cap_small_factor2(x, sp), n2));
    }
  } else {
#pragma unroll
    for (int i = 0; i < 32; i += 2) put_pair(u, i, __ffma2_rn(tanh_exp2(pair_of(u, i), sp), make_float2(sp.c2, sp.c2), n2));
  }
  if (partial) mask_columns(u, lim, -INFINITY);
}

// Adds the bias to 64 scores: raw ones (to which sl2 and nref go as well), or capped
// ones, which are complete but for it.
template <int SCORE>
__device__ __forceinline__ void bias_args(uint32_t (&u)[2][32], float sl2, const ScoreTile& s, float nref) {
  const float mul = score_capped(SCORE) ? 1.f : sl2, start = score_capped(SCORE) ? 0.f : nref;
#pragma unroll
  for (int hh = 0; hh < 2; ++hh) {
    if (s.linear) {
      BiasSteps b(s, 32 * hh, start);
#pragma unroll
      for (int i = 0; i < 32; i += 2)
        put_pair(u[hh], i, __ffma2_rn(pair_of(u[hh], i), make_float2(mul, mul), b.next((i >> 1) & 3)));
    } else {
#pragma unroll
      for (int i = 0; i < 32; i += 2) {
        const float d = s.far + (float)(32 * hh + i);
        const float2 x = __ffma2_rn(pair_of(u[hh], i), make_float2(mul, mul), make_float2(start, start));
        put_pair(u[hh], i, make_float2(fmaf(-s.slope, fabsf(d), x.x), fmaf(-s.slope, fabsf(d + 1.f), x.y)));
      }
    }
  }
}

// The arguments of the exponential, u2 + nref in log2 units, from a row's 64 raw
// scores; -inf where masked. Returns their maximum (MAX).
template <int SCORE, bool MAX>
__device__ __forceinline__ float score_args(uint32_t (&u)[2][32], const ScoreParams& sp, float sl2, const ScoreTile& s,
                                            float nref) {
  if constexpr (score_capped(SCORE)) {
    float most;
    const bool small = cap_vote(u, sp, s.partial, s.lim, s.live, most);
    cap_args(u[0], sp, s.partial, s.lim, small, nref);
    cap_args(u[1], sp, s.partial, s.lim - 32, small, nref);
  } else if (s.partial) {
    mask_columns(u[0], s.lim, -INFINITY);
    mask_columns(u[1], s.lim - 32, -INFINITY);
  }
  if (SCORE == kScoreBias || (SCORE == kScoreCap && s.bias)) bias_args<SCORE>(u, sl2, s, nref);
  return MAX ? row_max(u) : 0.f;
}

}  // namespace

}  // namespace fa
