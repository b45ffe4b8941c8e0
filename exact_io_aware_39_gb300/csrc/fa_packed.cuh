// Attention over packed sequences: what its translation units share (the plan
// of a call, parameter blocks, launchers). The C ABI is in flash_attn_packed.h.
#pragma once

#include "fa_common.cuh"
#include "fa_ptx.cuh"
#include "fa_scores.cuh"
#include "fa_warp.cuh"

namespace fa {

// A work item: rows start .. start + len - 1 are a sequence, c is the 128-query
// tile or pair of them (forward) or the 128-key tile (backward) of it, slot0 the
// first of its tiles in the padded order of the backward's row vectors.
struct PackedItem {
  int start, len, c, slot0;
};
// With a prefix mask, an item that is handed on (in a list or a ring) has its
// sequence's prefix length above the tile number in c.
constexpr int kPrefixShift = 11;
static_assert(kMaxN / kTile < (1 << kPrefixShift) && kMaxN <= (0x7FFFFFFF >> kPrefixShift), "prefix and tile number share c");
__host__ __device__ __forceinline__ int with_prefix(int c, int prefix) { return c | (prefix << kPrefixShift); }
__host__ __device__ __forceinline__ int tile_of(int c) { return c & ((1 << kPrefixShift) - 1); }
__host__ __device__ __forceinline__ int prefix_of(int c) { return c >> kPrefixShift; }

// Written by the plan kernel at the head of the workspace.
struct PackedPlan {
  int items;             // entries of the item list
  int tiles;             // entries of the tile list (backward)
  unsigned int sched;    // next item of the persistent main kernel
  int pad;
};

// Workspace sections (byte offsets, 256-aligned). The lists are sized for the
// most tiles B sequences of `total` tokens can have.
struct PackedWorkspace {
  size_t plan_off, sorted_off, item_off, tile_off, dq_off, lse2_off, delta_off, part_off, total;
  int cap_items, cap_tiles;
  int parts;   // backward: parts of a work item
  bool ok;   // the counts fit 32-bit work indices
};

// The forward's work item is one query tile of two neighbouring query heads of
// a key/value head where there are such pairs, else two query tiles of a head
// (24 sequences of 16-2048 tokens, 32 / 8 heads, d = 128: 105 us with pairs of
// heads, 118 with pairs of tiles; one of 16384: 1211 and 1232).
inline bool packed_pair_heads(int Hq, int Hk) { return (Hq / Hk) % 2 == 0; }

// Where there are not more query tiles than SMs, the forward's item is one query
// tile whose key tiles the two softmax groups take in turn (SPLIT), so that the
// longest item is half as long: one sequence of 2176 tokens, 5 heads, causal, 17.9
// us against 27.2 in pairs at d = 128, 14.9 against 21.5 at 64. Causal, whose items
// differ in length, up to 256 tiles (two sequences of 3149 tokens, 4 heads: 24.2 and
// 39.3; 288 tiles of 1100 tokens 19.1 and 18.9); not causal, 192 tiles of 700 tokens
// would take 19.6 us and take 16.6. Sequences of one tile have nothing to share out.
inline bool packed_split(int B, int total, int Hq, int cap_tiles, bool causal) {
  return B <= 32 && total > kTile * B && (long long)cap_tiles * Hq <= (causal ? 256 : 152);
}

// Up to kDirect sequences: no plan kernel runs, every warp that needs the work
// list makes it from the bounds (DirectList): 10 us less for a forward call, 19
// for forward and backward (33 sequences of 40 tokens: 17.5 -> 8.2 and 47.7 ->
// 29.0 us).
constexpr int kDirect = 128, kManySlots = kDirect / 32;
inline bool packed_many(int B) { return B > 32 && B <= kDirect; }

// The backward's item is a key tile of a key/value head with all of its query
// tiles, of all G query heads: G n steps for the first tile of a sequence of n
// tiles. Where there are not two items for every SM, items are cut into parts
// of about as many steps as an SM gets in all, whose dK and dV are summed by the
// last pass.
constexpr int kMaxParts = 16;
inline int packed_bwd_parts(int B, int total, int Hk, int G, long long tiles) {
  constexpr double kSms = 152.;
  const double items = (double)tiles * Hk;
  if (items >= 2. * kSms || B < 1 || B > kDirect) return 1;   // (with more than kDirect sequences it would be 1)
  const double n = (double)((total + (long long)kTile * B - 1) / ((long long)kTile * B));   // tiles of an average sequence
  const double per_sm = items * G * (n + 1.) / 2. / kSms;
  const double parts = G * n / (per_sm > 1. ? per_sm : 1.);
  return parts >= kMaxParts ? kMaxParts : parts <= 1. ? 1 : (int)parts;
}

inline PackedWorkspace packed_workspace_layout(int B, int total, int Hq, int Hk, int d, bool backward) {
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  PackedWorkspace w;
  const long long tiles = (long long)total / kTile + B;
  w.ok = tiles * Hq < 0x7FFFFFFFll / kTile;
  w.cap_tiles = w.ok ? (int)tiles : 0;
  w.cap_items = !w.ok ? 0 : (int)(backward || packed_pair_heads(Hq, Hk) ? tiles : (long long)total / (2 * kTile) + B);
  w.plan_off = 0;
  w.sorted_off = al(sizeof(PackedPlan));
  w.item_off = al(w.sorted_off + (size_t)B * sizeof(int));
  w.tile_off = al(w.item_off + (size_t)w.cap_items * sizeof(PackedItem));
  w.dq_off = al(w.tile_off + (backward ? (size_t)w.cap_tiles * sizeof(PackedItem) : 0));
  const size_t rows = backward ? (size_t)Hq * w.cap_tiles * kTile : 0;
  w.lse2_off = al(w.dq_off + rows * d * sizeof(float));
  w.delta_off = al(w.lse2_off + rows * sizeof(float));
  w.part_off = al(w.delta_off + rows * sizeof(float));
  w.parts = backward && w.ok ? packed_bwd_parts(B, total, Hk, Hq / Hk, tiles) : 1;
  w.total = w.part_off;
  if (w.parts > 1) w.total = al(w.part_off + (size_t)w.parts * 2 * Hk * w.cap_tiles * kTile * d * sizeof(float));
  return w;
}

struct PackedFwdParams {
  const int32_t* cu;          // [B + 1]
  int B;
  const PackedItem* items;    // B > kDirect
  PackedPlan* plan;
  uint16_t* o;
  int64_t o_tok, o_head;
  float* lse;                 // [Hq, total]
  unsigned int* err;
  int total, Hq, G, d, causal;
  float scale_log2;
  uint32_t wait_us, stall;
  int cap_items;
  int pair_heads;             // an item's two query tiles: one tile of two heads, or two tiles of one head
  int split;                  // an item is one query tile, its keys shared out between the softmax groups
  int heads;                  // Hq, or with pair_heads Hq / 2
  int group;                  // of those, per group of the work order
  ScoreParams score;
};

struct PackedBwdParams {
  const int32_t* cu;          // [B + 1]
  int B;
  // B > kDirect:
  const PackedItem* items;    // (sequence, key tile)
  const PackedItem* tiles;    // every tile, in padded order
  PackedPlan* plan;
  const uint16_t *o, *dout;   // strided
  int64_t o_tok, o_head, do_tok, do_head;
  const float* lse;
  float* dq_acc;              // [Hq, cap_tiles * 128, d]
  float* lse2;                // [Hq, cap_tiles * 128]: LSE * log2(e), +inf on padding
  float* delta;               // the same: rowsum(dO * O)
  uint16_t *dq, *dk, *dv;
  int64_t dq_tok, dq_head, dk_tok, dk_head, dv_tok, dv_head;
  unsigned int* err;
  int total, Hq, Hk, G, d, causal, cap_tiles;
  float scale, scale_log2;
  uint32_t wait_us, stall;
  int parts;                  // of an item
  float* part;                // parts > 1: fp32 [parts, 2 (dK, dV), Hk, cap_tiles * 128, d]
  int group;                  // (key/value head, part) pairs per group of the work order
  ScoreParams score;
};

// Rows [start, start + len) of sequence b; an empty one (bad set) where its
// bounds decrease, leave [0, total] or span more than kMaxN tokens.
__device__ __forceinline__ int seq_bounds(const int32_t* cu, int b, int total, int& start, bool& bad) {
  const int s = cu[b], e = cu[b + 1];
  bad = s < 0 || e < s || e > total || e - s > kMaxN;
  start = s;
  return bad ? 0 : e - s;
}

// The prefix of sequence b (len tokens); 0 without a prefix mask.
__device__ __forceinline__ int seq_prefix(const int32_t* prefix, int b, int len) {
  return prefix == nullptr ? 0 : max(0, min(prefix[b], len));
}

__device__ __forceinline__ void report_bounds(unsigned int* err, int b) {
  if (atomicCAS(err, 0u, (unsigned)kErrInternal) == 0u) {
    err[1] = 300u;
    err[2] = blockIdx.x;
    err[3] = (unsigned)b;
  }
}

// The work list of up to kDirect sequences, held by a warp: lane l has the
// sequences l, l + 32, ... (its slots) and their n units of `rows` rows, slot0
// the units before each of them, lane by lane. A sequence that would end past
// `cap` units in all (only bounds that overlap can name so many) is left out.
// Units are listed as the plan kernel lists them: causal, by the number c of
// units before them, descending, and for each c the sequences that have one; not
// causal, sequence by sequence, the longest first (prefixes change what a unit
// costs, but not its place). All lanes call the members
// together. kSlots = kManySlots holds them all, 1 up to 32
// (kernels are built for either: the claim of an item stands before its loads, and
// with four slots for every call 24 prompts took 107 us, not 105).
// kPre: the sequences' prefixes too (that of the last one named is in `prefix`).
template <int kSlots, bool kPre = false>
struct DirectList {
  int start[kSlots], len[kSlots], n[kSlots], slot0[kSlots], items;
  int pre[kPre ? kSlots : 1], prefix;
  int c, off;          // causal: items with more than c units before them, and how many
  int first[kSlots];   // not causal: list place of a sequence's first unit
  // the sequences alone (err may be null)
  __device__ __forceinline__ void read(const int32_t* cu, const int32_t* prefixes, int B, int total, int rows, int cap,
                                       unsigned int* err) {
    const int lane = threadIdx.x & 31;
    bool bad[kSlots];
    int mine = 0;
    prefix = 0;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      const int b = 32 * s + lane;
      start[s] = len[s] = 0;
      bad[s] = false;
      if (b < B) len[s] = seq_bounds(cu, b, total, start[s], bad[s]);
      if constexpr (kPre) pre[s] = b < B ? seq_prefix(prefixes, b, len[s]) : 0;
      n[s] = (len[s] + rows - 1) / rows;
      mine += n[s];
    }
    int upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
    upto -= mine;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      slot0[s] = upto;
      upto += n[s];
      if (upto > cap) {
        bad[s] = bad[s] || n[s] > 0;
        len[s] = n[s] = 0;
      }
      if (bad[s] && err != nullptr) report_bounds(err, 32 * s + lane);
    }
  }
  __device__ __forceinline__ int most() const {
    int m = 0;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) m = max(m, n[s]);
    return __reduce_max_sync(0xFFFFFFFFu, m);
  }
  // sequences with more than c units
  __device__ __forceinline__ int count(int c) const {
    int x = 0;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) x += __popc(__ballot_sync(0xFFFFFFFFu, n[s] > c));
    return x;
  }
  // (per: the units are so many of those of `rows` rows, which slot0 goes on counting)
  __device__ __forceinline__ void init(const int32_t* cu, const int32_t* prefixes, int B, int total, int rows, int cap,
                                       bool causal, unsigned int* err, int per = 1) {
    const int lane = threadIdx.x & 31;
    read(cu, prefixes, B, total, rows, cap, err);
    if (per > 1)
#pragma unroll
      for (int s = 0; s < kSlots; ++s) n[s] = (n[s] + per - 1) / per;
    items = 0;
#pragma unroll
    for (int s = 0; s < kSlots; ++s) {
      items += n[s];
      first[s] = 0;
    }
    items = __reduce_add_sync(0xFFFFFFFFu, items);
    c = most() - 1;
    off = 0;
    if (!causal)
#pragma unroll
      for (int s = 0; s < kSlots; ++s)
#pragma unroll 1
        for (int l = 0; l < 32; ++l) {
          const int o = __shfl_sync(0xFFFFFFFFu, n[s], l);
#pragma unroll
          for (int t = 0; t < kSlots; ++t)
            if (o > n[t] || (o == n[t] && (s < t || (s == t && l < lane)))) first[t] += o;
        }
  }
  __device__ __forceinline__ PackedItem at(int idx, bool causal) {
    uint32_t mine = 0u;
    int t = 0;           // the slot; the lane is mine's lowest
    if (causal) {
      if (idx < off) {     // the order starts again for another group of heads
        c = most() - 1;
        off = 0;
      }
      int x = count(c);
#pragma unroll 1
      while (c > 0 && idx >= off + x) {
        off += x;
        --c;
        x = count(c);
      }
      int r = idx - off;
      mine = __ballot_sync(0xFFFFFFFFu, n[0] > c);
#pragma unroll
      for (int s = 1; s < kSlots; ++s)
        if (t == s - 1 && r >= __popc(mine)) {
          r -= __popc(mine);
          t = s;
          mine = __ballot_sync(0xFFFFFFFFu, n[s] > c);
        }
#pragma unroll 1
      for (; r > 0; --r) mine &= mine - 1;
    } else {
#pragma unroll
      for (int s = 0; s < kSlots; ++s)
        if (mine == 0u) {
          mine = __ballot_sync(0xFFFFFFFFu, n[s] > 0 && idx >= first[s] && idx < first[s] + n[s]);
          t = s;
        }
    }
    PackedItem it = get(t, __ffs(mine) - 1);
    it.c = causal ? c : idx - it.c;
    return it;
  }
  // the unit at place `slot` of the sequences' order; len 0 where there is none
  __device__ __forceinline__ PackedItem unit(int slot) {
    uint32_t mine = 0u;
    int t = 0;
#pragma unroll
    for (int s = 0; s < kSlots; ++s)
      if (mine == 0u) {
        mine = __ballot_sync(0xFFFFFFFFu, slot >= slot0[s] && slot < slot0[s] + n[s]);
        t = s;
      }
    if (mine == 0u) return PackedItem{0, 0, 0, 0};
    PackedItem it = get(t, __ffs(mine) - 1);
    it.c = slot - it.slot0;
    return it;
  }
  // the sequence in slot t of lane l (c: its `first`)
  __device__ __forceinline__ PackedItem get(int t, int l) {
    int st = start[0], le = len[0], sl = slot0[0], fi = first[0];
    if constexpr (kPre) {
      int pr = pre[0];
#pragma unroll
      for (int s = 1; s < kSlots; ++s)
        if (t == s) pr = pre[s];
      prefix = __shfl_sync(0xFFFFFFFFu, pr, l);
    }
#pragma unroll
    for (int s = 1; s < kSlots; ++s)
      if (t == s) {
        st = start[s];
        le = len[s];
        sl = slot0[s];
        fi = first[s];
      }
    return PackedItem{__shfl_sync(0xFFFFFFFFu, st, l), __shfl_sync(0xFFFFFFFFu, le, l), __shfl_sync(0xFFFFFFFFu, fi, l),
                      __shfl_sync(0xFFFFFFFFu, sl, l)};
  }
};

// Warp-wide MMAs as mma_ss_w / mma_ts_w, with a shared-memory descriptor given
// by its low word: only the address field, there, changes from one product to
// the next, and the high word of every descriptor of these kernels (stride
// 1024 bytes, version 1, 128-byte swizzle) is one constant.
constexpr uint32_t kDescHi = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void mma_ss_lo(uint32_t d_tmem, uint32_t a_lo, uint32_t b_lo, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 a, b;\n\t"
      "mov.b64 a, {%1, %5};\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a_lo), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi));
}
__device__ __forceinline__ void mma_ts_lo(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_lo, uint32_t idesc,
                                          uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t.reg .b64 b;\n\t"
      "mov.b64 b, {%2, %5};\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "@e tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n\t}"
      :: "r"(d_tmem), "r"(a_tmem), "r"(b_lo), "r"(idesc), "r"(accumulate), "r"(kDescHi));
}
// low words of desc_kmajor / desc_mnmajor at step 0, and their steps
__device__ __forceinline__ uint32_t desc_lo(uint64_t d) { return (uint32_t)d; }

// Zeroes rows r0 .. 127 of a 128-row tile (64-column atoms of 16 KB, D / 64 of
// them), executed by a whole warp on a tile that TMA has written: the rows
// behind a sequence's end hold other sequences' data or none, and a zero
// weight times what they hold must be zero. The fence orders the writes
// before the tensor core's reads (and later TMA writes).
template <int D>
__device__ __forceinline__ void zero_tail_rows(uint8_t* tile, int r0) {
  const int lane = threadIdx.x & 31;
#pragma unroll 1
  for (int i = 8 * r0 + lane; i < 8 * kTile; i += 32)
#pragma unroll
    for (int h = 0; h < D / 64; ++h) *reinterpret_cast<uint4*>(tile + h * 16384 + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

// Byte offset of 16-byte chunk c of row r in a 128-row tile stored as
// 64-column atoms 16 KB apart with 128-byte swizzling.
__device__ __forceinline__ uint32_t tile_chunk(int r, int c) {
  return (uint32_t)((c >> 3) * 16384 + (r >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4));
}

// rows: rows of a unit (a work item's share of a sequence). prefix: [B] or null.
cudaError_t launch_packed_plan(const int32_t* cu, const int32_t* prefix, int B, int total, int rows, int causal,
                               bool backward, PackedPlan* plan, int* sorted, PackedItem* items, int cap_items, PackedItem* tiles, int cap_tiles,
                               unsigned int* err, cudaStream_t s);

// One for each kind of score (kScorePlain, kScoreCap, kScoreBias; forward: kScoreCapOnly), from a
// translation unit of its own.
using PackedFwdLaunch = cudaError_t(bool f16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                    const PackedFwdParams& p, cudaStream_t s);
using PackedBwdLaunch = cudaError_t(bool f16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                    const CUtensorMap& tdo, const CUtensorMap& tdq, const PackedBwdParams& p,
                                    cudaStream_t s);
PackedFwdLaunch launch_packed_fwd, launch_packed_fwd_cap, launch_packed_fwd_bias, launch_packed_fwd_cap_bias;
PackedBwdLaunch launch_packed_bwd, launch_packed_bwd_cap, launch_packed_bwd_bias;

}  // namespace fa
