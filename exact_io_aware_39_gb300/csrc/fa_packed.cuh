// Attention over packed sequences: what its translation units share (the plan
// of a call, parameter blocks, launchers). The C ABI is in flash_attn_packed.h.
#pragma once

#include "fa_common.cuh"
#include "fa_ptx.cuh"

namespace fa {

// A work item: rows start .. start + len - 1 are a sequence, c is the pair of
// 128-query tiles (forward) or the 128-key tile (backward) of it, slot0 the
// first of its tiles in the padded order of the backward's row vectors.
struct PackedItem {
  int start, len, c, slot0;
};

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
  size_t plan_off, sorted_off, item_off, tile_off, dq_off, lse2_off, delta_off, total;
  int cap_items, cap_tiles;
  bool ok;   // the counts fit 32-bit work indices
};

inline PackedWorkspace packed_workspace_layout(int B, int total, int Hq, int Hk, int d, bool backward) {
  auto al = [](size_t x) { return (x + 255) & ~size_t(255); };
  PackedWorkspace w;
  const long long tiles = (long long)total / kTile + B;
  const long long items = backward ? tiles : (long long)total / (2 * kTile) + B;
  w.ok = tiles * Hq < 0x7FFFFFFFll / kTile;
  w.cap_tiles = w.ok ? (int)tiles : 0;
  w.cap_items = w.ok ? (int)items : 0;
  w.plan_off = 0;
  w.sorted_off = al(sizeof(PackedPlan));
  w.item_off = al(w.sorted_off + (size_t)B * sizeof(int));
  w.tile_off = al(w.item_off + (size_t)w.cap_items * sizeof(PackedItem));
  w.dq_off = al(w.tile_off + (backward ? (size_t)w.cap_tiles * sizeof(PackedItem) : 0));
  const size_t rows = backward ? (size_t)Hq * w.cap_tiles * kTile : 0;
  w.lse2_off = al(w.dq_off + rows * d * sizeof(float));
  w.delta_off = al(w.lse2_off + rows * sizeof(float));
  w.total = al(w.delta_off + rows * sizeof(float));
  return w;
}

struct PackedFwdParams {
  const PackedItem* items;
  PackedPlan* plan;
  uint16_t* o;
  int64_t o_tok, o_head;
  float* lse;                 // [Hq, total]
  unsigned int* err;
  int total, Hq, G, d, causal;
  float scale_log2;
  uint32_t wait_us, stall;
  int cap_items;
  int group;                  // query heads per group of the work order
};

struct PackedBwdParams {
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
  int group;                  // key/value heads per group of the work order
};

// Zeroes rows r0 .. 127 of a 128-row tile (64-column atoms of 16 KB, D / 64 of
// them), executed by a whole warp on a tile that TMA has written: the rows
// behind a sequence's end hold other sequences' data or none, and a zero
// weight times what they hold must be zero. The fence orders the writes
// before the tensor core's reads (and later TMA writes).
template <int D>
__device__ __forceinline__ void zero_tail_rows(uint8_t* tile, int r0) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int h = 0; h < D / 64; ++h)
    for (int i = 8 * r0 + lane; i < 8 * kTile; i += 32)
      *reinterpret_cast<uint4*>(tile + h * 16384 + 16 * i) = make_uint4(0u, 0u, 0u, 0u);
  fence_proxy_async_smem();
  __syncwarp();
}

// Byte offset of 16-byte chunk c of row r in a 128-row tile stored as
// 64-column atoms 16 KB apart with 128-byte swizzling.
__device__ __forceinline__ uint32_t tile_chunk(int r, int c) {
  return (uint32_t)((c >> 3) * 16384 + (r >> 3) * 1024 + (r & 7) * 128 + (((c & 7) ^ (r & 7)) << 4));
}

cudaError_t launch_packed_plan(const int32_t* cu, int B, int total, int causal, bool backward, PackedPlan* plan,
                               int* sorted, PackedItem* items, int cap_items, PackedItem* tiles, int cap_tiles,
                               unsigned int* err, cudaStream_t s);

cudaError_t launch_packed_fwd(bool f16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& to, const PackedFwdParams& p, cudaStream_t s);

cudaError_t launch_packed_bwd(bool f16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tdo, const CUtensorMap& tdk, const CUtensorMap& tdv,
                              const CUtensorMap& tdq, const PackedBwdParams& p, cudaStream_t s);

}  // namespace fa
