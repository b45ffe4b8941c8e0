// Attention over packed sequences: argument checks, tensor maps, the plan
// kernel and the launch sequences. The kernels are in fa_packed_fwd.cuh,
// fa_packed_bwd.cuh and fa_packed_dots.cuh.
#include "flash_attn_scored.h"
#include "fa_packed.cuh"

#include <cmath>

namespace fa {

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kMaxUnits = kMaxN / kTile;   // most tiles of a sequence: 1024

// The plan: which (sequence, tile) pairs there are, heaviest first, so that
// the persistent kernels end together. cu_seqlens lives on the device, so the
// list is made there, by one block. Sequences are sorted by their unit count
// (a counting sort; a unit is a query tile or a pair of them in the forward pass,
// a key tile in the backward). Causal: a unit with c units before it in the forward
// (or behind it in the backward) costs c + 1 tile pairs, so units are listed
// by c, descending: those of rank c are held by the first sequences of the
// sorted order, which gives every unit its place without a search. Not causal:
// a unit costs its sequence's length, so the units follow the sorted order.
// (Prefixes are not in the order: a forward unit that begins in one costs the tiles up
// to its end, however few come before it. 12 prompts whose longest, 4022 tokens, has a
// prefix of 3862: by a list schedule the busiest of 152 SMs gets 93 key tiles of pairs
// of query tiles, 73 in the order of their cost; the mean is 72.)
__global__ void __launch_bounds__(kPlanThreads)
packed_plan_kernel(const int32_t* __restrict__ cu, const int32_t* __restrict__ prefix, int B, int total, int rows, int causal, int backward,
                   PackedPlan* plan, int* sorted, PackedItem* items, int cap_items, PackedItem* tiles, int cap_tiles,
                   unsigned int* err) {
  __shared__ int hist[kMaxUnits + 1];      // sequences with that many units; then the next free rank
  __shared__ int off[kMaxUnits + 1];       // first list place of the units with c units before them
  __shared__ int warp_sum[2][32];
  __shared__ int carry[2];
  grid_dep_launch();   // the main kernel may set itself up (it waits for this one's end)
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  auto seq = [&](int b, int& start, bool& bad) -> int { return seq_bounds(cu, b, total, start, bad); };
  auto units = [&](int len) -> int { return (len + rows - 1) / rows; };

  for (int i = tid; i <= kMaxUnits; i += kPlanThreads) hist[i] = 0;
  if (tid < 2) carry[tid] = 0;
  __syncthreads();
  for (int b = tid; b < B; b += kPlanThreads) {
    int start;
    bool bad;
    const int len = seq(b, start, bad);
    if (bad) report_bounds(err, b);
    if (len > 0) atomicAdd(&hist[units(len)], 1);
  }
  __syncthreads();
  // Thread i stands for k = 1024 - i units: ge = sequences with at least k,
  // and the list places of the units with c = k - 1 units before them follow
  // those of all larger c.
  auto block_scan = [&](int v, int which, int& sum) -> int {   // inclusive
    int x = v;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
      if (lane >= o) x += y;
    }
    if (lane == 31) warp_sum[which][warp] = x;
    __syncthreads();
    int before = 0;
    sum = 0;
#pragma unroll
    for (int w = 0; w < 32; ++w) {
      const int y = warp_sum[which][w];
      if (w < warp) before += y;
      sum += y;
    }
    return x + before;
  };
  const int k = kMaxUnits - tid;
  const int mine = hist[k];
  int live = 0, n_causal = 0;
  const int ge = block_scan(mine, 0, live);
  const int upto = block_scan(ge, 1, n_causal);
  off[k - 1] = upto - ge;
  hist[k] = ge - mine;      // rank of the first sequence with k units
  __syncthreads();
  for (int b = tid; b < B; b += kPlanThreads) {
    int start;
    bool bad;
    const int len = seq(b, start, bad);
    if (len > 0) sorted[atomicAdd(&hist[units(len)], 1)] = b;
  }
  __syncthreads();
  // In sorted order, 1024 sequences at a time: the places of the units in that
  // order (the not causal list, and the padded order of tiles).
  for (int base = 0; base < live; base += kPlanThreads) {
    const int rank = base + tid;
    int start = 0, len = 0;
    bool bad;
    int pre = 0;
    if (rank < live) {
      len = seq(sorted[rank], start, bad);
      pre = seq_prefix(prefix, sorted[rank], len);
    }
    const int n = units(len);
    int sum = 0;
    const int first = carry[0] + block_scan(n, (base / kPlanThreads) & 1, sum) - n;
    __syncthreads();
    if (tid == 0) carry[0] += sum;
    // a warp writes the units of its 32 sequences, one sequence after another
    for (int l = 0; l < 32; ++l) {
      const int nn = __shfl_sync(0xFFFFFFFFu, n, l);
      if (nn == 0) continue;
      const int s = __shfl_sync(0xFFFFFFFFu, start, l), ln = __shfl_sync(0xFFFFFFFFu, len, l);
      const int f = __shfl_sync(0xFFFFFFFFu, first, l), rk = __shfl_sync(0xFFFFFFFFu, rank, l);
      const int pr = __shfl_sync(0xFFFFFFFFu, pre, l);
      for (int c = lane; c < nn; c += 32) {
        // backward, causal: key tile kj has nn - 1 - kj query tiles behind it
        // (a sequence past the padded rows -- bounds that overlap -- is left out)
        const PackedItem it{s, backward && f + nn > cap_tiles ? 0 : ln, with_prefix(backward && causal ? nn - 1 - c : c, pr), f};
        const int at = causal ? off[c] + rk : f + c;
        if (at < cap_items) items[at] = it;
        if (backward && f + c < cap_tiles) tiles[f + c] = PackedItem{s, ln, with_prefix(c, pr), f};
      }
    }
    __syncthreads();
  }
  if (tid == 0) {
    // (bounds that overlap can name more tiles than the lists hold)
    const int n = carry[0];
    plan->items = n < cap_items ? n : cap_items;
    plan->tiles = n < cap_tiles ? n : cap_tiles;
    plan->sched = 0u;
  }
}

fa_status check_packed_shape(int B, int total, int Hq, int Hk, int d) {
  if (B < 0 || total < 0 || Hk < 1 || Hq < 1 || Hq % Hk != 0) return FA_ERR_INVALID_ARG;
  if (d < 8 || d > 128 || d % 8 != 0) return FA_ERR_UNSUPPORTED;
  if (!packed_workspace_layout(B, total, Hq, Hk, d, true).ok) return FA_ERR_UNSUPPORTED;
  return FA_OK;
}

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

struct Strides {
  int64_t tok, head;
};

bool read_strides(const int64_t* strides, int i, int H, int d, Strides* out) {
  if (strides == nullptr) {
    *out = Strides{(int64_t)H * d, d};
    return true;
  }
  *out = Strides{strides[2 * i], strides[2 * i + 1]};
  for (int64_t x : {out->tok, out->head})
    if (x <= 0 || (x & 7) != 0 || x >= ((int64_t)1 << 36)) return false;
  return true;
}

// Strided [total, H, d] tensor as {d, H, total}, box 64 columns x 1 head x rows.
int packed_map(CUtensorMap* m, const void* base, bool f16, int total, int H, int d, const Strides& st, int rows) {
  const uint64_t dims[3] = {(uint64_t)d, (uint64_t)H, (uint64_t)total};
  const uint64_t strides[2] = {(uint64_t)st.head * 2, (uint64_t)st.tok * 2};
  const uint32_t box[3] = {64, 1, (uint32_t)rows};
  return internal_tensor_map(m, f16 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT16 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, base, dims,
                             strides, box, CU_TENSOR_MAP_SWIZZLE_128B);
}

struct PackedOptions {
  bool f16;
  uint32_t wait_us, stall;
};

fa_status packed_options(const fa_options* options, PackedOptions* o) {
  bool record = false;
  const int st = internal_read_check_options(options, &o->f16, &record, &o->wait_us, &o->stall);
  if (st != FA_OK) return static_cast<fa_status>(st);
  return record ? FA_ERR_UNSUPPORTED : FA_OK;
}

}  // namespace

cudaError_t launch_packed_plan(const int32_t* cu, const int32_t* prefix, int B, int total, int rows, int causal,
                               bool backward, PackedPlan* plan, int* sorted, PackedItem* items, int cap_items, PackedItem* tiles,
                               int cap_tiles, unsigned int* err, cudaStream_t s) {
  packed_plan_kernel<<<1, kPlanThreads, 0, s>>>(cu, prefix, B, total, rows, causal, backward ? 1 : 0, plan, sorted, items,
                                                cap_items, tiles, cap_tiles, err);
  return cudaGetLastError();
}

namespace {

fa_status packed_fwd_call(const void* Q, const void* K, const void* V, void* O, float* LSE,
                                const int32_t* cu_seqlens, int B, int total, int Hq, int Hk, int d,
                                const int64_t* strides, float scale, int causal, const fa_scores* scores, const fa_options* options,
                                void* workspace, size_t workspace_bytes, void* stream) {
  fa_status st = check_packed_shape(B, total, Hq, Hk, d);
  if (st != FA_OK) return st;
  if (!std::isfinite(scale) || scale <= 0.f || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARG;
  PackedOptions o;
  if ((st = packed_options(options, &o)) != FA_OK) return st;
  ScoreParams score;
  if ((st = read_scores(scores, scale, causal, false, &score)) != FA_OK) return st;
  Strides sq, sk, sv, so;
  if (!read_strides(strides, 0, Hq, d, &sq) || !read_strides(strides, 1, Hk, d, &sk) ||
      !read_strides(strides, 2, Hk, d, &sv) || !read_strides(strides, 3, Hq, d, &so))
    return FA_ERR_INVALID_ARG;
  if (B == 0 || total == 0) return FA_OK;
  const void* ptrs[] = {Q, K, V, O};
  for (const void* x : ptrs)
    if (x == nullptr || !aligned(x, 16)) return FA_ERR_INVALID_ARG;
  if (LSE == nullptr || !aligned(LSE, 4) || cu_seqlens == nullptr || !aligned(cu_seqlens, 4)) return FA_ERR_INVALID_ARG;
  const PackedWorkspace w = packed_workspace_layout(B, total, Hq, Hk, d, false);
  if (!(B <= kDirect && workspace == nullptr) &&   // (up to kDirect sequences use none)
      (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < w.total))
    return FA_ERR_WORKSPACE;
  unsigned int* err = nullptr;
  const int e = internal_device_error_word(&err);
  if (e != FA_OK) return static_cast<fa_status>(e);
  CUtensorMap tq, tk, tv;
  if (packed_map(&tq, Q, o.f16, total, Hq, d, sq, kTile) || packed_map(&tk, K, o.f16, total, Hk, d, sk, kTile) ||
      packed_map(&tv, V, o.f16, total, Hk, d, sv, kTile))
    return FA_ERR_CUDA;
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PackedFwdParams p{};
  if (B > kDirect) {
    p.items = reinterpret_cast<PackedItem*>(ws + w.item_off);
    p.plan = reinterpret_cast<PackedPlan*>(ws + w.plan_off);
  }
  p.o = static_cast<uint16_t*>(O);
  p.o_tok = so.tok;
  p.o_head = so.head;
  p.lse = LSE;
  p.err = err;
  p.total = total;
  p.Hq = Hq;
  p.G = Hq / Hk;
  p.d = d;
  p.causal = causal;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_us = o.wait_us;
  p.stall = o.stall;
  p.cu = cu_seqlens;
  p.B = B;
  p.score = score;
  p.split = packed_split(B, total, Hq, w.cap_tiles, causal != 0);
  p.cap_items = p.split ? w.cap_tiles : w.cap_items;
  p.pair_heads = !p.split && packed_pair_heads(Hq, Hk);
  p.heads = p.pair_heads ? Hq / 2 : Hq;
  if (B > kDirect &&
      launch_packed_plan(cu_seqlens, p.score.prefix, B, total, p.pair_heads ? kTile : 2 * kTile, causal, false, p.plan,
                         reinterpret_cast<int*>(ws + w.sorted_off), reinterpret_cast<PackedItem*>(ws + w.item_off),
                         w.cap_items, nullptr, 0, err, s) != cudaSuccess)
    return FA_ERR_CUDA;
  const auto launch = score.cap ? (score.slopes ? launch_packed_fwd_cap_bias : launch_packed_fwd_cap)
                      : score.slopes || score.prefix ? launch_packed_fwd_bias : launch_packed_fwd;
  return launch(o.f16, tq, tk, tv, p, s) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

fa_status packed_bwd_call(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                                const float* LSE, void* dQ, void* dK, void* dV, const int32_t* cu_seqlens, int B,
                                int total, int Hq, int Hk, int d, const int64_t* strides, float scale, int causal,
                                const fa_scores* scores, const fa_options* options, void* workspace, size_t workspace_bytes, void* stream) {
  fa_status st = check_packed_shape(B, total, Hq, Hk, d);
  if (st != FA_OK) return st;
  if (!std::isfinite(scale) || scale <= 0.f || (causal != 0 && causal != 1)) return FA_ERR_INVALID_ARG;
  PackedOptions o;
  if ((st = packed_options(options, &o)) != FA_OK) return st;
  ScoreParams score;
  if ((st = read_scores(scores, scale, causal, false, &score)) != FA_OK) return st;
  Strides ss[8];   // Q, K, V, O, dO, dQ, dK, dV
  const int heads[8] = {Hq, Hk, Hk, Hq, Hq, Hq, Hk, Hk};
  for (int i = 0; i < 8; ++i)
    if (!read_strides(strides, i, heads[i], d, &ss[i])) return FA_ERR_INVALID_ARG;
  if (B == 0 || total == 0) return FA_OK;
  const void* ptrs[] = {Q, K, V, O, dO, dQ, dK, dV};
  for (const void* x : ptrs)
    if (x == nullptr || !aligned(x, 16)) return FA_ERR_INVALID_ARG;
  if (LSE == nullptr || !aligned(LSE, 4) || cu_seqlens == nullptr || !aligned(cu_seqlens, 4)) return FA_ERR_INVALID_ARG;
  const PackedWorkspace w = packed_workspace_layout(B, total, Hq, Hk, d, true);
  if (workspace == nullptr || !aligned(workspace, 256) || workspace_bytes < w.total) return FA_ERR_WORKSPACE;
  unsigned int* err = nullptr;
  const int e = internal_device_error_word(&err);
  if (e != FA_OK) return static_cast<fa_status>(e);
  uint8_t* ws = static_cast<uint8_t*>(workspace);
  float* dq_acc = reinterpret_cast<float*>(ws + w.dq_off);
  CUtensorMap tq, tk, tv, tdo, tdq;
  if (packed_map(&tq, Q, o.f16, total, Hq, d, ss[0], kTile) || packed_map(&tk, K, o.f16, total, Hk, d, ss[1], kTile) ||
      packed_map(&tv, V, o.f16, total, Hk, d, ss[2], kTile) || packed_map(&tdo, dO, o.f16, total, Hq, d, ss[4], kTile))
    return FA_ERR_CUDA;
  {
    // the dQ accumulator [Hq, padded rows, d], box 32 fp32 columns: whole
    // 128-row tiles at a tile width of 64, each warp its 32 rows at 128
    const uint64_t rows = (uint64_t)w.cap_tiles * kTile;
    const uint64_t dims[3] = {(uint64_t)d, rows, (uint64_t)Hq};
    const uint64_t str[2] = {(uint64_t)d * 4, rows * d * 4};
    const uint32_t box[3] = {32, d <= 64 ? (uint32_t)kTile : 32u, 1};
    if (internal_tensor_map(&tdq, CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 3, dq_acc, dims, str, box, CU_TENSOR_MAP_SWIZZLE_128B))
      return FA_ERR_CUDA;
  }
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  PackedBwdParams p{};
  p.items = reinterpret_cast<PackedItem*>(ws + w.item_off);
  p.tiles = reinterpret_cast<PackedItem*>(ws + w.tile_off);
  p.plan = reinterpret_cast<PackedPlan*>(ws + w.plan_off);
  p.o = static_cast<const uint16_t*>(O);
  p.dout = static_cast<const uint16_t*>(dO);
  p.o_tok = ss[3].tok;
  p.o_head = ss[3].head;
  p.do_tok = ss[4].tok;
  p.do_head = ss[4].head;
  p.lse = LSE;
  p.dq_acc = dq_acc;
  p.lse2 = reinterpret_cast<float*>(ws + w.lse2_off);
  p.delta = reinterpret_cast<float*>(ws + w.delta_off);
  p.dq = static_cast<uint16_t*>(dQ);
  p.dk = static_cast<uint16_t*>(dK);
  p.dv = static_cast<uint16_t*>(dV);
  p.dq_tok = ss[5].tok;
  p.dq_head = ss[5].head;
  p.dk_tok = ss[6].tok;
  p.dk_head = ss[6].head;
  p.dv_tok = ss[7].tok;
  p.dv_head = ss[7].head;
  p.err = err;
  p.total = total;
  p.Hq = Hq;
  p.Hk = Hk;
  p.G = Hq / Hk;
  p.d = d;
  p.causal = causal;
  p.cap_tiles = w.cap_tiles;
  p.parts = w.parts;
  p.part = reinterpret_cast<float*>(ws + w.part_off);
  p.scale = scale;
  p.scale_log2 = scale * 1.4426950408889634f;
  p.wait_us = o.wait_us;
  p.stall = o.stall;
  p.cu = cu_seqlens;
  p.B = B;
  p.score = score;
  if (B > kDirect &&
      launch_packed_plan(cu_seqlens, p.score.prefix, B, total, kTile, causal, true, p.plan, reinterpret_cast<int*>(ws + w.sorted_off),
                         reinterpret_cast<PackedItem*>(ws + w.item_off), w.cap_items,
                         reinterpret_cast<PackedItem*>(ws + w.tile_off), w.cap_tiles, err, s) != cudaSuccess)
    return FA_ERR_CUDA;
  const auto launch = score.cap ? launch_packed_bwd_cap : score.slopes || score.prefix ? launch_packed_bwd_bias : launch_packed_bwd;
  return launch(o.f16, tq, tk, tv, tdo, tdq, p, s) == cudaSuccess ? FA_OK : FA_ERR_CUDA;
}

}  // namespace

}  // namespace fa

using namespace fa;

extern "C" {

size_t flash_attn_packed_workspace_size(int B, int total, int Hq, int Hk, int d, int backward) {
  if (check_packed_shape(B, total, Hq, Hk, d) != FA_OK) return 0;
  return packed_workspace_layout(B, total, Hq, Hk, d, backward != 0).total;
}

fa_status flash_attn_packed_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE,
                                const int32_t* cu_seqlens, int B, int total, int Hq, int Hk, int d,
                                const int64_t* strides, float scale, int causal, const fa_options* options,
                                void* workspace, size_t workspace_bytes, void* stream) {
  return packed_fwd_call(Q, K, V, O, LSE, cu_seqlens, B, total, Hq, Hk, d, strides, scale, causal, nullptr, options,
                         workspace, workspace_bytes, stream);
}

fa_status flash_attn_packed_scored_fwd(const void* Q, const void* K, const void* V, void* O, float* LSE,
                                       const int32_t* cu_seqlens, int B, int total, int Hq, int Hk, int d,
                                       const int64_t* strides, float scale, int causal, const fa_scores* scores,
                                       const fa_options* options, void* workspace, size_t workspace_bytes,
                                       void* stream) {
  return packed_fwd_call(Q, K, V, O, LSE, cu_seqlens, B, total, Hq, Hk, d, strides, scale, causal, scores, options,
                         workspace, workspace_bytes, stream);
}

fa_status flash_attn_packed_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                                const float* LSE, void* dQ, void* dK, void* dV, const int32_t* cu_seqlens, int B,
                                int total, int Hq, int Hk, int d, const int64_t* strides, float scale, int causal,
                                const fa_options* options, void* workspace, size_t workspace_bytes, void* stream) {
  return packed_bwd_call(Q, K, V, O, dO, LSE, dQ, dK, dV, cu_seqlens, B, total, Hq, Hk, d, strides, scale, causal,
                         nullptr, options, workspace, workspace_bytes, stream);
}

fa_status flash_attn_packed_scored_bwd(const void* Q, const void* K, const void* V, const void* O, const void* dO,
                                       const float* LSE, void* dQ, void* dK, void* dV, const int32_t* cu_seqlens,
                                       int B, int total, int Hq, int Hk, int d, const int64_t* strides, float scale,
                                       int causal, const fa_scores* scores, const fa_options* options,
                                       void* workspace, size_t workspace_bytes, void* stream) {
  return packed_bwd_call(Q, K, V, O, dO, LSE, dQ, dK, dV, cu_seqlens, B, total, Hq, Hk, d, strides, scale, causal,
                         scores, options, workspace, workspace_bytes, stream);
}

}  // extern "C"
