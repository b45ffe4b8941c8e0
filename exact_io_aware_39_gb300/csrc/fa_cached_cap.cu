// The attention of the newest tokens against the cache (fa_cached.cuh), scores capped by a tanh (and lowered with distance, where there are slopes).
// (64 sequences of 144891 tokens in all, 32 / 8 heads, d = 128, bf16: 106-110 us, plain scores 102.)
#include "fa_cached.cuh"

namespace fa {

cudaError_t launch_cached_cap(bool e4m3, bool f16, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tks,
                              const CUtensorMap& tvs, const CachedParams& p, cudaStream_t s) {
  return launch_cached_score<kScoreCap>(e4m3, f16, tk, tv, tks, tvs, p, s);
}

}  // namespace fa
