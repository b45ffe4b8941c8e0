// The attention of the newest tokens against the cache (fa_cached.cuh), scores capped by a tanh (and lowered with distance, where there are slopes).
#include "fa_cached.cuh"

namespace fa {

cudaError_t launch_cached_cap(bool e4m3, bool f16, const CUtensorMap& tk, const CUtensorMap& tv, const CUtensorMap& tks,
                              const CUtensorMap& tvs, const CachedParams& p, cudaStream_t s) {
  return launch_cached_score<kScoreCap>(e4m3, f16, tk, tv, tks, tvs, p, s);
}

}  // namespace fa
