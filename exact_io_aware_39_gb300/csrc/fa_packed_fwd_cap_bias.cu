// The packed forward (fa_packed_fwd.cuh) of scores capped by a tanh and lowered with distance.
#include "fa_packed_fwd.cuh"

namespace fa {

cudaError_t launch_packed_fwd_cap_bias(bool f16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                       const PackedFwdParams& p, cudaStream_t s) {
  return launch_packed_fwd_score<kScoreCap>(f16, tq, tk, tv, p, s);
}

}  // namespace fa
