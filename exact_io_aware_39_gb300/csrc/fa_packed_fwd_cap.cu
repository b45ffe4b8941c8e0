// The packed forward (fa_packed_fwd.cuh) of scores capped by a tanh, without slopes.
// (Two sequences of 4547 and 5127 tokens, 32 / 8 heads, d = 128, bf16: 332 us, 1.16 PFLOP/s; plain scores 242.)
#include "fa_packed_fwd.cuh"

namespace fa {

cudaError_t launch_packed_fwd_cap(bool f16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                  const PackedFwdParams& p, cudaStream_t s) {
  return launch_packed_fwd_score<kScoreCapOnly>(f16, tq, tk, tv, p, s);
}

}  // namespace fa
