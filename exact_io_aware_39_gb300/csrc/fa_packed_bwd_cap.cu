// The packed backward (fa_packed_bwd.cuh) of scores capped by a tanh (and lowered with distance, where there are slopes).
// (Two sequences of 4547 and 5127 tokens, 32 / 8 heads, d = 128, bf16: 985 us beside the pass over D; plain scores 929.)
#include "fa_packed_bwd.cuh"

namespace fa {

cudaError_t launch_packed_bwd_cap(bool f16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                  const CUtensorMap& tdo, const CUtensorMap& tdq, const PackedBwdParams& p, cudaStream_t s) {
  return launch_packed_bwd_score<kScoreCap>(f16, tq, tk, tv, tdo, tdq, p, s);
}

}  // namespace fa
