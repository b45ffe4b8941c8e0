// The packed forward (fa_packed_fwd.cuh) of scores lowered with distance, or with a prefix mask alone.
// (11 sequences of 64-4096 tokens with prefixes, 16 heads, d = 64, fp16: 169 us.)
#include "fa_packed_fwd.cuh"

namespace fa {

cudaError_t launch_packed_fwd_bias(bool f16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                                   const PackedFwdParams& p, cudaStream_t s) {
  return launch_packed_fwd_score<kScoreBias>(f16, tq, tk, tv, p, s);
}

}  // namespace fa
