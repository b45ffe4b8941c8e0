// The packed backward (fa_packed_bwd.cuh) of plain scores.
#include "fa_packed_bwd.cuh"

namespace fa {

cudaError_t launch_packed_bwd(bool f16, const CUtensorMap& tq, const CUtensorMap& tk, const CUtensorMap& tv,
                              const CUtensorMap& tdo, const CUtensorMap& tdq, const PackedBwdParams& p, cudaStream_t s) {
  return launch_packed_bwd_score<kScorePlain>(f16, tq, tk, tv, tdo, tdq, p, s);
}

}  // namespace fa
