// Weight-accumulating decode, block-scaled e4m3 caches.
#include "decode_scored.cuh"

namespace kvc {

template kvc_status scored_launch<fp8e4m3>(const ScoredParams&, int, int, int, const CUtensorMap&, const CUtensorMap&,
                                         cudaStream_t);

}  // namespace kvc
