// Weight-accumulating decode, block-scaled int8 caches.
#include "decode_scored.cuh"

namespace kvc {

template kvc_status scored_launch<s8q>(const ScoredParams&, int, int, int, const CUtensorMap&, const CUtensorMap&,
                                         cudaStream_t);

}  // namespace kvc
