// Weight-accumulating decode, f16 caches.
#include "decode_scored.cuh"

namespace kvc {

template kvc_status scored_launch<__half>(const ScoredParams&, int, int, int, const CUtensorMap&, const CUtensorMap&,
                                         cudaStream_t);

}  // namespace kvc
