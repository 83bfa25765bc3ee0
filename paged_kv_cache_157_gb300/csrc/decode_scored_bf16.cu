// Weight-accumulating decode, bf16 caches.
#include "decode_scored.cuh"

namespace kvc {

template kvc_status scored_launch<__nv_bfloat16>(const ScoredParams&, int, int, int, const CUtensorMap&, const CUtensorMap&,
                                         cudaStream_t);

}  // namespace kvc
