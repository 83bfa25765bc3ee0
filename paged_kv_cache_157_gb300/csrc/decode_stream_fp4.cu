// Decode with a window and sinks, four-bit caches.
#include "decode_scored.cuh"

namespace kvc {

template kvc_status stream_launch<fp4e2m1>(const ScoredParams&, int, int, int, const CUtensorMap&, const CUtensorMap&,
                                      cudaStream_t);

}  // namespace kvc
