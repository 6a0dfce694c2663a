// Instances for K format K_INT4_TOK of the paged decode that leaves its scores for
// kvq_weigh_decode.
#include "decode_launch.cuh"

namespace kvq {
template cudaError_t plan_decode_kf<K_INT4_TOK, true>(int, int, int, int, int, bool, DecodePlan *);
template cudaError_t launch_decode_kf<K_INT4_TOK, true>(int, int, const DecodeArgs &, const DecodePlan &, const DecodeMaps &,
                                                 cudaStream_t);
}  // namespace kvq
