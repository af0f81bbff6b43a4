// cm_attn_decode over caches of type kInt8Block.
#include "attn_decode.cuh"

namespace cm {
template int launch_decode_kind<kInt8Block>(DecodeArgs&, int, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
}  // namespace cm
