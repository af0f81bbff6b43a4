// cm_attn_decode over caches of type kE4m3Block.
#include "attn_decode.cuh"

namespace cm {
template int launch_decode_kind<kE4m3Block>(DecodeArgs&, int, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
}  // namespace cm
