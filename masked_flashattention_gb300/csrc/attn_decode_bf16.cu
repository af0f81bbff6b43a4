// cm_attn_decode over caches of type kBf16.
#include "attn_decode.cuh"

namespace cm {
template int launch_decode_kind<kBf16>(DecodeArgs&, int, const CUtensorMap&, const CUtensorMap&, cudaStream_t);
}  // namespace cm
