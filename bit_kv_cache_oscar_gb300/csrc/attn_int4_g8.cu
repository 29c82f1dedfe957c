// The INT4 attention kernels for 8 query heads a kv head.
#include "attn_int4.cuh"

namespace oscar {
template cudaError_t launch_attn4<8>(const Attn4Args &, int, bool, const CUtensorMap &, const CUtensorMap &, int, cudaStream_t);
}  // namespace oscar
