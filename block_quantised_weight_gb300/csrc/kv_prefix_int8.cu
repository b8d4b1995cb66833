// Attention over a shared prefix, int8 codes.
#include "kv_prefix.cuh"

namespace qg {

template int launch_prefix<true>(AttnArgs&, cudaStream_t);

}  // namespace qg
