// The row kernel for a shared prefix and what is behind it, int8 codes.
#include "kv_rows.cuh"

namespace qg {

template int launch_rows<true, true>(const AttnArgs&, cudaStream_t);

}  // namespace qg
