// The row kernel for what is behind a shared prefix, int8 codes.
#include "kv_rows.cuh"

namespace qg {

template int launch_rows<true, true>(const AttnArgs&, cudaStream_t);

}  // namespace qg
