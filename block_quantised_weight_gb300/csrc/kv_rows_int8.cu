// Attention of few rows, int8 codes.
#include "kv_rows.cuh"

namespace qg {

template int launch_rows<true, false>(const AttnArgs&, cudaStream_t);

}  // namespace qg
