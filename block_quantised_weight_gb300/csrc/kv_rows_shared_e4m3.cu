// The row kernel for what is behind a shared prefix, e4m3 codes; the launcher for both formats.
#include "kv_rows.cuh"

namespace qg {

template int launch_rows<false, true>(const AttnArgs&, cudaStream_t);
extern template int launch_rows<true, true>(const AttnArgs&, cudaStream_t);

int launch_attn_rows_shared(const AttnArgs& a, bool int8, cudaStream_t s) {
    return int8 ? launch_rows<true, true>(a, s) : launch_rows<false, true>(a, s);
}

}  // namespace qg
