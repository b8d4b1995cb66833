// Attention over a shared prefix, e4m3 codes; the launcher for both formats.
#include "kv_prefix.cuh"

namespace qg {

template int launch_prefix<false>(AttnArgs&, cudaStream_t);
extern template int launch_prefix<true>(AttnArgs&, cudaStream_t);

int launch_attn_prefix(AttnArgs& a, bool int8, cudaStream_t s) {
    return int8 ? launch_prefix<true>(a, s) : launch_prefix<false>(a, s);
}

}  // namespace qg
