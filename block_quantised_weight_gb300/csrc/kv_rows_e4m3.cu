// Attention of few rows, e4m3 codes; the launcher for both formats.
#include "kv_rows.cuh"

namespace qg {

template int launch_rows<false, false>(const AttnArgs&, cudaStream_t);
extern template int launch_rows<true, false>(const AttnArgs&, cudaStream_t);

bool encode_cache(CUtensorMap* map, const KVLayer& c, const uint8_t* base, int box_bytes, int box_tokens,
                  bool swizzle) {
    auto encode = tensor_map_encoder();
    if (!encode) return false;
    const cuuint64_t gdim[4] = {static_cast<cuuint64_t>(c.dim), cuuint64_t(1) << c.log2p,
                                static_cast<cuuint64_t>(c.heads), static_cast<cuuint64_t>(c.pages)};
    const cuuint64_t gstride[3] = {static_cast<cuuint64_t>(c.token_stride), static_cast<cuuint64_t>(c.head_stride),
                                   static_cast<cuuint64_t>(c.page_stride)};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(box_bytes), static_cast<cuuint32_t>(box_tokens), 1, 1};
    const cuuint32_t estr[4] = {1, 1, 1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<uint8_t*>(base), gdim, gstride, box, estr,
                  CU_TENSOR_MAP_INTERLEAVE_NONE,
                  !swizzle ? CU_TENSOR_MAP_SWIZZLE_NONE : box_bytes == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_128B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int launch_attn_rows(const AttnArgs& a, bool int8, cudaStream_t s) {
    return int8 ? launch_rows<true, false>(a, s) : launch_rows<false, false>(a, s);
}

}  // namespace qg
