// Arguments and launchers of the attention over the 8-bit paged cache.
#pragma once
#include "kv_common.cuh"

namespace qg {

struct AttnArgs {
    KVLayer c;
    const void* q;
    void* out;
    float* lse;
    int64_t q_row, q_head;  // elements
    int type, q_heads, group;
    const int32_t* table;
    int64_t width;
    const int32_t* lens;
    const int32_t* starts;
    int batch;
    int64_t rows;
    float scale_log2;  // softmax scale * log2(e)
    float* part;
    unsigned* count;
    unsigned* status;
};

// Rows start, number of rows and length of sequence b.  A length beyond the
// table is cut to it (kStatusBounds).
struct Seq {
    int64_t row0;
    int n;
    int len;
};
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b) {
    Seq s;
    s.row0 = b;
    s.n = 1;
    if (a.starts) {
        const int64_t r0 = a.starts[b], r1 = a.starts[b + 1];
        s.row0 = r0;
        s.n = static_cast<int>(r1 - r0);
        if (r0 < 0 || r1 < r0 || r1 > a.rows) {
            atomicOr(a.status, kStatusBounds);
            s.n = 0;
        }
    }
    s.len = a.lens[b];
    const int64_t most = a.width << a.c.log2p;
    if (s.len < 0 || s.len > most) {
        atomicOr(a.status, kStatusBounds);
        s.len = s.len < 0 ? 0 : static_cast<int>(most);
    }
    return s;
}

__device__ __forceinline__ void store_out(void* out, int type, int64_t at, float x) {
    if (type == QGKV_F32) static_cast<float*>(out)[at] = x;
    else if (type == QGKV_F16) static_cast<__half*>(out)[at] = __float2half_rn(x);
    else static_cast<__nv_bfloat16*>(out)[at] = __float2bfloat16_rn(x);
}

// 16 consecutive query values.
__device__ __forceinline__ void load_q16(const void* q, int type, int64_t at, float (&x)[16]) {
    if (type == QGKV_F32) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(q) + at);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float4 v = p[i];
            x[4 * i] = v.x, x[4 * i + 1] = v.y, x[4 * i + 2] = v.z, x[4 * i + 3] = v.w;
        }
    } else {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(q) + at);
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint4 v = p[i];
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (type == QGKV_F16) {
                    const f2 f = h2_to_f2(w[j]);
                    x[8 * i + 2 * j] = f.x, x[8 * i + 2 * j + 1] = f.y;
                } else {
                    x[8 * i + 2 * j] = __uint_as_float(w[j] << 16);
                    x[8 * i + 2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
                }
            }
        }
    }
}

int launch_attn_rows(const AttnArgs& a, bool int8, cudaStream_t s);
int launch_attn_prompt(const AttnArgs& a, bool int8, cudaStream_t s);

}  // namespace qg
