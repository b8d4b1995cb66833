// Shared by the kernels of qgkv.h: workspace layout, cache addressing, the
// exact conversions of 8-bit codes, warp matrix products.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "../../include/qgkv.h"
#include "common.cuh"

namespace qg {

// Device status bit next to common.cuh's.
constexpr unsigned kStatusPages = 4u;

// 4D tiled TMA load; x innermost, x * element size a multiple of 16.
__device__ __forceinline__ void tma_load_4d(void* dst, const CUtensorMap* map, int x, int y, int z, int w,
                                            uint64_t* bar) {
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
        " [%0], [%1, {%2, %3, %4, %5}], [%6];"
        ::"r"(smem_u32(dst)), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_u32(bar))
        : "memory");
}

// ------------------------------------------------------------- workspace
// Counters and kWsDelta are zero between calls (each call that uses them puts
// the zeros back); the rest holds values only within a call, so the page
// operations' lists and the others' partial results share it.
constexpr int64_t kWsCounters = 0;                               // 16384 words
constexpr int64_t kWsDelta = kWsCounters + 16384 * 4;            // per page: change of its count
constexpr int64_t kWsShared = kWsDelta + int64_t(QGKV_MAX_PAGES) * 4;
constexpr int64_t kWsRefs = kWsShared;
constexpr int64_t kWsHoles = kWsRefs + int64_t(QGKV_MAX_PAGES) * 4;
constexpr int64_t kWsMovers = kWsHoles + int64_t(QGKV_MAX_PAGES) * 4;
constexpr int64_t kWsRank = kWsMovers + int64_t(QGKV_MAX_PAGES) * 4;
constexpr int64_t kWsChunks = kWsRank + int64_t(QGKV_MAX_PAGES) * 4;  // 4096 words
constexpr int64_t kWsScalars = kWsChunks + 4096 * 4;                  // 256 words
constexpr int64_t kWsPart = kWsShared;                                // partial results
constexpr int64_t kWsPartBytes = int64_t(320) * 256 * 130 * 4;        // 320 of 256 rows x 128 dims, references and sums
constexpr int64_t kWsSplits = kWsPart + kWsPartBytes;                 // prompts whose keys are split: [160] x 32 bytes
constexpr int64_t kWsTotal = kWsSplits + 160 * 32;
static_assert(kWsScalars + 256 * 4 <= kWsTotal, "lists exceed the shared part");

// Counter words by user.
constexpr int kCntAttn = 0;      // [kMaxAttnCtas]
constexpr int kCntPrompt = 4096; // [2] (from the attention's counters)
constexpr int kCntPages = 8192;  // [1]
constexpr int kCntBeam = 8320;   // [QGKV_MAX_BATCH]

// ------------------------------------------------------------- values
__device__ __forceinline__ float to_f32(float x) { return x; }
__device__ __forceinline__ float to_f32(__half x) { return __half2float(x); }
__device__ __forceinline__ float to_f32(__nv_bfloat16 x) { return __bfloat162float(x); }

// Two e4m3 codes -> f16x2 (exact: e4m3's range and precision lie inside f16's).
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t two) {
    uint32_t r;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<unsigned short>(two)));
    return r;
}

__device__ __forceinline__ uint32_t hsub2_1152(uint32_t a) {
    uint32_t r;
    asm("sub.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(0x64806480u));
    return r;
}

// Four codes of one token (a 32-bit word) as two f16x2 operands, for a product
// with q.  e4m3: bytes (0, 1) and (2, 3), exact.  int8: bytes (0, 2) and
// (1, 3), exact: 0x6400 | (code + 128) is the f16 1152 + code.  (As subnormals
// (code + 128) * 2^-24 they cost one operation less, but 128 * sum(q) then rides
// on the fp32 sums and takes their last bits: scores 5 to 10 times less exact.)
template <bool INT8>
__device__ __forceinline__ void k_codes(uint32_t x, uint32_t& a, uint32_t& b) {
    if (INT8) {
        a = hsub2_1152((x & 0x00FF00FFu) ^ 0x64806480u);
        b = hsub2_1152(((x >> 8) & 0x00FF00FFu) ^ 0x64806480u);
    } else {
        a = e4m3x2_f16x2(x & 0xFFFFu);
        b = e4m3x2_f16x2(x >> 16);
    }
}

// Words of two tokens -> four operands (token 0, token 1), one for each byte,
// exact.  int8: 0x6400 | (code + 128) is the f16 1152 + code.
template <bool INT8>
__device__ __forceinline__ void v_codes(uint32_t t0, uint32_t t1, uint32_t (&r)[4]) {
    if (INT8) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t p = prmt(t0, t1, i ? 0x7632u : 0x5410u);
            r[2 * i] = hsub2_1152((p & 0x00FF00FFu) ^ 0x64806480u);
            r[2 * i + 1] = hsub2_1152(((p >> 8) & 0x00FF00FFu) ^ 0x64806480u);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const uint32_t p = prmt(t0, t1, i ? 0x7362u : 0x5140u);
            r[2 * i] = e4m3x2_f16x2(p & 0xFFFFu);
            r[2 * i + 1] = e4m3x2_f16x2(p >> 16);
        }
    }
}

// (hi, lo) f32 pair -> f16x2 with `lo` in the low half, round to nearest.
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// x = part 1 + part 2 with both f16: what the first rounding left over.
__device__ __forceinline__ uint32_t rest_f16x2(float lo, float hi, uint32_t first) {
    const f2 f = h2_to_f2(first);
    return pack_f16x2(lo - f.x, hi - f.y);
}

// D += A (16 x 16, row) * B (16 x 8, col), f16 in, f32 out.
__device__ __forceinline__ void mma16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// Transpose of an 8 x 8 matrix of 16-bit values held as a fragment.
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
    return r;
}

__device__ __forceinline__ float exp2_fast(float x) {
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// 16-byte load of data read once.
__device__ __forceinline__ uint4 ldg_stream16(const void* p) {
    uint4 r;
    asm volatile("ld.global.nc.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p));
    return r;
}
__device__ __forceinline__ uint2 ldg_stream8(const void* p) {
    uint2 r;
    asm volatile("ld.global.nc.L1::no_allocate.v2.u32 {%0,%1}, [%2];" : "=r"(r.x), "=r"(r.y) : "l"(p));
    return r;
}

// One layer of a cache as the kernels take it.
struct KVLayer {
    uint8_t* k;
    uint8_t* v;
    float* ks;
    float* vs;
    int64_t page_stride, pages;
    int head_stride, token_stride;
    int heads, dim, log2p;
};

inline int log2_of(int x) {
    int n = 0;
    while ((1 << n) < x) ++n;
    return n;
}

inline KVLayer layer_of(const qgkv_cache& c, int64_t layer) {
    KVLayer l = {};
    l.k = c.k + layer * c.layer_stride;
    l.v = c.v + layer * c.layer_stride;
    l.ks = c.k_scale + layer * c.pages * c.heads;
    l.vs = c.v_scale + layer * c.pages * c.heads;
    l.page_stride = c.page_stride;
    l.pages = c.pages;
    l.head_stride = c.order == QGKV_HND ? c.page_tokens * c.head_dim : c.head_dim;
    l.token_stride = c.order == QGKV_HND ? c.head_dim : c.heads * c.head_dim;
    l.heads = c.heads;
    l.dim = c.head_dim;
    l.log2p = log2_of(c.page_tokens);
    return l;
}

}  // namespace qg
