// Quantise new keys and values into the 8-bit paged cache.
//
// Mathematics (qgkv.h, qgkv_append): one scale for each block (the tokens of a
// page) and head; a block that already holds tokens keeps its scale or grows
// it, and then its codes are rescaled.  Every step is one correctly rounded
// fp32 operation, so the codes are a function of the inputs alone.
//
// Bound.  Reads the new values once and writes a quarter or half of their
// bytes; for one token a sequence it is a single short dependency chain
// (table -> scale -> codes).  One CTA takes one (block, head) of K or V: the
// largest magnitude needs the whole block before its first code, so the
// values are read twice, the second time from L1/L2.
#include "kv_common.cuh"
#include "launch_common.cuh"
#include "qgkv_launch.h"

namespace qg {
namespace {

struct AppendArgs {
    KVLayer c;
    const void* k;
    const void* v;
    int64_t row_stride, head_stride;
    const int32_t* table;
    int64_t width;
    const int32_t* lens;
    const int32_t* starts;
    int batch;
    int64_t rows;
    unsigned* status;
};

// 16 bytes of values -> fp32.
template <class T>
__device__ __forceinline__ void load_values(const T* p, float (&x)[16 / sizeof(T)]) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const T* e = reinterpret_cast<const T*>(&a);
#pragma unroll
    for (int i = 0; i < static_cast<int>(16 / sizeof(T)); ++i) x[i] = to_f32(e[i]);
}

// Code of y = x / scale.
template <bool INT8>
__device__ __forceinline__ uint32_t code_of(float y) {
    if (INT8) {
        if (!(y == y)) return 0u;
        return static_cast<uint32_t>(__float2int_rn(fminf(fmaxf(y, -127.f), 127.f))) & 0xFFu;
    }
    unsigned short r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(y));
    return r & 0xFFu;
}

template <bool INT8>
__device__ __forceinline__ float scale_for(float amax) {
    if (INT8) return __fdiv_rn(amax, 127.f);
    if (!(amax > 0.f)) return 0.f;
    // smallest e >= -126 with amax <= 1.75 * 2^(8 + e)
    const uint32_t u = __float_as_uint(amax);
    int e = static_cast<int>(u >> 23) - 127 - 8 + ((u & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    e = max(e, -126);
    return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

template <class T, bool INT8, int THREADS>
__global__ void __launch_bounds__(THREADS) qg_append_kernel(const AppendArgs a) {
    constexpr int V = 16 / sizeof(T);
    __shared__ int found[4];
    __shared__ float red[THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const KVLayer& c = a.c;
    const int h = blockIdx.y;
    const int page_tokens = 1 << c.log2p;

    // ---- which sequence and which of its blocks
    int b, block;  // block counted from the first that the new tokens touch
    if (!a.starts) {
        b = blockIdx.x;
        block = 0;
    } else {
        if (tid == 0) found[0] = -1;
        __syncthreads();
        int64_t base = 0;
        for (int b0 = 0; b0 < a.batch; b0 += 32) {
            // every warp scans the same 32 sequences; warp 0 records the hit
            const int bb = b0 + lane;
            int64_t n = 0;
            int len = 0;
            if (bb < a.batch) {
                n = static_cast<int64_t>(a.starts[bb + 1]) - a.starts[bb];
                len = max(a.lens[bb], 0);
            }
            const int64_t touched = n > 0 ? ((len + n - 1) >> c.log2p) - (len >> c.log2p) + 1 : 0;
            int64_t x = touched;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(~0u, x, o);
                if (lane >= o) x += y;
            }
            const int64_t mine = static_cast<int64_t>(blockIdx.x) - base;
            if (mine < x && mine >= x - touched && warp == 0) {
                found[0] = bb;
                found[1] = static_cast<int>(mine - (x - touched));
            }
            base += __shfl_sync(~0u, x, 31);
            if (base > blockIdx.x) break;
        }
        __syncthreads();
        if (found[0] < 0) return;
        b = found[0];
        block = found[1];
    }
    const int64_t r0 = a.starts ? a.starts[b] : b;
    const int64_t r1 = a.starts ? a.starts[b + 1] : b + 1;
    const int64_t len = a.lens[b];
    const int64_t page_at = (len >> c.log2p) + block;
    if (len < 0 || r0 < 0 || r1 > a.rows || page_at >= a.width) {
        if (tid == 0) atomicOr(a.status, kStatusBounds);
        return;
    }
    const int64_t page = a.table[b * a.width + page_at];
    if (page < 0 || page >= c.pages) {
        if (tid == 0) atomicOr(a.status, kStatusBounds);
        return;
    }
    const int off = block == 0 ? static_cast<int>(len & (page_tokens - 1)) : 0;  // tokens the block holds
    const int64_t row = r0 + (block == 0 ? 0 : (page_at << c.log2p) - len);
    const int n = static_cast<int>(min(static_cast<int64_t>(page_tokens - off), r1 - row));

    const T* src = static_cast<const T*>(blockIdx.z ? a.v : a.k) + row * a.row_stride + h * a.head_stride;
    uint8_t* dst = (blockIdx.z ? c.v : c.k) + page * c.page_stride + static_cast<int64_t>(h) * c.head_stride;
    float* scale_at = (blockIdx.z ? c.vs : c.ks) + page * c.heads + h;
    const int per = c.dim / V;  // vectors of a token

    // ---- largest finite magnitude
    const float old = off > 0 ? *scale_at : 0.f;
    float amax = 0.f;
    for (int i = tid; i < n * per; i += THREADS) {
        const int tok = i / per, d = (i - tok * per) * V;
        float x[V];
        load_values(src + tok * a.row_stride + d, x);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float y = fabsf(x[j]);
            if (y <= 3.4028235e38f) amax = fmaxf(amax, y);
        }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, o));
    if (THREADS > 32) {
        if (lane == 0) red[warp] = amax;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < THREADS / 32; ++w) amax = fmaxf(amax, red[w]);
    }
    const float scale = fmaxf(old, scale_for<INT8>(amax));

    // ---- codes held, where the scale grows
    if (scale > old && off > 0) {
        const float f = __fdiv_rn(old, scale);
        const int words = c.dim / 4;
        for (int i = tid; i < off * words; i += THREADS) {
            const int tok = i / words;
            uint32_t* p = reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(tok) * c.token_stride) + (i - tok * words);
            const uint32_t x = *p;
            uint32_t r = 0;
            if (INT8) {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    r |= code_of<true>(__fmul_rn(static_cast<float>(static_cast<signed char>(x >> (8 * j))), f))
                         << (8 * j);
            } else {
                const f2 lo = h2_to_f2(e4m3x2_f16x2(x & 0xFFFFu)), hi = h2_to_f2(e4m3x2_f16x2(x >> 16));
                r = code_of<false>(__fmul_rn(lo.x, f)) | code_of<false>(__fmul_rn(lo.y, f)) << 8 |
                    code_of<false>(__fmul_rn(hi.x, f)) << 16 | code_of<false>(__fmul_rn(hi.y, f)) << 24;
            }
            *p = r;
        }
    }
    if (tid == 0) *scale_at = scale;

    // ---- new codes
    const float inv = INT8 || scale == 0.f ? 0.f : __fdiv_rn(1.f, scale);  // e4m3: a power of two, exact
    for (int i = tid; i < n * per; i += THREADS) {
        const int tok = i / per, d = (i - tok * per) * V;
        float x[V];
        load_values(src + tok * a.row_stride + d, x);
        uint32_t w[V / 4];
#pragma unroll
        for (int j = 0; j < V / 4; ++j) {
            w[j] = 0;
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                // a zero block's codes are 0, NaN aside
                float y = x[4 * j + q];
                if (scale == 0.f) y = y == y && fabsf(y) <= 3.4028235e38f ? 0.f : y;
                else y = INT8 ? __fdiv_rn(y, scale) : __fmul_rn(y, inv);
                w[j] |= code_of<INT8>(y) << (8 * q);
            }
        }
        uint8_t* p = dst + static_cast<int64_t>(off + tok) * c.token_stride + d;
        if (V == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
        else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[V / 4 - 1]);
    }
}

template <class T, bool INT8>
void launch_typed(const AppendArgs& a, int64_t units, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(units), a.c.heads, 2);
    if (!a.starts) qg_append_kernel<T, INT8, 32><<<grid, 32, 0, s>>>(a);
    else qg_append_kernel<T, INT8, 128><<<grid, 128, 0, s>>>(a);
}

}  // namespace

int launch_append(const qgkv_cache& c, int64_t layer, const void* k, const void* v, int type, int64_t rows,
                  int64_t row_stride, int64_t head_stride, const int32_t* table, int64_t width, const int32_t* lens,
                  const int32_t* starts, int batch, unsigned* status, cudaStream_t s) {
    AppendArgs a = {};
    a.c = layer_of(c, layer);
    a.k = k, a.v = v, a.row_stride = row_stride, a.head_stride = head_stride;
    a.table = table, a.width = width, a.lens = lens, a.starts = starts, a.batch = batch, a.rows = rows;
    a.status = status;
    // a sequence of n rows touches at most (n - 1) / page + 2 blocks
    const int64_t units = starts ? rows / c.page_tokens + 2 * static_cast<int64_t>(batch) : batch;
    if (units <= 0) return QG_OK;
    const bool i8 = c.format == QGKV_INT8;
    if (type == QGKV_F32) i8 ? launch_typed<float, true>(a, units, s) : launch_typed<float, false>(a, units, s);
    else if (type == QGKV_F16) i8 ? launch_typed<__half, true>(a, units, s) : launch_typed<__half, false>(a, units, s);
    else i8 ? launch_typed<__nv_bfloat16, true>(a, units, s) : launch_typed<__nv_bfloat16, false>(a, units, s);
    return launch_status();
}

}  // namespace qg
