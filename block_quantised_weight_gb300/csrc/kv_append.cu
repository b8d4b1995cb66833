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
// block's values wait in registers (up to 16 vectors of 16 bytes a thread;
// larger blocks are read a second time).  int8's quotient is formed as a
// product, whose error is below 2^-16 of a code: only quotients that close to
// a tie (or not finite) take the division, one in 2^14.  Measured: 5 prompts of
// up to 4001 rows, 14801 in all, 8 heads of 128, bf16: int8 28.7 us (3.2 TB/s),
// e4m3 21.7 us; int8 by 18 instructions a value (256 threads a CTA: 29.7 us),
// both by one chain a CTA (lengths, values, maximum, codes) with nothing of
// its next block on the way.  48 single tokens: 2.4 us.
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

// Four codes of int8 by division: out of line, the way there is rare.
__device__ __noinline__ uint32_t codes_by_division(float x0, float x1, float x2, float x3, float scale) {
    const float x[4] = {x0, x1, x2, x3};
    uint32_t r = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const bool finite = fabsf(x[i]) <= 3.4028235e38f;
        r |= code_of<true>(scale == 0.f ? (finite ? 0.f : x[i]) : __fdiv_rn(x[i], scale)) << (8 * i);
    }
    return r;
}

// Codes of four values.  inv: 1 / scale rounded (for e4m3 a power of two,
// exact), 0 for a zero block.
template <bool INT8>
__device__ __forceinline__ uint32_t codes_of(float x0, float x1, float x2, float x3, float scale, float inv) {
    if (!INT8) {
        if (scale == 0.f) inv = 1.f;  // zeros stay zeros, infinities and NaN keep their codes
        unsigned short lo, hi;
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(lo) : "f"(x1 * inv), "f"(x0 * inv));
        asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(hi) : "f"(x3 * inv), "f"(x2 * inv));
        return lo | static_cast<uint32_t>(hi) << 16;
    }
    const float x[4] = {x0, x1, x2, x3};
    uint32_t z[4];
    bool sure = true;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float y = x[i] * inv;
        const float big = y + 12582912.f;  // 1.5 * 2^23: the sum's low bits are y rounded to an integer
        z[i] = __float_as_uint(big);
        // further than 2^-15 from a tie; false for NaN and infinities
        sure &= fabsf(fabsf(y - (big - 12582912.f)) - 0.5f) > 0x1p-15f;
    }
    if (!sure) return codes_by_division(x0, x1, x2, x3, scale);
    return prmt(prmt(z[0], z[1], 0x0040u), prmt(z[2], z[3], 0x0040u), 0x5410u);
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

// The running largest magnitude of pairs of 16-bit values; NaN is passed over.
template <class T>
struct Pair {
    __device__ void take(uint32_t) {}
    __device__ float largest() const { return 0.f; }
};
template <>
struct Pair<__half> {
    __half2 m = __floats2half2_rn(0.f, 0.f);
    __device__ void take(uint32_t two) {
        two &= 0x7FFF7FFFu;
        m = __hmax2(m, *reinterpret_cast<__half2*>(&two));
    }
    __device__ float largest() const { return fmaxf(__low2float(m), __high2float(m)); }
};
template <>
struct Pair<__nv_bfloat16> {
    __nv_bfloat162 m = __floats2bfloat162_rn(0.f, 0.f);
    __device__ void take(uint32_t two) {
        two &= 0x7FFF7FFFu;
        m = __hmax2(m, *reinterpret_cast<__nv_bfloat162*>(&two));
    }
    __device__ float largest() const { return fmaxf(__low2float(m), __high2float(m)); }
};

// NV: vectors of 16 bytes that a thread holds, 0 to read the values twice.
template <class T, bool INT8, int THREADS, int NV>
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
    const int off = block == 0 ? static_cast<int>(len & (page_tokens - 1)) : 0;  // tokens the block holds
    const int64_t row = r0 + (block == 0 ? 0 : (page_at << c.log2p) - len);
    const int n = static_cast<int>(min(static_cast<int64_t>(page_tokens - off), r1 - row));

    const T* src = static_cast<const T*>(blockIdx.z ? a.v : a.k) + row * a.row_stride + h * a.head_stride;
    const int per = c.dim / V;  // vectors of a token

    // ---- the values, on their way while the page is looked up
    const int vecs = n * per;
    // vector tid of the block and the step to tid + THREADS
    const int tok_first = tid / per, vec_first = tid - tok_first * per;
    const int tok_step = THREADS / per, vec_step = THREADS - tok_step * per;
    uint4 held[NV > 0 ? NV : 1];
    if (NV > 0) {
        int tok = tok_first, vec = vec_first;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            held[i] = make_uint4(0, 0, 0, 0);
            if (tid + i * THREADS < vecs) held[i] = ldg_stream16(src + tok * a.row_stride + vec * V);
            tok += tok_step, vec += vec_step;
            if (vec >= per) vec -= per, ++tok;
        }
    }
    const int64_t page = a.table[b * a.width + page_at];
    if (page < 0 || page >= c.pages) {
        if (tid == 0) atomicOr(a.status, kStatusBounds);
        return;
    }
    uint8_t* dst = (blockIdx.z ? c.v : c.k) + page * c.page_stride + static_cast<int64_t>(h) * c.head_stride;
    float* scale_at = (blockIdx.z ? c.vs : c.ks) + page * c.heads + h;
    const float old = off > 0 ? *scale_at : 0.f;

    // ---- largest finite magnitude
    float amax = 0.f;
    auto each = [&](auto f) {  // every vector of this thread
        if (NV > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) f(held[i]);  // those past the last are 0
        } else {
            int tok = tok_first, vec = vec_first;
            for (int i = tid; i < vecs; i += THREADS) {
                f(*reinterpret_cast<const uint4*>(src + tok * a.row_stride + vec * V));
                tok += tok_step, vec += vec_step;
                if (vec >= per) vec -= per, ++tok;
            }
        }
    };
    auto largest_finite = [&](const uint4& v) {
        const T* e = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int j = 0; j < V; ++j) {
            const float y = fabsf(to_f32(e[j]));
            if (y <= 3.4028235e38f) amax = fmaxf(amax, y);
        }
    };
    if (sizeof(T) == 4) {
        each(largest_finite);
    } else {
        // two values an instruction; NaN is passed over, an infinity sends the thread back
        Pair<T> m;
        each([&](const uint4& v) { m.take(v.x), m.take(v.y), m.take(v.z), m.take(v.w); });
        amax = m.largest();
        if (amax == INFINITY) {
            amax = 0.f;
            each(largest_finite);
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
    const float inv = scale == 0.f ? 0.f : __fdiv_rn(1.f, scale);
    auto write = [&](const uint4& v, int tok, int vec) {
        const T* e = reinterpret_cast<const T*>(&v);
        float x[V];
#pragma unroll
        for (int j = 0; j < V; ++j) x[j] = to_f32(e[j]);
        uint32_t w[V / 4];
#pragma unroll
        for (int j = 0; j < V / 4; ++j)
            w[j] = codes_of<INT8>(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3], scale, inv);
        uint8_t* p = dst + static_cast<int64_t>(off + tok) * c.token_stride + vec * V;
        if (V == 4) *reinterpret_cast<uint32_t*>(p) = w[0];
        else *reinterpret_cast<uint2*>(p) = make_uint2(w[0], w[V / 4 - 1]);
    };
    int tok = tok_first, vec = vec_first;
    if (NV > 0) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (tid + i * THREADS < vecs) write(held[i], tok, vec);
            tok += tok_step, vec += vec_step;
            if (vec >= per) vec -= per, ++tok;
        }
    } else {
        for (int i = tid; i < vecs; i += THREADS) {
            write(*reinterpret_cast<const uint4*>(src + tok * a.row_stride + vec * V), tok, vec);
            tok += tok_step, vec += vec_step;
            if (vec >= per) vec -= per, ++tok;
        }
    }
}

template <class T, bool INT8>
void launch_typed(const AppendArgs& a, int64_t units, cudaStream_t s) {
    const dim3 grid(static_cast<unsigned>(units), a.c.heads, 2);
    if (!a.starts) {  // one token: at most 64 vectors
        qg_append_kernel<T, INT8, 32, 2><<<grid, 32, 0, s>>>(a);
        return;
    }
    // vectors of a whole block over 128 threads
    const int need = ((1 << a.c.log2p) * a.c.dim * static_cast<int>(sizeof(T)) / 16 + 127) / 128;
    if (need <= 2) qg_append_kernel<T, INT8, 128, 2><<<grid, 128, 0, s>>>(a);
    else if (need <= 4) qg_append_kernel<T, INT8, 128, 4><<<grid, 128, 0, s>>>(a);
    else if (need <= 8) qg_append_kernel<T, INT8, 128, 8><<<grid, 128, 0, s>>>(a);
    else if (need <= 16) qg_append_kernel<T, INT8, 128, 16><<<grid, 128, 0, s>>>(a);
    else qg_append_kernel<T, INT8, 128, 0><<<grid, 128, 0, s>>>(a);
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
