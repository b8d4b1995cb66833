// Turn new keys and queries to their positions, and quantise the keys and
// values into the 8-bit paged cache in the same pass.
//
// Mathematics (qgkv.h, qgkv_append_rotary).  The pair (a, b) number i of a head
// at position p becomes (a c - b s, a s + b c), c and s the i-th cosine and sine
// of row p of the table; products and sums are rounded to fp32 one by one.  Keys
// go on as in qgkv_append: the block's largest magnitude after the turn, its
// scale, codes.  Queries are rounded once to their type.
//
// Bound.  Reads q, k, v once, writes q and the codes: HBM for prompts, one
// dependency chain (lengths -> position -> cosines -> maximum -> code) for single
// tokens.  A thread's item is the two 16-byte vectors of one token that are
// turned into one another (neighbouring pairs: two adjacent vectors; halves: two
// half the turned dims apart), so that it needs one run of cosines and one of
// sines.  A CTA takes a block (the tokens of a page) of one head of K or V, whose
// turned values wait in registers for the block's scale; or the block's rows of
// several query heads, cosines and sines read once for them.
//
// Measured (GB300; bytes at the copy rate in brackets): 5 prompts of up to 4001 rows, 32 / 8
// heads of 128, bf16, 62 us (50), fp32 104; 48 single tokens 2.7 us, launch and chain.
// Five CTAs of 128 threads an SM (102 registers): with four the prompts took 63
// to 69 us, six spill into the L1 (74).  Loads of 4 heads on their way: 2 took 76 us, 8 72.
#include "kv_quant.cuh"
#include "launch_common.cuh"
#include "qgkv_launch.h"

namespace qg {
namespace {

struct RotaryArgs {
    KVLayer c;
    const void* q;
    const void* k;
    const void* v;
    void* out;
    int64_t q_row, q_head, kv_row, kv_head;
    int q_heads, q_chunk, q_chunks;  // query heads of a CTA, CTAs that they take
    const float* rope;
    int64_t positions;
    int turned;
    bool halves;
    const int32_t* table;
    int64_t width;
    const int32_t* lens;
    const int32_t* starts;
    int batch;
    int64_t rows;
    unsigned* status;
};

// The two vectors of item p of a token: their first dims, and the first pair that they hold (-1: not turned).
template <int V>
struct Item {
    int d0, d1, pair;
    __device__ Item(const RotaryArgs& a, int p, bool turn) {
        d0 = 2 * p * V, d1 = d0 + V, pair = -1;
        if (turn && d0 < a.turned) {
            pair = p * V;
            if (a.halves) d0 = pair, d1 = pair + a.turned / 2;
        }
    }
};

template <class T, int V>
__device__ __forceinline__ void to_values(const uint4& raw, float (&x)[V]) {
    const T* e = reinterpret_cast<const T*>(&raw);
#pragma unroll
    for (int j = 0; j < V; ++j) x[j] = to_f32(e[j]);
}

// V pairs turned.  halves: pair j is (x0[j], x1[j]); else pairs are neighbours in x0, then x1.
template <int V>
__device__ __forceinline__ void turn(float (&x0)[V], float (&x1)[V], const float (&c)[V], const float (&s)[V], bool halves) {
    auto one = [](float& a, float& b, float c, float s) {
        const float lo = __fsub_rn(__fmul_rn(a, c), __fmul_rn(b, s));
        const float hi = __fadd_rn(__fmul_rn(a, s), __fmul_rn(b, c));
        a = lo, b = hi;
    };
    if (halves) {
#pragma unroll
        for (int j = 0; j < V; ++j) one(x0[j], x1[j], c[j], s[j]);
    } else {
#pragma unroll
        for (int j = 0; j < V / 2; ++j) one(x0[2 * j], x0[2 * j + 1], c[j], s[j]);
#pragma unroll
        for (int j = 0; j < V / 2; ++j) one(x1[2 * j], x1[2 * j + 1], c[V / 2 + j], s[V / 2 + j]);
    }
}

template <int V>
__device__ __forceinline__ void load_angles(const RotaryArgs& a, int64_t pos, int pair, float (&c)[V], float (&s)[V]) {
    const float* row = a.rope + pos * a.turned + pair;
#pragma unroll
    for (int j = 0; j < V; j += 4) {
        const float4 x = __ldg(reinterpret_cast<const float4*>(row + j));
        const float4 y = __ldg(reinterpret_cast<const float4*>(row + a.turned / 2 + j));
        c[j] = x.x, c[j + 1] = x.y, c[j + 2] = x.z, c[j + 3] = x.w;
        s[j] = y.x, s[j + 1] = y.y, s[j + 2] = y.z, s[j + 3] = y.w;
    }
}

template <class T, int V>
__device__ __forceinline__ uint4 to_raw(const float (&x)[V]) {
    uint4 r;
    uint32_t* w = reinterpret_cast<uint32_t*>(&r);
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = __float_as_uint(x[j]);
    } else if constexpr (std::is_same<T, __half>::value) {
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = pack_f16x2(x[2 * j], x[2 * j + 1]);
    } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[j]) : "f"(x[2 * j + 1]), "f"(x[2 * j]));
    }
    return r;
}

// ITEMS: items that a thread holds, 0 to read and turn the values twice.
template <class T, bool INT8, int THREADS, int ITEMS>
__global__ void __launch_bounds__(THREADS, THREADS == 128 ? 5 : 1) qg_append_rotary_kernel(const RotaryArgs a) {
    constexpr int V = 16 / sizeof(T);
    __shared__ int found[2];
    __shared__ float red[THREADS / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const KVLayer& c = a.c;
    const int page_tokens = 1 << c.log2p;

    // ---- which sequence and which of its blocks
    int b, block = 0;  // block counted from the first that the new tokens touch
    if (!a.starts) {
        b = blockIdx.x;
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
    const int64_t len = max(a.lens[b], 0);
    if (a.lens[b] < 0 || r0 < 0 || r1 > a.rows) {
        if (tid == 0) atomicOr(a.status, kStatusBounds);
        if (r0 < 0 || r1 > a.rows) return;
    }
    const int64_t page_at = (len >> c.log2p) + block;
    const int off = block == 0 ? static_cast<int>(len & (page_tokens - 1)) : 0;  // tokens the block holds
    const int64_t row = r0 + (block == 0 ? 0 : (page_at << c.log2p) - len);
    const int64_t pos = (page_at << c.log2p) + off;
    const int n = static_cast<int>(min(static_cast<int64_t>(page_tokens - off), r1 - row));
    // tokens whose position the table has
    const int known = a.lens[b] < 0 ? 0 : static_cast<int>(max(int64_t(0), min(static_cast<int64_t>(n), a.positions - pos)));
    const int items = c.dim / (2 * V);  // of a token

    // ---- queries
    if (static_cast<int>(blockIdx.y) < a.q_chunks) {
        if (known < n && tid == 0) atomicOr(a.status, kStatusBounds);
        // Threads over items, then tokens, then (few tokens) heads; a thread
        // keeps its cosines and sines for its heads.
        const int slots = THREADS / items;
        const int slot = tid / items, p = tid - slot * items;
        if (slot >= slots) return;
        const int h_end = min(a.q_heads, static_cast<int>(blockIdx.y + 1) * a.q_chunk);
        const int apart = max(1, slots / n);      // heads that threads take side by side
        const int side = n < slots ? slot / n : 0;
        if (side >= apart) return;
        const Item<V> it(a, p, true);
        for (int t = n < slots ? slot - side * n : slot; t < n; t += slots) {
            float cs[V], sn[V];
            const bool there = t < known;
            if (there && it.pair >= 0) load_angles<V>(a, pos + t, it.pair, cs, sn);
            const T* src = static_cast<const T*>(a.q) + (row + t) * a.q_row;
            T* dst = static_cast<T*>(a.out) + (row + t) * a.q_heads * c.dim;
            constexpr int N = 4;  // heads on their way at once
            for (int h0 = blockIdx.y * a.q_chunk + side; h0 < h_end; h0 += N * apart) {
                uint4 u0[N], u1[N];
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int h = h0 + i * apart;
                    if (h < h_end) {
                        // not through the read-only path: out may be q itself
                        u0[i] = __ldcs(reinterpret_cast<const uint4*>(src + h * a.q_head + it.d0));
                        u1[i] = __ldcs(reinterpret_cast<const uint4*>(src + h * a.q_head + it.d1));
                    }
                }
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const int h = h0 + i * apart;
                    if (h < h_end) {
                        if (it.pair >= 0) {
                            float x0[V], x1[V];
                            to_values<T>(u0[i], x0);
                            to_values<T>(u1[i], x1);
                            if (there) {
                                turn<V>(x0, x1, cs, sn, a.halves);
                            } else {
#pragma unroll
                                for (int j = 0; j < V; ++j) x0[j] = x1[j] = __int_as_float(0x7FC00000);
                            }
                            u0[i] = to_raw<T>(x0), u1[i] = to_raw<T>(x1);
                        }
                        *reinterpret_cast<uint4*>(dst + h * c.dim + it.d0) = u0[i];
                        *reinterpret_cast<uint4*>(dst + h * c.dim + it.d1) = u1[i];
                    }
                }
            }
        }
        return;
    }

    // ---- keys and values
    if (known <= 0 || page_at >= a.width) {
        if (tid == 0) atomicOr(a.status, kStatusBounds);
        return;
    }
    if (known < n && tid == 0) atomicOr(a.status, kStatusBounds);
    const int hv = static_cast<int>(blockIdx.y) - a.q_chunks;
    const bool values = hv >= c.heads;
    const int h = values ? hv - c.heads : hv;
    const T* src = static_cast<const T*>(values ? a.v : a.k) + row * a.kv_row + h * a.kv_head;
    const int total = known * items;
    const int tok_first = tid / items, p_first = tid - tok_first * items;
    const int tok_step = THREADS / items, p_step = THREADS - tok_step * items;
    float amax = 0.f;
    auto largest = [&](const float (&x)[V]) {
#pragma unroll
        for (int j = 0; j < V; ++j) amax = fmaxf(amax, fabsf(x[j]));  // NaN is passed over
    };
    auto largest_finite = [&](const float (&x)[V]) {
#pragma unroll
        for (int j = 0; j < V; ++j)
            if (fabsf(x[j]) <= 3.4028235e38f) amax = fmaxf(amax, fabsf(x[j]));
    };
    auto turned_item = [&](const uint4& u0, const uint4& u1, int tok, const Item<V>& it, float (&x0)[V], float (&x1)[V]) {
        to_values<T>(u0, x0);
        to_values<T>(u1, x1);
        if (it.pair >= 0) {
            float cs[V], sn[V];
            load_angles<V>(a, pos + tok, it.pair, cs, sn);
            turn<V>(x0, x1, cs, sn, a.halves);
        }
    };
    auto read_item = [&](int tok, int p, float (&x0)[V], float (&x1)[V]) {
        const Item<V> it(a, p, !values);
        turned_item(ldg_stream16(src + tok * a.kv_row + it.d0), ldg_stream16(src + tok * a.kv_row + it.d1), tok, it, x0, x1);
    };
    float x0[ITEMS > 0 ? ITEMS : 1][V], x1[ITEMS > 0 ? ITEMS : 1][V];
    if (ITEMS > 0) {
        uint4 u0[ITEMS > 0 ? ITEMS : 1], u1[ITEMS > 0 ? ITEMS : 1];
        int tok = tok_first, p = p_first;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            u0[i] = u1[i] = make_uint4(0, 0, 0, 0);
            if (tid + i * THREADS < total) {
                const Item<V> it(a, p, !values);
                u0[i] = ldg_stream16(src + tok * a.kv_row + it.d0);
                u1[i] = ldg_stream16(src + tok * a.kv_row + it.d1);
            }
            tok += tok_step, p += p_step;
            if (p >= items) p -= items, ++tok;
        }
        tok = tok_first, p = p_first;
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (tid + i * THREADS < total) {
                turned_item(u0[i], u1[i], tok, Item<V>(a, p, !values), x0[i], x1[i]);
                largest(x0[i]);
                largest(x1[i]);
            }
            tok += tok_step, p += p_step;
            if (p >= items) p -= items, ++tok;
        }
    } else {
        int tok = tok_first, p = p_first;
        for (int i = tid; i < total; i += THREADS) {
            read_item(tok, p, x0[0], x1[0]);
            largest(x0[0]);
            largest(x1[0]);
            tok += tok_step, p += p_step;
            if (p >= items) p -= items, ++tok;
        }
    }
    if (amax == INFINITY) {  // once more without the infinities
        amax = 0.f;
        if (ITEMS > 0) {
#pragma unroll
            for (int i = 0; i < ITEMS; ++i)
                if (tid + i * THREADS < total) {
                    largest_finite(x0[i]);
                    largest_finite(x1[i]);
                }
        } else {
            int tok = tok_first, p = p_first;
            for (int i = tid; i < total; i += THREADS) {
                read_item(tok, p, x0[0], x1[0]);
                largest_finite(x0[0]);
                largest_finite(x1[0]);
                tok += tok_step, p += p_step;
                if (p >= items) p -= items, ++tok;
            }
        }
    }
    const int64_t page = a.table[b * a.width + page_at];
    if (page < 0 || page >= c.pages) {  // the same in all threads
        if (tid == 0) atomicOr(a.status, kStatusBounds);
        return;
    }
    uint8_t* dst = (values ? c.v : c.k) + page * c.page_stride + static_cast<int64_t>(h) * c.head_stride;
    float* scale_at = (values ? c.vs : c.ks) + page * c.heads + h;
    const float old = off > 0 ? *scale_at : 0.f;
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
            uint32_t* w = reinterpret_cast<uint32_t*>(dst + static_cast<int64_t>(tok) * c.token_stride) + (i - tok * words);
            *w = rescaled<INT8>(*w, f);
        }
    }
    if (THREADS == 32) __syncwarp();  // every thread has read the old scale (more threads: before the barrier above)
    if (tid == 0) *scale_at = scale;

    // ---- new codes
    const float inv = scale == 0.f ? 0.f : __fdiv_rn(1.f, scale);
    auto write = [&](const float (&x)[V], int tok, int d) {
        uint32_t w[V / 4];
#pragma unroll
        for (int j = 0; j < V / 4; ++j)
            w[j] = codes_of<INT8>(x[4 * j], x[4 * j + 1], x[4 * j + 2], x[4 * j + 3], scale, inv);
        uint8_t* at = dst + static_cast<int64_t>(off + tok) * c.token_stride + d;
        if (V == 4) *reinterpret_cast<uint32_t*>(at) = w[0];
        else *reinterpret_cast<uint2*>(at) = make_uint2(w[0], w[V / 4 - 1]);
    };
    int tok = tok_first, p = p_first;
    if (ITEMS > 0) {
#pragma unroll
        for (int i = 0; i < ITEMS; ++i) {
            if (tid + i * THREADS < total) {
                const Item<V> it(a, p, !values);
                write(x0[i], tok, it.d0);
                write(x1[i], tok, it.d1);
            }
            tok += tok_step, p += p_step;
            if (p >= items) p -= items, ++tok;
        }
    } else {
        for (int i = tid; i < total; i += THREADS) {
            const Item<V> it(a, p, !values);
            read_item(tok, p, x0[0], x1[0]);
            write(x0[0], tok, it.d0);
            write(x1[0], tok, it.d1);
            tok += tok_step, p += p_step;
            if (p >= items) p -= items, ++tok;
        }
    }
}

template <class T, bool INT8>
void launch_typed(RotaryArgs a, int64_t units, cudaStream_t s) {
    // A CTA's query heads, for which each block's angles are read once: sixteen, fewer where that leaves SMs idle.
    // 16 / 8 / 4 / 2 heads a CTA, us: 5 prompts of up to 4001 rows, 32 heads of 128, bf16: 61.6 / 64.8 / 66.6 / 74.4;
    // 400 single tokens, 32 heads of 64, fp32: 5.5 / 5.6 / 6.3 / 8.0; 8 chunks of up to 300 rows, 12 heads of 96, fp16:
    // 11.1 / 8.7 / 6.7 / 8.4; 7 of up to 131 rows: 9.3 / 7.1 / 5.2 / 5.1.
    a.q_chunk = 16;
    const int64_t busy = sm_count(current_device());
    while (a.q_chunk > 2 && units * ((a.q_heads + a.q_chunk - 1) / a.q_chunk) < busy) a.q_chunk /= 2;
    a.q_chunks = a.q ? (a.q_heads + a.q_chunk - 1) / a.q_chunk : 0;
    const dim3 grid(static_cast<unsigned>(units), a.q_chunks + 2 * a.c.heads);
    constexpr int held = 64 / (2 * (16 / sizeof(T)));  // items whose values take 64 registers
    const int values = (1 << a.c.log2p) * a.c.dim;     // of a block
    if (!a.starts) qg_append_rotary_kernel<T, INT8, 32, 1><<<grid, 32, 0, s>>>(a);  // one token: at most 32 items
    else if (values <= 64 * 128) qg_append_rotary_kernel<T, INT8, 128, held><<<grid, 128, 0, s>>>(a);
    else if (values <= 64 * 256) qg_append_rotary_kernel<T, INT8, 256, held><<<grid, 256, 0, s>>>(a);
    else qg_append_rotary_kernel<T, INT8, 256, 0><<<grid, 256, 0, s>>>(a);
}

}  // namespace

int launch_append_rotary(const qgkv_cache& c, int64_t layer, const void* q, const void* k, const void* v, int type,
                         int64_t rows, int q_heads, int64_t q_row, int64_t q_head, int64_t kv_row, int64_t kv_head,
                         const float* rope, int64_t positions, int turned, int pairs, void* out, const int32_t* table,
                         int64_t width, const int32_t* lens, const int32_t* starts, int batch, unsigned* status,
                         cudaStream_t s) {
    RotaryArgs a = {};
    a.c = layer_of(c, layer);
    a.q = q, a.k = k, a.v = v, a.out = out;
    a.q_heads = q_heads, a.q_row = q_row, a.q_head = q_head, a.kv_row = kv_row, a.kv_head = kv_head;
    a.rope = rope, a.positions = positions, a.turned = turned, a.halves = pairs == QGKV_HALVES;
    a.table = table, a.width = width, a.lens = lens, a.starts = starts, a.batch = batch, a.rows = rows;
    a.status = status;
    // a sequence of n rows touches at most (n - 1) / page + 2 blocks
    const int64_t units = starts ? rows / c.page_tokens + 2 * static_cast<int64_t>(batch) : batch;
    const bool i8 = c.format == QGKV_INT8;
    if (type == QGKV_F32) i8 ? launch_typed<float, true>(a, units, s) : launch_typed<float, false>(a, units, s);
    else if (type == QGKV_F16) i8 ? launch_typed<__half, true>(a, units, s) : launch_typed<__half, false>(a, units, s);
    else i8 ? launch_typed<__nv_bfloat16, true>(a, units, s) : launch_typed<__nv_bfloat16, false>(a, units, s);
    return launch_status();
}

}  // namespace qg
