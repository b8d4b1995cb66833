// Adjustment of logits before a selection: penalties for tokens that have come
// before, listed biases, temperature, a grammar's mask.
//
// Mathematics: qgkv.h, qglogits_adjust; each operation is rounded to fp32 by
// itself, so the result is a function of the inputs alone.
//
// Bound.  Every logit is read and written once: HBM for batches.  Few tokens of a
// row have come before or have a bias, so a CTA takes a span of the row's
// vocabulary in two parts.  It gathers those tokens of its span from the whole
// history and list of the row, in a table in shared memory with a word a token (how
// often it came, which bias is its last), lists each once, and works out their
// logits; and it streams the span with a division and the mask alone, the listed ones written
// over it.  The table's atomics are integer additions and maxima: the order
// of arrival does not show.  In place and without a temperature only what changes
// is touched.
//
// Out of place the stream may come first, and it overlaps the history's reading by other warps; only the listed tokens
// wait for both.  In place their logits are read, and kept, before the stream writes them.
//
// Measured (GB300, bytes read and written at the copy rate in brackets): 384 x
// 128257 fp32, histories of up to 2500, 90 us (59); 96 x 50257 in bf16 11 us (2.9), 4 x
// 32000 3.2 us: launch and the chain lengths -> history -> marks -> listed logits.  The largest
// is bound by issue (half of its rows, in 38 spans each, in a profile: 80 % of the slots, half of the instructions
// the stream's, of which a division is ten, in pairs five, a quarter the history's, which every CTA of a row reads).
// Logits that are 0 or infinite are divided one by one, with those of their vector and its warp: -inf in every
// 64th place 133 us and 22, in all 172 and 29, in the last 16th of the row 95 and 14.  In place the three take 90, 11 and
// 4 us; without a temperature, when only what changes is written, value by value, 113, 8 and 4, without the mask too 53 and 8.
// Slower, of the time then: a barrier behind each step and loads in their place 18 %, no prefetch of the span to L2
// 19 %, two vectors of a thread on their way at once 5 %, spans of 2048 or 512 threads 35 %, 6 CTAs an SM 8 %, the
// stream's loads in registers ahead of the histories twice the time.
//
#include <algorithm>
#include <cmath>

#include "kv_common.cuh"
#include "launch_common.cuh"
#include "qgkv_launch.h"

namespace qg {
namespace {

constexpr int kThreadsL = 256;
constexpr int kLeastSpan = 1024, kMostSpan = 4096;  // tokens of a CTA: a table and a list of 6 bytes each, of 8 CTAs an SM
constexpr int kCtasL = 8;
// A token's word: how often it was produced, whether it came at all, and the
// place in the list, counted from 1, of the last bias for it.
constexpr unsigned kCame = 1u << 20;
constexpr int kBiasShift = 21;
static_assert(QGKV_MAX_HISTORY < kCame && QGKV_MAX_BIASES < (1 << (32 - kBiasShift)), "a word holds them");

struct LogitArgs {
    const void* x;
    void* out;
    int64_t vocab, x_row, out_row, width;
    int chunks, span;
    const int32_t* history;
    const int32_t* lens;
    const int32_t* prompt_lens;
    const float* repetition;
    const float* presence;
    const float* frequency;
    const int32_t* bias_tokens;
    const float* bias;
    int biases;
    const float* temperature;
    const uint32_t* mask;
    int64_t mask_row;
    int masks;
    const int32_t* mask_rows;
    bool in_place;
    unsigned* status;
};

__device__ __forceinline__ void store_as(float* p, float x) { __stcs(p, x); }
__device__ __forceinline__ void store_as(__half* p, float x) { *p = __float2half_rn(x); }
__device__ __forceinline__ void store_as(__nv_bfloat16* p, float x) { *p = __float2bfloat16_rn(x); }

// An addition in shared memory that each lane makes by itself: few lanes come here at once, and joining them
// first costs more than it saves.
__device__ __forceinline__ unsigned add_shared(unsigned* p, unsigned x) {
    unsigned was;
    asm volatile("atom.shared.add.u32 %0, [%1], %2;"
                 : "=r"(was) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(p))), "r"(x) : "memory");
    return was;
}

// x / t for many x, correctly rounded: from the rounded reciprocal of t, two remainders each exact in one fma
// (Markstein, IBM J. Res. Dev. 34, 1990), where no quotient, product or remainder leaves fp32's normal range;
// other operands (zeros, infinities, far ends) take the division itself.
struct Divisor {
    float t, r;
    bool near_one;
    __device__ explicit Divisor(float by) {
        t = by, r = __frcp_rn(by);
        near_one = fabsf(by) >= 0x1p-40f && fabsf(by) <= 0x1p40f;
    }
    template <int N>
    __device__ __forceinline__ void divide(float (&x)[N]) const {
        static_assert(N % 2 == 0, "pairs");
        float most = 0.f, least = INFINITY;  // NaN is passed over: it stays NaN either way
#pragma unroll
        for (int i = 0; i < N; i += 2) {
            asm("max.abs.f32 %0, %0, %1, %2;" : "+f"(most) : "f"(x[i]), "f"(x[i + 1]));
            asm("min.abs.f32 %0, %0, %1, %2;" : "+f"(least) : "f"(x[i]), "f"(x[i + 1]));
        }
        if (near_one && least >= 0x1p-60f && most <= 0x1p60f) {
#pragma unroll
            for (int i = 0; i < N; i += 2) {
                f2 q = fmul2(f2{x[i], x[i + 1]}, f2{r, r});
#pragma unroll
                for (int again = 0; again < 2; ++again) {
                    f2 rest = {x[i], x[i + 1]};
                    ffma2(rest, q, f2{-t, -t});
                    ffma2(q, rest, f2{r, r});
                }
                x[i] = q.x, x[i + 1] = q.y;
            }
        } else {
#pragma unroll 1
            for (int i = 0; i < N; ++i) {
                float y = 0.f;
#pragma unroll
                for (int k = 0; k < N; ++k) y = k == i ? x[k] : y;
                y = __fdiv_rn(y, t);
#pragma unroll
                for (int k = 0; k < N; ++k) x[k] = k == i ? y : x[k];
            }
        }
    }
};

// 16 bytes of values, and N values stored in whole 16 bytes.
template <class T, int N>
__device__ __forceinline__ void values_of(const uint4& u, float (&x)[N]) {
    const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
    for (int i = 0; i < N; ++i) x[i] = to_f32(e[i]);
}
template <int N>
__device__ __forceinline__ void store_all(float* p, const float (&x)[N]) {
#pragma unroll
    for (int i = 0; i < N; i += 4) __stcs(reinterpret_cast<float4*>(p + i), make_float4(x[i], x[i + 1], x[i + 2], x[i + 3]));
}
template <class O, int N>
__device__ __forceinline__ void store_all(O* p, const float (&x)[N]) {
    O e[N];
#pragma unroll
    for (int i = 0; i < N; ++i) store_as(e + i, x[i]);
    __stcs(reinterpret_cast<uint4*>(p), *reinterpret_cast<const uint4*>(e));
}

template <class T, class O, bool TABLE>
__global__ void __launch_bounds__(kThreadsL, kCtasL) qg_logits_kernel(const LogitArgs a) {
    extern __shared__ __align__(16) unsigned table[];              // [span], then
    uint16_t* listed = reinterpret_cast<uint16_t*>(table + a.span);  // [span] tokens with a word
    __shared__ unsigned count;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / a.chunks;
    const int64_t lo = (blockIdx.x - row * a.chunks) * static_cast<int64_t>(a.span);
    const int n = static_cast<int>(min(static_cast<int64_t>(a.span), a.vocab - lo));
    const T* x = static_cast<const T*>(a.x) + row * a.x_row + lo;
    O* out = static_cast<O*>(a.out) + row * a.out_row + lo;
    const bool heat = a.temperature != nullptr, all = !a.in_place || heat;  // not all: others than the listed stay but for the mask
    if (TABLE && all && tid == 0) {  // the span comes to L2 while the table is filled
        const uintptr_t from = (reinterpret_cast<uintptr_t>(x) + 15) & ~uintptr_t(15);
        const uintptr_t to = reinterpret_cast<uintptr_t>(x + n) & ~uintptr_t(15);
        if (to > from)
            asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(from), "r"(static_cast<uint32_t>(to - from)) : "memory");
    }
    // What the steps below need comes on its way together: lengths and the first biases, then the first of the history.
    int len = 0, made_from = 0;  // tokens of the history, the first that was produced
    float rho = 1.f, presence = 0.f, frequency = 0.f;
    int32_t biased = -1;
    const int32_t* past = nullptr;
    const int32_t* bias_at = nullptr;
    if (TABLE) {
        if (a.bias_tokens) {
            bias_at = a.bias_tokens + row * a.biases;
            if (tid < a.biases) biased = __ldg(bias_at + tid);
        }
        if (a.history) {
            past = a.history + row * a.width;
            len = a.lens[row];
            if (a.prompt_lens) made_from = a.prompt_lens[row];
            if (a.repetition) rho = a.repetition[row];
            if (a.presence) presence = a.presence[row];
            if (a.frequency) frequency = a.frequency[row];
        }
    }
    const Divisor temperature(heat ? a.temperature[row] : 1.f);
    const uint32_t* mask = nullptr;
    if (a.mask) {
        const int64_t m = a.mask_rows ? a.mask_rows[row] : row;
        if (m >= 0 && m < a.masks) mask = a.mask + m * a.mask_row + (lo >> 5);  // lo: a multiple of 32
        else if (m != -1 && tid == 0) atomicOr(a.status, kStatusBounds);
    }
    if (TABLE) {
        for (int i = tid; i < a.span / 4; i += kThreadsL) reinterpret_cast<uint4*>(table)[i] = make_uint4(0, 0, 0, 0);
        if (tid == 0) count = 0;
        if (len < 0 || len > a.width) {
            if (tid == 0) atomicOr(a.status, kStatusBounds);
            len = len < 0 ? 0 : static_cast<int>(a.width);
        }
        constexpr int kMarks = 8;
        int32_t token[kMarks];
        auto tokens_from = [&](int i0) {  // on their way at once
#pragma unroll
            for (int u = 0; u < kMarks; ++u) token[u] = i0 + u * kThreadsL < len ? __ldg(past + i0 + u * kThreadsL) : -1;
        };
        tokens_from(tid);
        __syncthreads();
        const int32_t lo32 = static_cast<int32_t>(lo);
        int t;
        auto within = [&](int32_t x) {  // a token of the span, at t
            t = static_cast<int>(static_cast<unsigned>(x) - static_cast<unsigned>(lo32));
            return x >= lo32 && t < n;
        };
        auto first = [&](unsigned was) {
            if (was == 0u) listed[add_shared(&count, 1u)] = static_cast<uint16_t>(t);
        };
        for (int i = tid; i < a.biases; i += kThreadsL) {
            if (i != tid) biased = __ldg(bias_at + i);
            if (!within(biased)) continue;
            unsigned was = table[t], seen;  // the last of the list counts, whatever the history adds meanwhile
            do {
                seen = was;
                was = atomicCAS(table + t, seen, (seen & (2 * kCame - 1)) | max(seen >> kBiasShift, static_cast<unsigned>(i + 1)) << kBiasShift);
            } while (was != seen);
            first(was);
        }
        // Few of a row's tokens lie in the span: a thread marks which of its next eight do, and a warp goes
        // through the few marks of its lanes together.
        for (int i0 = tid; i0 < len; i0 += kMarks * kThreadsL) {
            if (i0 != tid) tokens_from(i0);
            unsigned marks = 0;
#pragma unroll
            for (int u = 0; u < kMarks; ++u) marks |= within(token[u]) ? 1u << u : 0u;
            while (marks) {
                const int i = i0 + (__ffs(marks) - 1) * kThreadsL;
                marks &= marks - 1;
                within(__ldg(past + i));
                first(i >= made_from ? add_shared(table + t, 1u) : atomicOr(table + t, kCame));
            }
        }
    }
    // A listed token's logit.
    auto adjusted = [&](int t) {
        const unsigned word = table[t], times = word & (kCame - 1), with = word >> kBiasShift;
        float y = to_f32(x[t]);
        const float bias = with ? __ldg(a.bias + row * a.biases + with - 1) : 0.f;
        const uint32_t allowed = mask ? __ldg(mask + (t >> 5)) : ~0u;  // on its way with the others
        if (word & (2 * kCame - 1)) {  // in the history
            if (a.repetition) y = y > 0.f ? __fdiv_rn(y, rho) : __fmul_rn(y, rho);
            if (times) {
                if (a.frequency) y = __fsub_rn(y, __fmul_rn(frequency, static_cast<float>(times)));
                if (a.presence) y = __fsub_rn(y, presence);
            }
        }
        if (with) y = __fadd_rn(y, bias);
        if (heat) y = __fdiv_rn(y, temperature.t);
        return allowed >> (t & 31) & 1u ? y : -INFINITY;
    };
    if (TABLE && a.in_place) {  // the listed tokens' logits are read before the stream writes them
        __syncthreads();
        for (unsigned i = tid; i < count; i += kThreadsL) {
            const int t = listed[i];
            table[t] = __float_as_uint(adjusted(t));
        }
        __syncthreads();
    }
    auto shown = [&](int t) { return !mask || ((__ldg(mask + (t >> 5)) >> (t & 31)) & 1u); };
    auto one = [&](int t) {
        const bool hidden = !shown(t);
        if (!all && !hidden) return;
        float y = hidden ? -INFINITY : to_f32(x[t]);
        if (heat && !hidden) y = __fdiv_rn(y, temperature.t);
        store_as(out + t, y);
    };
    // Whole 16 bytes where input and output meet their borders at the same tokens (a vocabulary of odd size
    // shifts both alike), the few before and behind them one by one.
    constexpr int V = 16 / sizeof(T);
    const int head = static_cast<int>(((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / sizeof(T));
    if (all && n >= 2 * V && (reinterpret_cast<uintptr_t>(out + head) & 15) == 0) {
        const int vectors = (n - head) / V, rest = head + vectors * V;
        const int last_word = (n - 1) >> 5;
        for (int v = tid; v < vectors; v += kThreadsL) {  // their latency is the other warps' time: 64 an SM
            const int t = head + v * V;
            const uint4 u = __ldcs(reinterpret_cast<const uint4*>(x + t));
            const uint32_t bits = mask ? __funnelshift_r(__ldg(mask + (t >> 5)), __ldg(mask + min((t >> 5) + 1, last_word)), t & 31) : ~0u;
            float y[V];
            values_of<T>(u, y);
            if (heat) temperature.divide(y);
#pragma unroll
            for (int k = 0; k < V; ++k)
                if (!(bits >> k & 1u)) y[k] = -INFINITY;
            store_all(out + t, y);
        }
        if (tid < head) one(tid);
        if (rest + tid < n) one(rest + tid);
    } else if (all || mask) {
        for (int t = tid; t < n; t += kThreadsL) one(t);
    }
    if (TABLE) {
        __syncthreads();  // behind the marks and the stream's writes
        for (unsigned i = tid; i < count; i += kThreadsL) {
            const int t = listed[i];
            store_as(out + t, a.in_place ? __uint_as_float(table[t]) : adjusted(t));
        }
    }
}

template <class T, class O>
int launch_typed(const LogitArgs& a, int64_t rows, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(rows * a.chunks);
    if (a.history || a.bias_tokens) qg_logits_kernel<T, O, true><<<grid, kThreadsL, a.span * 6, s>>>(a);
    else qg_logits_kernel<T, O, false><<<grid, kThreadsL, 0, s>>>(a);
    return launch_status();
}

}  // namespace

int launch_logits_adjust(const void* logits, int type, int64_t rows, int64_t vocab, int64_t row_stride, void* out,
                         int out_type, int64_t out_stride, const int32_t* history, int64_t width, const int32_t* lens,
                         const int32_t* prompt_lens, const float* repetition, const float* presence,
                         const float* frequency, const int32_t* bias_tokens, const float* bias, int biases,
                         const float* temperature, const uint32_t* mask, int64_t mask_words, int masks,
                         const int32_t* mask_rows, unsigned* status, cudaStream_t s) {
    const int sms = sm_count(current_device());
    if (sms <= 0) return cuda_fail(cudaGetLastError());
    LogitArgs a = {};
    a.x = logits, a.out = out, a.vocab = vocab, a.x_row = row_stride, a.out_row = out_stride;
    a.history = history, a.width = width, a.lens = lens, a.prompt_lens = prompt_lens;
    a.repetition = repetition, a.presence = presence, a.frequency = frequency;
    a.bias_tokens = biases ? bias_tokens : nullptr, a.bias = bias, a.biases = biases;
    a.temperature = temperature, a.mask = mask, a.mask_row = mask_words, a.masks = masks, a.mask_rows = mask_rows;
    a.in_place = logits == out;
    a.status = status;
    // Spans long enough that reading the history again for each costs little, short enough that few rows keep every SM
    // busy: the least waves x (a span and what a CTA costs beside it, as much as some 2000 tokens).  Many waves
    // count whole, for the last takes as long with few CTAs (384 x 128257: 34 spans, 10.7 waves, 90 us, 32 spans, 10.1
    // waves, 92); few overlap, and half a wave stands for their latencies (96 x 50257: 13 spans, 1.03 waves, 10.9 us,
    // 25 spans 13.3; 4 x 32000: spans of 1024 tokens 3.1 us, of 4096 4.0).
    const double slots = static_cast<double>(kCtasL) * sms;
    const int64_t fewest = (vocab + kMostSpan - 1) / kMostSpan, most = (vocab + kLeastSpan - 1) / kLeastSpan;
    int64_t span = 0;
    double best = INFINITY;
    for (int64_t n = fewest; n <= most; n += std::max<int64_t>(1, fewest / 16)) {
        const int64_t of = ((vocab + n - 1) / n + 31) / 32 * 32;
        const double waves = static_cast<double>(rows * n) / slots;
        const double cost = ((waves > 4 ? std::ceil(waves) : waves) + 0.5) * static_cast<double>(of + 2048);
        if (cost < best) best = cost, span = of;
    }
    const int64_t chunks = (vocab + span - 1) / span;
    if (rows * chunks > INT32_MAX) return QG_EINVAL;
    a.span = static_cast<int>(span), a.chunks = static_cast<int>(chunks);
    if (type == QGKV_F32) return launch_typed<float, float>(a, rows, s);
    if (type == QGKV_F16)
        return out_type == QGKV_F32 ? launch_typed<__half, float>(a, rows, s) : launch_typed<__half, __half>(a, rows, s);
    return out_type == QGKV_F32 ? launch_typed<__nv_bfloat16, float>(a, rows, s)
                                : launch_typed<__nv_bfloat16, __nv_bfloat16>(a, rows, s);
}

}  // namespace qg
