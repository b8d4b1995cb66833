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
// logits; then it streams the span with a division and the mask alone, and writes the
// listed ones over it.  The table's atomics are integer additions and maxima: the order
// of arrival does not show.  In place and without a temperature only what changes
// is touched.
//
#include <algorithm>

#include "kv_common.cuh"
#include "launch_common.cuh"
#include "qgkv_launch.h"

namespace qg {
namespace {

constexpr int kThreadsL = 256;
constexpr int kPerL = 8;           // logits of a thread on their way at once
constexpr int kMostSpan = 4096;    // tokens of a CTA: a table of 16 KB, a list of 8
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

// x / t for many x, correctly rounded: from the rounded reciprocal of t, two remainders each exact in one fma
// (Markstein, IBM J. Res. Dev. 34, 1990).  Operands whose quotients, products or remainders could leave
// fp32's normal range, zeros, infinities and NaN take the division itself.
struct Divisor {
    float t, r;
    bool near_one;
    __device__ explicit Divisor(float by) {
        t = by, r = __frcp_rn(by);
        near_one = fabsf(by) >= 0x1p-40f && fabsf(by) <= 0x1p40f;
    }
    __device__ __forceinline__ float of(float x) const {
        const float ax = fabsf(x);
        if (!(near_one && ax >= 0x1p-60f && ax <= 0x1p60f)) return __fdiv_rn(x, t);
        float q = __fmul_rn(x, r);
        q = __fmaf_rn(__fmaf_rn(-q, t, x), r, q);
        return __fmaf_rn(__fmaf_rn(-q, t, x), r, q);
    }
};

template <class T, class O, bool TABLE>
__global__ void __launch_bounds__(kThreadsL) qg_logits_kernel(const LogitArgs a) {
    extern __shared__ __align__(16) unsigned table[];              // [span], then
    uint16_t* listed = reinterpret_cast<uint16_t*>(table + a.span);  // [span] tokens with a word
    __shared__ int count;
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / a.chunks;
    const int64_t lo = (blockIdx.x - row * a.chunks) * static_cast<int64_t>(a.span);
    const int n = static_cast<int>(min(static_cast<int64_t>(a.span), a.vocab - lo));
    const T* x = static_cast<const T*>(a.x) + row * a.x_row + lo;
    O* out = static_cast<O*>(a.out) + row * a.out_row + lo;
    const bool heat = a.temperature != nullptr;
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
        __syncthreads();
        auto first = [&](unsigned was, int t) {
            if (was == 0u) listed[atomicAdd(&count, 1)] = static_cast<uint16_t>(t);
        };
        if (a.bias_tokens) {
            const int32_t* at = a.bias_tokens + row * a.biases;
            for (int i = tid; i < a.biases; i += kThreadsL) {
                const int64_t t = at[i] - lo;
                if (t >= 0 && t < n) first(atomicMax(table + t, static_cast<unsigned>(i + 1) << kBiasShift), static_cast<int>(t));
            }
            __syncthreads();
        }
        if (a.history) {
            int64_t len = a.lens[row];
            const int64_t prompt = a.prompt_lens ? a.prompt_lens[row] : 0;
            if (len < 0 || len > a.width) {
                if (tid == 0) atomicOr(a.status, kStatusBounds);
                len = len < 0 ? 0 : a.width;
            }
            const int32_t* at = a.history + row * a.width;
            for (int i0 = tid; i0 < len; i0 += 4 * kThreadsL) {
                int32_t token[4];  // on their way at once
#pragma unroll
                for (int u = 0; u < 4; ++u) token[u] = i0 + u * kThreadsL < len ? __ldg(at + i0 + u * kThreadsL) : -1;
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const int64_t t = token[u] - lo;
                    if (token[u] < 0 || t < 0 || t >= n) continue;
                    first(i0 + u * kThreadsL >= prompt ? atomicAdd(table + t, 1u) : atomicOr(table + t, kCame), static_cast<int>(t));
                }
            }
        }
        __syncthreads();
        const float rho = a.repetition ? a.repetition[row] : 1.f;
        const float presence = a.presence ? a.presence[row] : 0.f, frequency = a.frequency ? a.frequency[row] : 0.f;
        const int have = count;
        for (int i = tid; i < have; i += kThreadsL) {  // each token once: its word becomes its logit
            const int t = listed[i];
            const unsigned word = table[t], times = word & (kCame - 1), with = word >> kBiasShift;
            float y = to_f32(x[t]);
            if (word & (2 * kCame - 1)) {  // in the history
                if (a.repetition) y = y > 0.f ? __fdiv_rn(y, rho) : __fmul_rn(y, rho);
                if (times) {
                    if (a.frequency) y = __fsub_rn(y, __fmul_rn(frequency, static_cast<float>(times)));
                    if (a.presence) y = __fsub_rn(y, presence);
                }
            }
            if (with) y = __fadd_rn(y, a.bias[row * a.biases + with - 1]);
            if (heat) y = __fdiv_rn(y, temperature.t);
            if (mask && !((__ldg(mask + (t >> 5)) >> (t & 31)) & 1u)) y = -INFINITY;
            table[t] = __float_as_uint(y);
        }
        __syncthreads();  // all have read their logits before they are written in place
    }
    const bool all = !a.in_place || heat;  // else the others stay but for the mask
    if (all || mask) {
        int at = tid;
        for (; at + (kPerL - 1) * kThreadsL < n; at += kThreadsL * kPerL) {
            float v[kPerL];
            uint32_t bits[kPerL];
#pragma unroll
            for (int i = 0; i < kPerL; ++i) {
                if (all) v[i] = to_f32(x[at + i * kThreadsL]);
                if (mask) bits[i] = __ldg(mask + ((at + i * kThreadsL) >> 5)) >> (at & 31);
            }
#pragma unroll
            for (int i = 0; i < kPerL; ++i) {
                if (heat) v[i] = temperature.of(v[i]);
                const bool hidden = mask && !(bits[i] & 1u);
                if (all || hidden) store_as(out + at + i * kThreadsL, hidden ? -INFINITY : v[i]);
            }
        }
        for (; at < n; at += kThreadsL) {
            const bool hidden = mask && !((__ldg(mask + (at >> 5)) >> (at & 31)) & 1u);
            if (hidden) store_as(out + at, -INFINITY);
            else if (all) store_as(out + at, heat ? temperature.of(to_f32(x[at])) : to_f32(x[at]));
        }
    }
    if (TABLE) {
        __syncthreads();  // behind the stream's writes
        for (int i = tid; i < count; i += kThreadsL) {
            const int t = listed[i];
            store_as(out + t, __uint_as_float(table[t]));
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
    // Spans long enough that reading the history again for each costs little,
    // short enough that few rows keep every SM busy.
    int64_t span = rows * vocab / (4 * static_cast<int64_t>(sms));
    span = std::min<int64_t>(std::max<int64_t>(span, 1024), kMostSpan) / 1024 * 1024;
    int64_t chunks = (vocab + span - 1) / span;
    if (rows * chunks > INT32_MAX) return QG_EINVAL;
    a.span = static_cast<int>(span), a.chunks = static_cast<int>(chunks);
    if (type == QGKV_F32) return launch_typed<float, float>(a, rows, s);
    if (type == QGKV_F16)
        return out_type == QGKV_F32 ? launch_typed<__half, float>(a, rows, s) : launch_typed<__half, __half>(a, rows, s);
    return out_type == QGKV_F32 ? launch_typed<__nv_bfloat16, float>(a, rows, s)
                                : launch_typed<__nv_bfloat16, __nv_bfloat16>(a, rows, s);
}

}  // namespace qg
