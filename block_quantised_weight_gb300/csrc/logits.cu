// Adjustment of logits before a selection: penalties for tokens that have come
// before, listed biases, temperature, a grammar's mask.
//
// Mathematics: qgkv.h, qglogits_adjust; each operation is rounded to fp32 by
// itself, so the result is a function of the inputs alone.
//
// Bound.  Every logit is read and written once: HBM for batches.  What a token's
// logit needs besides (how often it came, whether a bias is listed for it) is
// scattered, so a CTA takes a span of a row's vocabulary, gathers these for
// its span in a table in shared memory, one word a token, from the whole history
// and list of the row, and then streams the logits of the span.  The table's
// atomics are integer additions and maxima: the order of arrival does not show.
// In place and without a temperature only the logits that change are read.
#include <algorithm>

#include "kv_common.cuh"
#include "launch_common.cuh"
#include "qgkv_launch.h"

namespace qg {
namespace {

constexpr int kThreadsL = 256;
constexpr int kPerL = 8;           // logits of a thread on their way at once
constexpr int kMostSpan = 8192;    // tokens of a CTA: a table of 32 KB
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

template <class T, class O, bool TABLE>
__global__ void __launch_bounds__(kThreadsL) qg_logits_kernel(const LogitArgs a) {
    extern __shared__ unsigned table[];  // [span]
    const int tid = threadIdx.x;
    const int64_t row = blockIdx.x / a.chunks;
    const int64_t lo = (blockIdx.x - row * a.chunks) * static_cast<int64_t>(a.span);
    const int n = static_cast<int>(min(static_cast<int64_t>(a.span), a.vocab - lo));
    float rho = 1.f, presence = 0.f, frequency = 0.f;
    if (TABLE) {
        for (int i = tid; i < n; i += kThreadsL) table[i] = 0u;
        __syncthreads();
        if (a.bias_tokens) {
            const int32_t* at = a.bias_tokens + row * a.biases;
            for (int i = tid; i < a.biases; i += kThreadsL) {
                const int64_t t = at[i] - lo;
                if (t >= 0 && t < n) atomicMax(table + t, static_cast<unsigned>(i + 1) << kBiasShift);
            }
            __syncthreads();
        }
        if (a.history) {
            int64_t len = a.lens[row];
            int64_t prompt = a.prompt_lens ? a.prompt_lens[row] : 0;
            if (len < 0 || len > a.width) {
                if (tid == 0) atomicOr(a.status, kStatusBounds);
                len = len < 0 ? 0 : a.width;
            }
            const int32_t* at = a.history + row * a.width;
            for (int i = tid; i < len; i += kThreadsL) {
                const int64_t t = at[i] - lo;
                if (t < 0 || t >= n) continue;
                if (i >= prompt) atomicAdd(table + t, 1u);
                else atomicOr(table + t, kCame);
            }
            if (a.repetition) rho = a.repetition[row];
            if (a.presence) presence = a.presence[row];
            if (a.frequency) frequency = a.frequency[row];
            __syncthreads();
        }
    }
    const bool heat = a.temperature != nullptr;
    const float temperature = heat ? a.temperature[row] : 1.f;
    const uint32_t* mask = nullptr;
    if (a.mask) {
        const int64_t m = a.mask_rows ? a.mask_rows[row] : row;
        if (m >= 0 && m < a.masks) mask = a.mask + m * a.mask_row + (lo >> 5);  // lo: a multiple of 32
        else if (m != -1 && tid == 0) atomicOr(a.status, kStatusBounds);
    }
    const T* x = static_cast<const T*>(a.x) + row * a.x_row + lo;
    O* out = static_cast<O*>(a.out) + row * a.out_row + lo;
    const float* bias = a.bias ? a.bias + row * a.biases : nullptr;
    for (int at = tid; at < n; at += kThreadsL * kPerL) {
        float v[kPerL];
        unsigned word[kPerL];
        bool allowed[kPerL];
#pragma unroll
        for (int i = 0; i < kPerL; ++i) {
            const int t = at + i * kThreadsL;
            allowed[i] = true, word[i] = 0u, v[i] = 0.f;
            if (t < n) {
                if (mask) allowed[i] = (__ldg(mask + (t >> 5)) >> (t & 31)) & 1u;
                if (TABLE) word[i] = table[t];
                if (allowed[i] && (!a.in_place || heat || word[i])) v[i] = to_f32(x[t]);
            }
        }
#pragma unroll
        for (int i = 0; i < kPerL; ++i) {
            const int t = at + i * kThreadsL;
            if (t >= n) break;
            float y = v[i];
            if (TABLE && word[i]) {
                const unsigned count = word[i] & (kCame - 1);
                if (a.history && (word[i] & (2 * kCame - 1))) {
                    if (a.repetition) y = y > 0.f ? __fdiv_rn(y, rho) : __fmul_rn(y, rho);
                    if (count) {
                        if (a.frequency) y = __fsub_rn(y, __fmul_rn(frequency, static_cast<float>(count)));
                        if (a.presence) y = __fsub_rn(y, presence);
                    }
                }
                const unsigned listed = word[i] >> kBiasShift;
                if (listed) y = __fadd_rn(y, bias[listed - 1]);
            }
            if (heat) y = __fdiv_rn(y, temperature);
            if (!allowed[i]) y = -INFINITY;
            if (!a.in_place || heat || word[i] || !allowed[i]) store_as(out + t, y);
        }
    }
}

template <class T, class O>
int launch_typed(const LogitArgs& a, int64_t rows, cudaStream_t s) {
    const unsigned grid = static_cast<unsigned>(rows * a.chunks);
    if (a.history || a.bias_tokens) qg_logits_kernel<T, O, true><<<grid, kThreadsL, a.span * 4, s>>>(a);
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
