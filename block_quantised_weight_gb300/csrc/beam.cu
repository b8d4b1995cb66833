// Beam selection: the best continuations of each request over its beams and
// the vocabulary.
//
// Mathematics.  score = cum[beam] + x - lse(row), lse = m + log(sum 2^((x - m)
// log2 e)).  Within a row the order is that of the logits, so a row's part
// only has to keep its `keep` largest logits, whatever its lse; the scores
// are formed in 64 bits at the end, from few candidates.
//
// Bound.  Every logit is read once: HBM-bound for batches, latency-bound for
// one request.  A CTA streams a part of a row, the next step's values on
// their way while one is summed: the running maximum and sum per thread, and
// a buffer of candidates in shared memory.  A logit enters the buffer when it
// reaches a floor that at least `keep` values reach.  The floor comes from
// the threads' own maxima: every warp sorts its 32 and takes the
// ceil(keep / 8)-th; the least of these eight is reached at least `keep`
// times, and about 20 random values of a step pass it for keep = 8.  So a value
// costs five instructions, and a step one barrier.  The last CTA of a request
// to arrive merges the parts; all order is by (value, index), so the result
// does not depend on who arrives when.
// Measured: 48 requests x 8 beams x 128257 logits, keep 16: 62 us, 3.2 TB/s, bound by
// issue and the barrier of a step; 4 beams x 32000, keep 8: 12.5 us, latency.
#include <atomic>

#include "kv_common.cuh"
#include "launch_common.cuh"
#include "qgkv_launch.h"

namespace qg {
namespace {

constexpr int kBeamThreads = 256;
constexpr int kPer = 16;                           // values a thread takes in one step
constexpr int kStep = kBeamThreads * kPer;
constexpr int kWarps = kBeamThreads / 32;
constexpr int kKeepLimit = 1024;                   // buffered candidates above which the buffer is thinned
constexpr int kMergePer = 2;                       // parts' candidates a thread takes in one step of the merge
constexpr int kMergeStep = kBeamThreads * kMergePer;

// Larger is better; all keys of one selection differ.
struct Key1 {  // (logit, token): order of the logit's bits, then the lower token
    unsigned long long a;
    __device__ static Key1 lowest() { return {0ull}; }
    __device__ bool operator<(const Key1& o) const { return a < o.a; }
    __device__ Key1 from(int mask) const { return {__shfl_xor_sync(~0u, a, mask)}; }
    __device__ Key1 at(int lane) const { return {__shfl_sync(~0u, a, lane)}; }
};
struct Key2 {  // (score, flat index)
    unsigned long long a, b;
    __device__ static Key2 lowest() { return {0ull, 0ull}; }
    __device__ bool operator<(const Key2& o) const { return a < o.a || (a == o.a && b < o.b); }
    __device__ Key2 from(int mask) const { return {__shfl_xor_sync(~0u, a, mask), __shfl_xor_sync(~0u, b, mask)}; }
    __device__ Key2 at(int lane) const { return {__shfl_sync(~0u, a, lane), __shfl_sync(~0u, b, lane)}; }
};

__device__ __forceinline__ uint32_t ordered(float x) {
    const uint32_t u = __float_as_uint(x);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) {
    return __uint_as_float(u & 0x80000000u ? u & 0x7FFFFFFFu : ~u);
}
__device__ __forceinline__ unsigned long long ordered64(double x) {
    const unsigned long long u = static_cast<unsigned long long>(__double_as_longlong(x));
    return u >> 63 ? ~u : u | 0x8000000000000000ull;
}
__device__ __forceinline__ double unordered64(unsigned long long u) {
    return __longlong_as_double(static_cast<long long>(u >> 63 ? u & 0x7FFFFFFFFFFFFFFFull : ~u));
}

// A value that at least `keep` of the CTA's threads' values `mine` reach: the
// least over the warps of their ceil(keep / 8)-th largest.  scratch: 8 floats.
__device__ __forceinline__ float floor_of(float mine, int keep, float* scratch) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
        for (int step = size >> 1; step > 0; step >>= 1) {
            const float other = __shfl_xor_sync(~0u, mine, step);
            // the larger goes to the lower lane where the run falls
            mine = ((lane & step) == 0) == ((lane & size) == 0) ? fmaxf(mine, other) : fminf(mine, other);
        }
    const float kth = __shfl_sync(~0u, mine, (keep + kWarps - 1) / kWarps - 1);
    if (lane == 0) scratch[threadIdx.x >> 5] = kth;
    __syncthreads();
    float least = scratch[0];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) least = fminf(least, scratch[w]);
    return least;
}

// A sum in two floats: what rounding takes from the first is kept in the second.
struct Sum2 {
    float hi, lo;
    __device__ void add(float x, float x_lo = 0.f) {
        const float s = __fadd_rn(hi, x), b = __fsub_rn(s, hi);
        lo += __fadd_rn(__fsub_rn(hi, __fsub_rn(s, b)), __fsub_rn(x, b)) + x_lo;
        hi = s;
    }
    __device__ void add_lanes() {
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            const float h2 = __shfl_xor_sync(~0u, hi, o), l2 = __shfl_xor_sync(~0u, lo, o);
            // the same operands in both lanes of a pair, in the same order
            const bool low = (threadIdx.x & o) == 0;
            const float a = low ? hi : h2, b = low ? h2 : hi;
            const float s = __fadd_rn(a, b), t = __fsub_rn(s, a);
            lo = (lo + l2) + __fadd_rn(__fsub_rn(a, __fsub_rn(s, t)), __fsub_rn(b, t));
            hi = s;
        }
    }
};

// The candidates of a CTA and the threshold below which nothing is kept.
template <class K, int PUSHED>
struct Pool {
    static constexpr int kCap = kKeepLimit + PUSHED;  // PUSHED: the most that one step adds
    K buf[kCap];
    K top[kBeamThreads];
    K floor_key;
    int n;

    __device__ void reset() {
        if (threadIdx.x == 0) {
            n = 0;
            floor_key = K::lowest();
        }
        __syncthreads();
    }
    // floor_key = a key that at least `keep` of the threads' keys `mine`
    // reach (or the lowest): the least over the warps of their
    // ceil(keep / 8)-th largest.
    __device__ void raise(K mine, int keep) {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int size = 2; size <= 32; size <<= 1)
#pragma unroll
            for (int step = size >> 1; step > 0; step >>= 1) {
                const K other = mine.from(step);
                // the larger goes to the lower lane where the run falls
                const bool larger = ((lane & step) == 0) == ((lane & size) == 0);
                if (larger ? mine < other : other < mine) mine = other;
            }
        const K kth = mine.at((keep + kWarps - 1) / kWarps - 1);
        if (lane == 0) top[threadIdx.x >> 5] = kth;
        __syncthreads();
        if (threadIdx.x == 0) {
            K least = top[0];
            for (int w = 1; w < kWarps; ++w)
                if (top[w] < least) least = top[w];
            if (floor_key < least) floor_key = least;
        }
        __syncthreads();
    }
    // The same with the keep-th largest of all, by counting: bounds what is
    // left by keep threads' shares whatever the order of the values.
    __device__ void raise_exact(K mine, int keep) {
        top[threadIdx.x] = mine;
        __syncthreads();
        int above = 0;
#pragma unroll 8
        for (int i = 0; i < kBeamThreads; ++i)
            above += (mine < top[i] || (i < threadIdx.x && !(top[i] < mine))) ? 1 : 0;
        if (above == keep - 1 && floor_key < mine) floor_key = mine;
        __syncthreads();
    }
    __device__ void push(K k) { buf[atomicAdd(&n, 1)] = k; }
    // Thin the buffer: a floor from every thread's largest of its share; what
    // is below goes.
    __device__ void thin(int keep, bool exact) {
        constexpr int kShare = kCap / kBeamThreads;
        K mine[kShare];
        K best = K::lowest();
        const int have = n;
#pragma unroll
        for (int j = 0; j < kShare; ++j) {
            const int i = j * kBeamThreads + threadIdx.x;
            mine[j] = i < have ? buf[i] : K::lowest();
            if (best < mine[j]) best = mine[j];
        }
        if (exact) raise_exact(best, keep);
        else raise(best, keep);
        if (threadIdx.x == 0) n = 0;
        __syncthreads();
        const K f = floor_key;
#pragma unroll
        for (int j = 0; j < kShare; ++j)
            if (!(mine[j] < f) && K::lowest() < mine[j]) push(mine[j]);
        __syncthreads();
    }
    // Until at most `limit` (at least 256) are left; the counting form
    // where the sorted one does not halve the buffer.  Counting leaves at most
    // keep threads' shares, so it gets below 2 * keep.
    __device__ void thin_to(int limit, int keep) {
        bool exact = false;
        while (n > limit) {
            const int was = n;
            __syncthreads();
            thin(keep, exact);
            if (exact && n >= was) break;
            exact = 2 * n > was;
        }
        __syncthreads();
    }
    // After a step's pushes (one barrier): whether the buffer has to be
    // thinned.  The last thread to push sees the whole count.
    __device__ bool crowded() {
        return __syncthreads_or(*reinterpret_cast<volatile int*>(&n) > kKeepLimit) != 0;
    }
    // After the last push: calls f(rank, key) for the best `keep`.
    template <class F>
    __device__ void finish(int keep, F f) {
        if (n > 96) {  // the ranks below cost n comparisons each: one cheap pass
            __syncthreads();
            thin(keep, false);
        }
        thin_to(256, keep);
        const int have = n;
        for (int i = threadIdx.x; i < have; i += kBeamThreads) {
            const K k = buf[i];
            int rank = 0;
#pragma unroll 8
            for (int j = 0; j < have; ++j) rank += k < buf[j] ? 1 : 0;
            if (rank < keep) f(rank, k);
        }
    }
};

struct BeamArgs {
    const void* logits;
    const float* cum;
    int beams, keep, splits, part_keep;
    int64_t vocab, row_stride, span;
    unsigned long long* keys;  // [rows][splits][part_keep]
    float4* parts;             // [rows][splits] maximum, sum (two floats)
    unsigned* count;           // [requests]
    float* scores;
    int32_t* tokens;
    int32_t* parents;
};

// A thread's values of a step: tokens at + i * kBeamThreads, -inf from `end`
// on.  One value a load: a row may start anywhere (a vocabulary of odd size),
// and which thread sums which tokens must not depend on the address, or equal
// rows would get unequal sums.
template <class T>
__device__ __forceinline__ void load_step(const T* p, int at, int end, float (&x)[kPer]) {
    if (at + (kPer - 1) * kBeamThreads < end) {
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = to_f32(__ldcs(p + at + i * kBeamThreads));
    } else {
#pragma unroll
        for (int i = 0; i < kPer; ++i)
            x[i] = at + i * kBeamThreads < end ? to_f32(__ldcs(p + at + i * kBeamThreads)) : -INFINITY;
    }
}

template <class T>
__global__ void __launch_bounds__(kBeamThreads, 3) qg_beam_kernel(const BeamArgs a) {
    extern __shared__ __align__(16) unsigned char smem[];
    __shared__ float red_m[2 * kWarps];
    __shared__ Sum2 red_l[kWarps];
    __shared__ bool last;
    __shared__ double row_lse[QGKV_MAX_BEAMS];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int64_t row = blockIdx.x / a.splits;
    const int split = static_cast<int>(blockIdx.x - row * a.splits);
    const T* p = static_cast<const T*>(a.logits) + row * a.row_stride;
    const int lo = static_cast<int>(split * a.span), end = static_cast<int>(min(lo + a.span, a.vocab));

    Pool<Key1, kStep>& pool = *reinterpret_cast<Pool<Key1, kStep>*>(smem);
    pool.reset();
    float m = -INFINITY, l = 0.f, floor_value = -INFINITY;
    float next[kPer];
    load_step(p, lo + tid, end, next);
    int steps = 1;
    for (int at0 = lo; at0 < end; at0 += kStep) {
        const int at = at0 + tid;
        float x[kPer];
#pragma unroll
        for (int i = 0; i < kPer; ++i) x[i] = next[i];
        if (at0 + kStep < end) load_step(p, at + kStep, end, next);
        float top = x[0];
#pragma unroll
        for (int i = 1; i < kPer; ++i) top = fmaxf(top, x[i]);
        if (top > m) {
            l *= exp2_fast((m - top) * 1.4426950408889634f);
            m = top;
        }
        // a thread without a finite maximum keeps l = 0; NaN has to reach l
        const float ref = m == -INFINITY ? 0.f : m;
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) s += exp2_fast((x[i] - ref) * 1.4426950408889634f);
        l += s;
        auto key = [&](int i) {
            const int token = at + i * kBeamThreads;
            Key1 k = {0ull};
            if (token < end && x[i] == x[i])
                // + 0: the two zeros are equal, and rank by their tokens
                k.a = (static_cast<unsigned long long>(ordered(x[i] + 0.f)) << 32) | (0xFFFFFFFFu - static_cast<uint32_t>(token));
            return k;
        };
        // the floor from the threads' maxima so far, at steps 1, 2, 4, 8, ...
        if ((steps & (steps - 1)) == 0) {
            const float f = floor_of(m, a.keep, red_m + (steps & 1) * kWarps);
            floor_value = fmaxf(floor_value, f);
        }
        if (top >= floor_value) {
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (x[i] >= floor_value) {
                    const Key1 k = key(i);
                    if (k.a) pool.push(k);
                }
        }
        ++steps;
        if (pool.crowded()) {
            pool.thin_to(kKeepLimit, a.keep);
            if (pool.floor_key.a) floor_value = fmaxf(floor_value, unordered(static_cast<uint32_t>(pool.floor_key.a >> 32)));
        }
    }
    // the part's maximum and sum
    float M = m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) M = fmaxf(M, __shfl_xor_sync(~0u, M, o));
    if (lane == 0) red_m[warp] = M;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kWarps; ++w) M = fmaxf(M, red_m[w]);
    Sum2 L = {m == -INFINITY ? l : l * exp2_fast((m - M) * 1.4426950408889634f), 0.f};
    L.add_lanes();
    if (lane == 0) red_l[warp] = L;
    __syncthreads();
    const int64_t at_part = row * a.splits + split;
    if (tid == 0) {
#pragma unroll
        for (int w = 1; w < kWarps; ++w) L.add(red_l[w].hi, red_l[w].lo);
        a.parts[at_part] = make_float4(M, L.hi, L.lo, 0.f);
    }
    unsigned long long* out = a.keys + at_part * a.part_keep;
    for (int i = tid; i < a.part_keep; i += kBeamThreads)
        if (i >= pool.n) out[i] = 0ull;  // a part with fewer
    __syncthreads();
    pool.finish(a.part_keep, [&](int rank, Key1 k) { out[rank] = k.a; });

    // ---- the request's last part merges
    const int64_t request = row / a.beams;
    __threadfence();
    __syncthreads();
    if (tid == 0) {
        const unsigned need = static_cast<unsigned>(a.beams * a.splits);
        last = atomicAdd(a.count + request, 1u) == need - 1;
        if (last) a.count[request] = 0u;
        __threadfence();
    }
    __syncthreads();
    if (!last) return;
    const int64_t row0 = request * a.beams;
    for (int b = warp; b < a.beams; b += kWarps) {
        const float4* parts = a.parts + (row0 + b) * a.splits;
        float mm = -INFINITY;
        for (int s = lane; s < a.splits; s += 32) mm = fmaxf(mm, __ldcg(parts + s).x);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mm = fmaxf(mm, __shfl_xor_sync(~0u, mm, o));
        Sum2 sum = {0.f, 0.f};
        for (int s = lane; s < a.splits; s += 32) {
            const float4 q = __ldcg(parts + s);
            const float w = q.x == -INFINITY ? 1.f : exp2_fast((q.x - mm) * 1.4426950408889634f);
            sum.add(w * q.y, w * q.z);
        }
        sum.add_lanes();
        if (lane == 0) {
            const float cb = a.cum[row0 + b];
            const float total = sum.hi + sum.lo;
            const bool good = total > 0.f && total < INFINITY && mm < INFINITY && mm > -INFINITY && cb < INFINITY && cb > -INFINITY;
            // log(sum) = e log 2 + log(f), f in [1, 2): logf of f is right to 2^-25
            const int e = static_cast<int>(__float_as_uint(total) >> 23) - 127;
            const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            const float f = sum.hi * down;
            const double ln = static_cast<double>(logf(f)) + static_cast<double>(sum.lo * down / f) + e * 0.69314718055994530942;
            row_lse[b] = good ? static_cast<double>(mm) + ln : __longlong_as_double(0x7FF8000000000000ll);
        }
    }
    Pool<Key2, kMergeStep>& merge = *reinterpret_cast<Pool<Key2, kMergeStep>*>(smem);
    __syncthreads();
    merge.reset();
    const int per_row = a.splits * a.part_keep;
    const int total = a.beams * per_row;
    // Scores in 32 bits first: `keep` candidates reach the floor of their lower
    // bounds, and only those whose upper bound reaches it are formed in 64.
    floor_value = -INFINITY;
    for (int at0 = 0; at0 < total; at0 += kMergeStep) {
        unsigned long long k[kMergePer];
        float upper[kMergePer], best = -INFINITY;
        int beam[kMergePer];
#pragma unroll
        for (int i = 0; i < kMergePer; ++i) {
            const int e = at0 + i * kBeamThreads + tid;
            k[i] = 0ull;
            upper[i] = -INFINITY;
            beam[i] = 0;
            if (e < total) {
                beam[i] = e / per_row;
                k[i] = __ldcg(a.keys + (row0 + beam[i]) * per_row + (e - beam[i] * per_row));
                if (row_lse[beam[i]] == row_lse[beam[i]] && k[i]) {
                    const float lse = static_cast<float>(row_lse[beam[i]]), cum = a.cum[row0 + beam[i]];
                    const float v = unordered(static_cast<uint32_t>(k[i] >> 32));
                    const float score = cum + (v - lse);
                    const float off = v == -INFINITY ? 0.f : (fabsf(cum) + fabsf(v) + fabsf(lse)) * 4.8e-7f;
                    upper[i] = score + off;
                    best = fmaxf(best, score - off);
                }
            }
        }
        if (at0 == 0) floor_value = floor_of(best, a.keep, red_m);
#pragma unroll
        for (int i = 0; i < kMergePer; ++i) {
            const int e = at0 + i * kBeamThreads + tid;
            // a bound that is NaN (sums beyond fp32: -inf + inf) excludes nothing
            if (e >= total || upper[i] < floor_value) continue;
            const double lse = row_lse[beam[i]];
            double score = -INFINITY;
            int64_t token = e - beam[i] * per_row;  // of a row that scores -inf throughout: its first tokens
            bool real = token < a.vocab;
            if (lse == lse) {
                real = k[i] != 0ull;
                token = 0xFFFFFFFFu - static_cast<uint32_t>(k[i]);
                score = static_cast<double>(a.cum[row0 + beam[i]]) +
                        (static_cast<double>(unordered(static_cast<uint32_t>(k[i] >> 32))) - lse);
            }
            if (real)
                merge.push({ordered64(score),
                            0x7FFFFFFFFFFFFFFFull - static_cast<unsigned long long>(beam[i] * a.vocab + token)});
        }
        if (merge.crowded()) merge.thin_to(kKeepLimit, a.keep);
    }
    merge.finish(a.keep, [&](int rank, Key2 k) {
        const unsigned long long flat = 0x7FFFFFFFFFFFFFFFull - k.b;
        const uint32_t vocab = static_cast<uint32_t>(a.vocab);
        const int64_t b = flat >> 32 ? flat / vocab : static_cast<uint32_t>(flat) / vocab;
        const int64_t to = request * a.keep + rank;
        a.scores[to] = static_cast<float>(unordered64(k.a));
        a.tokens[to] = static_cast<int32_t>(flat - b * a.vocab);
        a.parents[to] = static_cast<int32_t>(row0 + b);
    });
}

template <class T>
int launch_beam(BeamArgs a, int requests, cudaStream_t s) {
    constexpr int smem = static_cast<int>(std::max(sizeof(Pool<Key1, kStep>), sizeof(Pool<Key2, kMergeStep>)));
    const int dev = current_device();
    static std::atomic<bool> done[64];
    if (dev < 0) return cuda_fail(cudaGetLastError());
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(qg_beam_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess)
            return cuda_fail(cudaGetLastError());
        done[dev].store(true, std::memory_order_release);
    }
    qg_beam_kernel<T><<<static_cast<unsigned>(requests * a.beams * a.splits), kBeamThreads, smem, s>>>(a);
    return launch_status();
}

}  // namespace

int launch_beam_select(const void* logits, int type, const float* cum, int requests, int beams, int64_t vocab,
                       int64_t row_stride, int keep, float* scores, int32_t* tokens, int32_t* parents,
                       uint8_t* workspace, cudaStream_t s) {
    const int sms = sm_count(current_device());
    if (sms <= 0) return cuda_fail(cudaGetLastError());
    BeamArgs a = {};
    a.logits = logits, a.cum = cum, a.beams = beams, a.keep = keep, a.vocab = vocab, a.row_stride = row_stride;
    a.scores = scores, a.tokens = tokens, a.parents = parents;
    const int64_t rows = static_cast<int64_t>(requests) * beams;
    // No more parts than the three CTAs an SM hold at once (384 rows of 128257
    // values: 62.5 us, with twice the parts 73.5, in two waves), each at least
    // 2048 values long.  One CTA merges a request's parts, so these are few: 8
    // beams of 128257 values in 456 parts 40 us, 256 parts 30, 128 parts 23, 64
    // parts 25; one beam in 63 parts 14 us, 32 parts 11, 16 parts 12.
    int64_t splits = 3 * sms / rows;
    splits = std::min<int64_t>(splits, (vocab + 2047) / 2048);
    splits = std::min({splits, static_cast<int64_t>(128 / beams), std::max<int64_t>(16, vocab / 8192)});
    const int64_t room = kWsPartBytes - 64;
    splits = std::max<int64_t>(1, std::min(splits, room / (rows * (keep * 8 + 16))));
    a.span = (vocab + splits - 1) / splits;
    splits = (vocab + a.span - 1) / a.span;
    a.splits = static_cast<int>(splits);
    a.part_keep = static_cast<int>(std::min<int64_t>(keep, vocab));
    if (rows * splits * (a.part_keep * 8 + 16) > room) return QG_ESCRATCH;
    uint8_t* part = workspace + kWsPart;
    a.parts = reinterpret_cast<float4*>(part);
    a.keys = reinterpret_cast<unsigned long long*>(part + rows * splits * 16);
    a.count = reinterpret_cast<unsigned*>(workspace + kWsCounters) + kCntBeam;
    if (type == QGKV_F32) return launch_beam<float>(a, requests, s);
    if (type == QGKV_F16) return launch_beam<__half>(a, requests, s);
    return launch_beam<__nv_bfloat16>(a, requests, s);
}

}  // namespace qg
