// Attention of sequences that share a prefix: what they have in common, and the
// join of the prefix's results with those of what is behind it.
//
// Mathematics.  The tokens of a row are those of the prefix and its own behind it.
// Each part gives its normalised result o, a reference m and the sum l of 2^(s - m);
// with m the larger of the two references and w = l 2^(m_i - m)
//   out = (w1 o1 + w2 o2) / (w1 + w2),   lse = (m + log2(w1 + w2)) / log2 e.
//
// The prefix is read once for all rows of its group: they are the rows of one
// sequence for it, whose queries all see every token.
#include "kv_attention.cuh"
#include "launch_common.cuh"
#include "qgkv_launch.h"

namespace qg {
namespace {

constexpr int kShareThreads = 512;

struct ShareArgs {
    const int32_t* table;
    int64_t width, pages, rows;
    int log2p;
    const int32_t* lens;
    const int32_t* starts;
    int batch;
    const int32_t* groups;
    int ngroups;
    int32_t* plan;
    unsigned* status;
};

// A CTA a group.  First the whole pages that every row of the group sees, then the
// columns in which all its sequences hold the same page.
__global__ void __launch_bounds__(kShareThreads) qg_share_kernel(const ShareArgs a) {
    __shared__ int least, same, first, busy, good;
    const int tid = threadIdx.x, g = blockIdx.x;
    const int g0 = a.groups[g], g1 = a.groups[g + 1];
    if (tid == 0) least = INT32_MAX, first = INT32_MAX, busy = 0, good = 1;
    __syncthreads();
    // the borders rise and lie in the batch, or nothing is shared anywhere
    for (int i = tid; i <= a.ngroups; i += kShareThreads) {
        const int x = a.groups[i], y = i < a.ngroups ? a.groups[i + 1] : a.batch;
        if (x < 0 || y < x || y > a.batch) good = 0;
    }
    __syncthreads();
    int32_t* skip = a.plan + 4 * static_cast<int64_t>(a.ngroups);
    const bool borders = good != 0;
    if (!borders) {
        if (tid == 0) atomicOr(a.status, kStatusBounds);
        if (tid < 4) a.plan[4 * g + tid] = 0;
        if (g == 0)
            for (int b = tid; b < a.batch; b += kShareThreads) skip[b] = 0;
        return;
    }
    if (g == 0)
        for (int b = tid; b < g0; b += kShareThreads) skip[b] = 0;
    if (g == a.ngroups - 1)
        for (int b = g1 + tid; b < a.batch; b += kShareThreads) skip[b] = 0;
    __syncthreads();  // every thread has read `good`
    // sequences with rows: how many, the first, and what the first row of each sees
    for (int b = g0 + tid; b < g1; b += kShareThreads) {
        int64_t n = 1;
        if (a.starts) {
            const int64_t r0 = a.starts[b], r1 = a.starts[b + 1];
            n = r1 - r0;
            if (r0 < 0 || n < 0 || r1 > a.rows) good = 0;  // the attention reports it
        }
        if (n <= 0) continue;
        const int64_t len = a.lens[b];
        if (len > a.width << a.log2p) good = 0;
        atomicMin(&least, static_cast<int>(max(int64_t(0), len - n + 1)));
        atomicMin(&first, b);
        atomicAdd(&busy, 1);
    }
    __syncthreads();
    const int f = first;
    const int64_t cols = good && busy > 1 ? least >> a.log2p : 0;
    if (tid == 0) same = static_cast<int>(cols);
    __syncthreads();
    if (cols > 0) {
        const int32_t* mine = a.table + f * a.width;
        const int members = g1 - f;
        const int64_t all = cols * members;
        for (int64_t i = tid; i < all; i += kShareThreads) {
            const int64_t m = i / cols;
            const int col = static_cast<int>(i - m * cols), b = f + static_cast<int>(m);
            const int page = mine[col];
            const bool differs = m == 0 ? page < 0 || page >= a.pages : a.table[b * a.width + col] != page;
            // a sequence without rows takes no part
            if (differs && !(a.starts && a.starts[b] == a.starts[b + 1])) atomicMin(&same, col);
        }
        __syncthreads();
    }
    const int tokens = same << a.log2p;
    if (tid == 0) {
        const int r0 = a.starts ? a.starts[g0] : g0, r1 = a.starts ? a.starts[g1] : g1;
        a.plan[4 * g] = good ? r0 : 0;
        a.plan[4 * g + 1] = good ? r1 - r0 : 0;
        a.plan[4 * g + 2] = tokens;
        a.plan[4 * g + 3] = f == INT32_MAX ? g0 : f;
    }
    for (int b = g0 + tid; b < g1; b += kShareThreads)
        skip[b] = a.starts && a.starts[b] == a.starts[b + 1] ? 0 : tokens;
}

// A CTA a row: all its heads.
struct JoinArgs {
    const float* o[2];
    const float2* ml[2];
    void* out;
    float* lse;
    const int4* groups;
    int ngroups, type, q_heads, dim;
    int64_t rows;
};

__global__ void __launch_bounds__(256) qg_shared_join_kernel(const JoinArgs a) {
    const int64_t row = blockIdx.x;
    bool mine = false;
    for (int g = threadIdx.x; g < a.ngroups; g += 256) {
        const int4 x = a.groups[g];
        mine |= x.z > 0 && row >= x.x && row < static_cast<int64_t>(x.x) + x.y;
    }
    if (!__syncthreads_or(mine)) return;
    const int per = a.dim / 4;
    for (int i = threadIdx.x; i < a.q_heads * per; i += 256) {
        const int h = i / per, d = (i - h * per) * 4;
        const int64_t at = row * a.q_heads + h;
        const float2 p = a.ml[0][at], q = a.ml[1][at];
        const float top = fmaxf(p.x, q.x), ref = top == -INFINITY ? 0.f : top;
        const float wp = exp2_fast(p.x - ref) * p.y, wq = exp2_fast(q.x - ref) * q.y;
        const float sum = wp + wq, inv = sum == 0.f ? 0.f : 1.f / sum;
        const float4 x = *reinterpret_cast<const float4*>(a.o[0] + at * a.dim + d);
        const float4 y = *reinterpret_cast<const float4*>(a.o[1] + at * a.dim + d);
        store_out4(a.out, a.type, at * a.dim + d,
                   make_float4((wp * x.x + wq * y.x) * inv, (wp * x.y + wq * y.y) * inv, (wp * x.z + wq * y.z) * inv,
                               (wp * x.w + wq * y.w) * inv));
        if (d == 0 && a.lse) a.lse[at] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
    }
}

}  // namespace

int launch_share(int64_t pages, int page_tokens, const int32_t* table, int64_t width, const int32_t* lens,
                 const int32_t* starts, int64_t rows, int batch, const int32_t* groups, int ngroups, int32_t* plan,
                 unsigned* status, cudaStream_t s) {
    ShareArgs a = {table, width, pages, rows, log2_of(page_tokens), lens, starts, batch, groups, ngroups, plan, status};
    qg_share_kernel<<<ngroups, kShareThreads, 0, s>>>(a);
    return launch_status();
}

int launch_attn_rows_shared(const AttnArgs& a, bool int8, cudaStream_t s);

// a: as for launch_attn_rows, with skip, own and own_ml of what is behind the prefix.
int launch_attn_shared(const AttnArgs& a, int groups, bool int8, cudaStream_t s) {
    const int64_t bytes = shared_bytes(a.rows, a.q_heads, a.c.dim), values = a.rows * a.q_heads * a.c.dim;
    AttnArgs first = a;
    first.prefix = true;
    first.batch = groups;
    first.own = reinterpret_cast<float*>(reinterpret_cast<uint8_t*>(a.own) + bytes);
    first.own_ml = reinterpret_cast<float2*>(first.own + values);
    int rc = launch_attn_rows_shared(first, int8, s);
    if (rc != QG_OK) return rc;
    rc = launch_attn_rows_shared(a, int8, s);
    if (rc != QG_OK) return rc;
    JoinArgs j = {{first.own, a.own}, {first.own_ml, a.own_ml}, a.out, a.lse, a.groups, groups, a.type, a.q_heads, a.c.dim, a.rows};
    qg_shared_join_kernel<<<static_cast<unsigned>(a.rows), 256, 0, s>>>(j);
    return launch_status();
}

}  // namespace qg
