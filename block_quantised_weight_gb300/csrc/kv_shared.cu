// What sequences of a group have in common: the whole pages at the head of their
// tables that all of them hold and every row sees.
//
// Bound.  Reads the shared part of the tables once; once a step of a decode, for
// all its layers: a chain of dependent loads (borders, starts and lengths, tables).
// A warp takes 128 columns of one table at a time; with a thread for each entry in
// turn, a 64-bit division for its place, 48 tables of 129 columns took 7.1 us, now
// 4.6, and 128 of them 14.5, now 7.7.  One group of 4 short tables 2.7 us.
#include "kv_common.cuh"
#include "launch_common.cuh"
#include "qgkv_launch.h"

namespace qg {
namespace {

constexpr int kShareThreads = 1024;
constexpr int kColumns = 4;  // a lane's, of a job of 128 columns of one table, on their way at once

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
        const int lane = tid & 31, pieces = static_cast<int>((cols + 32 * kColumns - 1) / (32 * kColumns));
        const int64_t jobs = static_cast<int64_t>(g1 - f) * pieces;
        for (int64_t j = tid >> 5; j < jobs; j += kShareThreads / 32) {
            const int m = static_cast<int>(j / pieces), b = f + m;
            const int c0 = static_cast<int>(j - static_cast<int64_t>(m) * pieces) * 32 * kColumns + lane;
            if (a.starts && a.starts[b] == a.starts[b + 1]) continue;  // a sequence without rows takes no part
            const int32_t* its = a.table + b * a.width;
            int32_t x[kColumns], y[kColumns];
#pragma unroll
            for (int i = 0; i < kColumns; ++i) {
                const int c = c0 + 32 * i;
                if (c < cols) x[i] = its[c], y[i] = mine[c];
            }
            int least_here = INT32_MAX;
#pragma unroll
            for (int i = kColumns - 1; i >= 0; --i) {
                const int c = c0 + 32 * i;
                if (c < cols && (m == 0 ? x[i] < 0 || x[i] >= a.pages : x[i] != y[i])) least_here = c;
            }
            if (least_here != INT32_MAX) atomicMin(&same, least_here);
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

}  // namespace

int launch_share(int64_t pages, int page_tokens, const int32_t* table, int64_t width, const int32_t* lens,
                 const int32_t* starts, int64_t rows, int batch, const int32_t* groups, int ngroups, int32_t* plan,
                 unsigned* status, cudaStream_t s) {
    ShareArgs a = {table, width, pages, rows, log2_of(page_tokens), lens, starts, batch, groups, ngroups, plan, status};
    qg_share_kernel<<<ngroups, kShareThreads, 0, s>>>(a);
    return launch_status();
}

}  // namespace qg
