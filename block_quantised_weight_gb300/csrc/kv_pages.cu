// Pages of the 8-bit cache: copies, forks (beam reordering with copy on
// write), compaction, reservation and freeing.
//
// A page is free when its reference count is 0, so there is no free list to
// keep: allocation takes the lowest free numbers, which makes every result a
// function of the inputs.  The counting passes read the reference counts in
// chunks of kChunk pages, one CTA each; the last CTA to arrive has the chunks'
// counts and does the planning that needs them, so that no kernel waits for
// another block.
//
// Bound.  A page moves as 2 * layers * heads * page_tokens * head_dim bytes
// of codes, read and written once: HBM-bound from a few dozen pages on; below
// that the chain of short launches counts.  Measured: compaction of 6000 pages, 16
// layers of 8 heads of 128: 204 us, 5.5 TB/s; of 700 pages, 4 layers: 13.7 us; fork
// of 48 x 5 beams over 22 layers 22.5 us, of 4 beams 10.6 us.
#include <atomic>

#include "kv_common.cuh"
#include "launch_common.cuh"
#include "qgkv_launch.h"

namespace qg {
namespace {

constexpr int kPlanThreads = 1024;
constexpr int kChunk = 4 * kPlanThreads;  // pages a CTA counts
static_assert(QGKV_MAX_PAGES / kChunk <= 4096, "chunk counts exceed the workspace");
// Up to this many chunks one CTA counts them all, in the launch before: about a
// microsecond a chunk, where a launch of its own costs two and more on the host.
constexpr int kMergeChunks = 4;

__device__ __forceinline__ int pages_of(int len, int log2p) { return (len + (1 << log2p) - 1) >> log2p; }

// The planning results lie in the workspace, so an index from there is checked
// like one from the caller: a workspace that was not zeroed before its first
// use gives wrong tables and QG_EBOUNDS, never an access outside an array.
__device__ __forceinline__ bool in_pages(int i, int64_t pages) { return i >= 0 && i < pages; }

// Length of row b cut to the table (kStatusBounds where it does not fit).
__device__ __forceinline__ int length_of(const int32_t* lens, int64_t b, int64_t width, int log2p, unsigned* status) {
    const int len = lens[b];
    const int64_t most = width << log2p;
    if (len >= 0 && len <= most) return len;
    atomicOr(status, kStatusBounds);
    return len < 0 ? 0 : static_cast<int>(most);
}

// Sum over a CTA of kPlanThreads; exclusive prefix in `before`.  red: 32 ints.
__device__ __forceinline__ int block_scan(int x, int& before, int* red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    int s = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, s, o);
        if (lane >= o) s += y;
    }
    __syncthreads();  // earlier readers of red are done
    if (lane == 31) red[warp] = s;
    __syncthreads();
    int w = red[lane];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(~0u, w, o);
        if (lane >= o) w += y;
    }
    const int below = warp ? __shfl_sync(~0u, w, warp - 1) : 0;
    before = below + s - x;
    return __shfl_sync(~0u, w, 31);
}

// The four counts of pages p .. p + 3 (pages from `pages` on read as `beyond`).
__device__ __forceinline__ int4 load4(const int32_t* refs, int64_t p, int64_t pages, int beyond) {
    if (p + 4 <= pages) return __ldcg(reinterpret_cast<const int4*>(refs + p));
    int4 r = make_int4(beyond, beyond, beyond, beyond);
    if (p < pages) r.x = __ldcg(refs + p);
    if (p + 1 < pages) r.y = __ldcg(refs + p + 1);
    if (p + 2 < pages) r.z = __ldcg(refs + p + 2);
    return r;
}
__device__ __forceinline__ void store4(int32_t* refs, int64_t p, int64_t pages, int4 r) {
    if (p + 4 <= pages) {
        *reinterpret_cast<int4*>(refs + p) = r;
        return;
    }
    if (p < pages) refs[p] = r.x;
    if (p + 1 < pages) refs[p + 1] = r.y;
    if (p + 2 < pages) refs[p + 2] = r.z;
}

// True in the last CTA of the grid to get here (all earlier writes visible).
__device__ __forceinline__ bool last_cta(unsigned* counter, int* flag) {
    __threadfence();
    __syncthreads();
    if (threadIdx.x == 0) {
        *flag = atomicAdd(counter, 1u) == gridDim.x - 1;
        if (*flag) *counter = 0u;
        __threadfence();
    }
    __syncthreads();
    return *flag != 0;
}

// ---------------------------------------------------------------- copies

struct CopyArgs {
    uint8_t* base[2];
    float* scale[2];
    int64_t layer_stride, page_stride, pages;
    int layers, heads, bytes;  // bytes of one page of one layer of K or V
    const int32_t* src;
    const int32_t* dst;
    const int32_t* count;
    int64_t most;
    unsigned* status;
};

constexpr int kCopyThreads = 256;
constexpr int kCopyVec = 4;  // 16-byte vectors a thread has in flight
constexpr int kCopyBytes = kCopyThreads * kCopyVec * 16;

__device__ __forceinline__ void copy_pages(const CopyArgs& a, int cta, int ctas) {
    int64_t n = a.most;
    if (a.count) n = min(n, static_cast<int64_t>(*a.count));
    const int parts = (a.bytes + kCopyBytes - 1) / kCopyBytes;
    const int64_t per = static_cast<int64_t>(a.layers) * 2 * parts;
    for (int64_t i = cta; i < n * per; i += ctas) {
        const int64_t pair = i / per;
        int r = static_cast<int>(i - pair * per);
        const int part = r % parts;
        r /= parts;
        const int which = r & 1, layer = r >> 1;
        const int64_t from = a.src[pair], to = a.dst[pair];
        if (from < 0 || to < 0 || from >= a.pages || to >= a.pages) {
            if (threadIdx.x == 0) atomicOr(a.status, kStatusBounds);
            continue;
        }
        uint8_t* base = a.base[which] + layer * a.layer_stride;
        const uint4* s = reinterpret_cast<const uint4*>(base + from * a.page_stride);
        uint4* d = reinterpret_cast<uint4*>(base + to * a.page_stride);
        const int first = part * (kCopyBytes / 16) + threadIdx.x, end = a.bytes / 16;
        uint4 x[kCopyVec];
#pragma unroll
        for (int j = 0; j < kCopyVec; ++j)
            if (first + j * kCopyThreads < end) x[j] = ldg_stream16(s + first + j * kCopyThreads);
#pragma unroll
        for (int j = 0; j < kCopyVec; ++j)
            if (first + j * kCopyThreads < end) d[first + j * kCopyThreads] = x[j];
        if (part == 0) {
            float* sc = a.scale[which] + static_cast<int64_t>(layer) * a.pages * a.heads;
            for (int h = threadIdx.x; h < a.heads; h += kCopyThreads)
                sc[to * a.heads + h] = sc[from * a.heads + h];
        }
    }
}

__global__ void __launch_bounds__(kCopyThreads) qg_copy_pages_kernel(const CopyArgs a) {
    copy_pages(a, blockIdx.x, gridDim.x);
}

// ---------------------------------------------------------------- fork

struct ForkArgs {
    const int32_t* table;
    const int32_t* lens;
    const int32_t* parent;
    const int32_t* refs;
    int64_t width, pages;
    int batch, batch2, log2p;
    int32_t* table2;
    int32_t* lens2;
    int32_t* refs2;
    int32_t* delta;
    int32_t* chunks;
    int32_t* src;
    int32_t* dst;
    int32_t* count;
    unsigned* counter;
    unsigned* status;
};

// Pages of one chunk: refs2 = refs + delta, delta back to 0; the chunk's free pages are counted.
__device__ __forceinline__ void fork_count(const ForkArgs& a, int chunk, int* red) {
    const int64_t p = static_cast<int64_t>(chunk) * kChunk + threadIdx.x * 4;
    int4 r = load4(a.refs, p, a.pages, 1);
    const int4 d = load4(a.delta, p, a.pages, 0);
    if (d.x | d.y | d.z | d.w) store4(a.delta, p, a.pages, make_int4(0, 0, 0, 0));
    r.x += d.x, r.y += d.y, r.z += d.z, r.w += d.w;
    store4(a.refs2, p, a.pages, r);
    int before;
    const int zeros = block_scan((r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0), before, red);
    if (threadIdx.x == 0) a.chunks[chunk] = zeros;
}

// Who needs a page of its own gets the lowest free ones.  One CTA; smem: tail,
// list and holders [batch2].
__device__ __forceinline__ void fork_plan(const ForkArgs& a, int32_t* smem, int* red) {
    const int tid = threadIdx.x;
    const int padded = (a.batch2 + 3) & ~3;
    int32_t* tail = smem;
    int32_t* list = smem + padded;
    int32_t* holders = list + padded;  // references of the tail
    if (tid < padded - a.batch2) tail[a.batch2 + tid] = -2;
    // the partly filled last page of each new sequence, -1 where it has none
    for (int i = tid; i < a.batch2; i += kPlanThreads) {
        const int len = __ldcg(a.lens2 + i);
        const int id = (len & ((1 << a.log2p) - 1)) ? __ldcg(a.table2 + i * a.width + (len >> a.log2p)) : -1;
        const bool there = id >= 0 && id < a.pages;
        tail[i] = there ? id : -1;
        holders[i] = there ? __ldcg(a.refs2 + id) : 0;
    }
    __syncthreads();
    // who needs a copy: a lower sequence has the same last page, or someone
    // outside holds it too
    for (int i = tid; i < a.batch2; i += kPlanThreads) {
        const int mine = tail[i];
        int same = 0, first = a.batch2;
#pragma unroll 4
        for (int j = 0; j < a.batch2; j += 4) {  // padded to whole fours
            const int4 t = *reinterpret_cast<const int4*>(tail + j);
            const int n = (t.x == mine) + (t.y == mine) + (t.z == mine) + (t.w == mine);
            if (n && first == a.batch2) first = t.x == mine ? j : t.y == mine ? j + 1 : t.z == mine ? j + 2 : j + 3;
            same += n;
        }
        list[i] = mine >= 0 && (first < i || holders[i] > same) ? 1 : 0;
    }
    __syncthreads();
    // their ranks; the list then holds the sequences
    int needed = 0;
    for (int i0 = 0; i0 < a.batch2; i0 += kPlanThreads) {
        const int i = i0 + tid;
        const int copy = i < a.batch2 ? list[i] : 0;
        int before;
        const int sum = block_scan(copy, before, red);  // every flag of this round has been read
        if (copy) {
            a.src[needed + before] = tail[i];
            list[needed + before] = i;
        }
        needed += sum;
    }
    __syncthreads();
    // the lowest free pages, chunk by chunk
    int given = 0;
    for (int ch = 0; given < needed && ch * static_cast<int64_t>(kChunk) < a.pages; ++ch) {
        if (__ldcg(a.chunks + ch) == 0) continue;
        const int64_t p = static_cast<int64_t>(ch) * kChunk + tid * 4;
        const int4 r = load4(a.refs2, p, a.pages, 1);
        int at;
        const int zeros = block_scan((r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0), at, red);
        at += given;
        const int v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (v[j] == 0) {
                if (at < needed) a.dst[at] = static_cast<int32_t>(p + j);
                ++at;
            }
        given += zeros;
    }
    __syncthreads();
    const int granted = min(given, needed);
    if (tid == 0) {
        *a.count = granted;
        if (granted < needed) atomicOr(a.status, kStatusPages);
    }
    for (int k = tid; k < needed; k += kPlanThreads) {
        const int i = list[k];
        const int from = a.src[k];
        const int to = k < granted ? a.dst[k] : -1;
        a.table2[i * a.width + (__ldcg(a.lens2 + i) >> a.log2p)] = to;
        atomicSub(a.refs2 + from, 1);
        if (to >= 0) a.refs2[to] = 1;
    }
}

// CTAs 0 .. batch-1: an old sequence's pages gain (children - 1) references.
// The others: a new sequence's table row and length.  With few pages (`merged`)
// the last CTA to end also counts and plans, which saves a launch; with many
// the counting is spread over CTAs of its own (qg_fork_plan_kernel).
__global__ void __launch_bounds__(kPlanThreads) qg_fork_rows_kernel(const ForkArgs a, int merged) {
    extern __shared__ __align__(16) int32_t smem[];
    __shared__ int children;
    __shared__ int red[32];
    __shared__ int flag;
    if (static_cast<int>(blockIdx.x) < a.batch) {
        const int r = blockIdx.x;
        if (threadIdx.x == 0) children = 0;
        __syncthreads();
        int mine = 0;
        for (int i = threadIdx.x; i < a.batch2; i += blockDim.x) mine += a.parent[i] == r ? 1 : 0;
        if (mine) atomicAdd(&children, mine);
        __syncthreads();
        const int change = children - 1;
        const int n = change ? pages_of(length_of(a.lens, r, a.width, a.log2p, a.status), a.log2p) : 0;
        for (int j = threadIdx.x; j < n; j += blockDim.x) {
            const int id = a.table[r * a.width + j];
            if (id >= 0 && id < a.pages) atomicAdd(a.delta + id, change);
            else atomicOr(a.status, kStatusBounds);
        }
    } else {
        const int i = blockIdx.x - a.batch;
        const int p = a.parent[i];
        const bool ok = p >= 0 && p < a.batch;
        if (!ok && threadIdx.x == 0) atomicOr(a.status, kStatusBounds);
        const int len = ok ? length_of(a.lens, p, a.width, a.log2p, a.status) : 0;
        const int n = pages_of(len, a.log2p);
        for (int64_t j = threadIdx.x; j < a.width; j += blockDim.x)
            a.table2[i * a.width + j] = j < n ? a.table[p * a.width + j] : -1;
        if (threadIdx.x == 0) a.lens2[i] = len;
    }
    if (!merged || !last_cta(a.counter, &flag)) return;
    for (int ch = 0; ch * static_cast<int64_t>(kChunk) < a.pages; ++ch) fork_count(a, ch, red);
    __syncthreads();
    fork_plan(a, smem, red);
}

// A CTA counts a chunk; the last plans.
__global__ void __launch_bounds__(kPlanThreads) qg_fork_plan_kernel(const ForkArgs a) {
    extern __shared__ __align__(16) int32_t smem[];
    __shared__ int red[32];
    __shared__ int flag;
    fork_count(a, blockIdx.x, red);
    if (last_cta(a.counter, &flag)) fork_plan(a, smem, red);
}

// ---------------------------------------------------------------- compact

struct CompactArgs {
    const int32_t* table;
    const int32_t* lens;
    const uint8_t* drop;
    const int32_t* refs;
    int64_t width, pages;
    int batch, log2p;
    int32_t* table2;
    int32_t* lens2;
    int32_t* refs2;
    int32_t* count;
    int32_t* delta;
    int32_t* now;     // counts after the drops
    int32_t* holes;
    int32_t* movers;
    int32_t* rank;
    int32_t* chunks;  // pages held below each chunk
    int32_t* scalars; // n, held pages below n, moves
    unsigned* counter;
    unsigned* status;
};

// A dropped sequence's pages lose a reference.
__device__ __forceinline__ void drop_row(const CompactArgs& a, int b) {
    if (!a.drop || !a.drop[b]) return;
    const int n = pages_of(length_of(a.lens, b, a.width, a.log2p, a.status), a.log2p);
    for (int j = threadIdx.x; j < n; j += blockDim.x) {
        const int id = a.table[b * a.width + j];
        if (id >= 0 && id < a.pages) atomicAdd(a.delta + id, -1);
        else atomicOr(a.status, kStatusBounds);
    }
}

// Pages of one chunk: counts after the drops, delta back to 0, pages held.
__device__ __forceinline__ void compact_count(const CompactArgs& a, int chunk, int* red) {
    const int64_t p = static_cast<int64_t>(chunk) * kChunk + threadIdx.x * 4;
    int4 r = load4(a.refs, p, a.pages, 0);
    const int4 d = load4(a.delta, p, a.pages, 0);
    if (d.x | d.y | d.z | d.w) store4(a.delta, p, a.pages, make_int4(0, 0, 0, 0));
    r.x += d.x, r.y += d.y, r.z += d.z, r.w += d.w;
    store4(a.now, p, a.pages, r);
    int before;
    const int held = block_scan((r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0), before, red);
    if (threadIdx.x == 0) a.chunks[chunk] = held;
}

// One CTA: n, the pages held below each chunk, and how many of them lie below n.
__device__ __forceinline__ void compact_total(const CompactArgs& a, int chunks, int* red) {
    const int tid = threadIdx.x;
    const int mine = tid < chunks ? __ldcg(a.chunks + tid) : 0;  // at most 256 chunks
    int before;
    const int n = block_scan(mine, before, red);
    if (tid < chunks) a.chunks[tid] = before;
    __syncthreads();
    const int ch = min(n / kChunk, chunks - 1);  // the chunk that n lies in
    const int64_t p = static_cast<int64_t>(ch) * kChunk + tid * 4;
    const int4 r = load4(a.now, p, a.pages, 0);
    int x;
    const int below = block_scan((r.x > 0 && p < n) + (r.y > 0 && p + 1 < n) + (r.z > 0 && p + 2 < n) +
                                     (r.w > 0 && p + 3 < n), x, red);
    if (tid == 0) {
        const int held_below = a.chunks[ch] + below;
        a.scalars[0] = n;
        a.scalars[1] = held_below;
        a.scalars[2] = n - held_below;
        *a.count = n;
    }
    __syncthreads();
}

// The holes below n and the held pages from n on, each in order.
__device__ __forceinline__ void compact_list(const CompactArgs& a, int chunk, int* red) {
    const int n = __ldcg(a.scalars), held_below = __ldcg(a.scalars + 1);
    const int64_t p = static_cast<int64_t>(chunk) * kChunk + threadIdx.x * 4;
    const int4 r = load4(a.now, p, a.pages, 0);
    int at;
    block_scan((r.x > 0) + (r.y > 0) + (r.z > 0) + (r.w > 0), at, red);
    at += __ldcg(a.chunks + chunk);  // held pages below p
    const int v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const int q = static_cast<int>(p + j);
        if (q >= a.pages) break;
        if (q < n) {
            if (v[j] > 0) a.refs2[q] = v[j];
            else if (in_pages(q - at, a.pages)) a.holes[q - at] = q;
            else atomicOr(a.status, kStatusBounds);
        } else {
            a.refs2[q] = 0;
            if (v[j] > 0) {
                const int i = at - held_below;
                a.rank[q] = i;
                if (in_pages(i, a.pages)) a.movers[i] = q;
                else atomicOr(a.status, kStatusBounds);
            }
        }
        at += v[j] > 0 ? 1 : 0;
    }
}

// Few pages: the drops, then all the counting in the last CTA to end.
__global__ void __launch_bounds__(kPlanThreads) qg_compact_plan_kernel(const CompactArgs a) {
    __shared__ int red[32];
    __shared__ int flag;
    drop_row(a, blockIdx.x);
    if (!last_cta(a.counter, &flag)) return;
    const int chunks = static_cast<int>((a.pages + kChunk - 1) / kChunk);
    for (int ch = 0; ch < chunks; ++ch) compact_count(a, ch, red);
    __syncthreads();
    compact_total(a, chunks, red);
    for (int ch = 0; ch < chunks; ++ch) compact_list(a, ch, red);
}

// Many pages: the same in three launches, a CTA a chunk.
__global__ void __launch_bounds__(256) qg_drop_rows_kernel(const CompactArgs a) { drop_row(a, blockIdx.x); }

__global__ void __launch_bounds__(kPlanThreads) qg_compact_count_kernel(const CompactArgs a) {
    __shared__ int red[32];
    __shared__ int flag;
    compact_count(a, blockIdx.x, red);
    if (last_cta(a.counter, &flag)) compact_total(a, gridDim.x, red);
}

__global__ void __launch_bounds__(kPlanThreads) qg_compact_list_kernel(const CompactArgs a) {
    __shared__ int red[32];
    compact_list(a, blockIdx.x, red);
}

// CTAs 0 .. batch-1: a table row; then a few for the counts of the filled
// holes; the others copy the pages.
__global__ void __launch_bounds__(kCopyThreads) qg_compact_move_kernel(const CompactArgs a, const CopyArgs copy, int ref_ctas) {
    const int n = a.scalars[0], moves = a.scalars[2];
    if (static_cast<int>(blockIdx.x) < a.batch) {
        const int b = blockIdx.x;
        const bool gone = a.drop && a.drop[b];
        const int len = gone ? 0 : length_of(a.lens, b, a.width, a.log2p, a.status);
        const int held = pages_of(len, a.log2p);
        for (int64_t j = threadIdx.x; j < a.width; j += blockDim.x) {
            int to = -1;
            if (j < held) {
                const int id = a.table[b * a.width + j];
                if (in_pages(id, a.pages) && a.now[id] > 0) {
                    if (id < n) to = id;
                    else if (in_pages(a.rank[id], a.pages)) to = a.holes[a.rank[id]];
                }
                if (to < 0) atomicOr(a.status, kStatusBounds);
            }
            a.table2[b * a.width + j] = to;
        }
        if (threadIdx.x == 0) a.lens2[b] = len;
    } else if (static_cast<int>(blockIdx.x) < a.batch + ref_ctas) {
        for (int64_t i = (blockIdx.x - a.batch) * blockDim.x + threadIdx.x; i < moves && i < a.pages;
             i += ref_ctas * blockDim.x) {
            const int to = a.holes[i], from = a.movers[i];
            if (in_pages(to, a.pages) && in_pages(from, a.pages)) a.refs2[to] = a.now[from];
            else atomicOr(a.status, kStatusBounds);
        }
    } else {
        copy_pages(copy, blockIdx.x - a.batch - ref_ctas, gridDim.x - a.batch - ref_ctas);
    }
}

// ---------------------------------------------------------------- reserve, free

struct ReserveArgs {
    int32_t* table;
    const int32_t* lens;
    const int32_t* add;
    int32_t* refs;
    int64_t width, pages;
    int batch, log2p;
    int32_t* chunks;
    unsigned* counter;
    unsigned* status;
};

__global__ void __launch_bounds__(kPlanThreads) qg_reserve_kernel(const ReserveArgs a) {
    extern __shared__ uint32_t pre[];  // [batch + 1] pages given to the sequences before, modulo 2^32
    __shared__ int red[32];
    __shared__ int flag;
    const int tid = threadIdx.x;
    {
        const int64_t p = static_cast<int64_t>(blockIdx.x) * kChunk + tid * 4;
        const int4 r = load4(a.refs, p, a.pages, 1);
        int before;
        const int zeros = block_scan((r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0), before, red);
        if (tid == 0) a.chunks[blockIdx.x] = zeros;
    }
    if (!last_cta(a.counter, &flag)) return;
    // Up to 4096 sequences may ask for up to 2^20 pages each: their sum takes 33
    // bits (that of the 1024 of one round 30).
    int64_t base = 0;
    for (int b0 = 0; b0 < a.batch; b0 += kPlanThreads) {
        const int b = b0 + tid;
        int need = 0;
        if (b < a.batch) {
            const int len = length_of(a.lens, b, a.width, a.log2p, a.status);
            const int64_t end = static_cast<int64_t>(len) + (a.add ? max(a.add[b], 0) : 1);
            const int64_t last = (end + (1 << a.log2p) - 1) >> a.log2p;
            if (last > a.width) atomicOr(a.status, kStatusBounds);
            else need = static_cast<int>(last) - pages_of(len, a.log2p);
        }
        int before;
        const int sum = block_scan(need, before, red);
        if (b < a.batch) pre[b + 1] = static_cast<uint32_t>(base) + before + need;
        base += sum;
    }
    if (tid == 0) pre[0] = 0;
    int x;
    const int avail = block_scan(tid < static_cast<int>(gridDim.x) ? __ldcg(a.chunks + tid) : 0, x, red);
    __syncthreads();
    if (base > avail) {  // one after the other: who does not fit gets none
        if (tid == 0) {
            int given = 0;
            uint32_t was = 0;
            for (int b = 0; b < a.batch; ++b) {
                const int need = static_cast<int>(pre[b + 1] - was);
                was = pre[b + 1];
                if (given + need <= avail) given += need;
                pre[b + 1] = given;
            }
            atomicOr(a.status, kStatusPages);
        }
        __syncthreads();
    }
    const int needed = static_cast<int>(pre[a.batch]);  // at most avail from here on
    int given = 0;
    for (int ch = 0; given < needed && ch < static_cast<int>(gridDim.x); ++ch) {
        const int in_chunk = __ldcg(a.chunks + ch);
        if (in_chunk == 0) continue;
        const int64_t p = static_cast<int64_t>(ch) * kChunk + tid * 4;
        const int4 r = load4(a.refs, p, a.pages, 1);
        int at;
        block_scan((r.x == 0) + (r.y == 0) + (r.z == 0) + (r.w == 0), at, red);
        at += given;
        const int v[4] = {r.x, r.y, r.z, r.w};
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (v[j] == 0) {
                if (at < needed) {
                    int lo = 0, hi = a.batch;  // the sequence whose share `at` lies in
                    while (hi - lo > 1) {
                        const int mid = (lo + hi) >> 1;
                        if (pre[mid] <= static_cast<uint32_t>(at)) lo = mid; else hi = mid;
                    }
                    const int len = length_of(a.lens, lo, a.width, a.log2p, a.status);
                    a.table[lo * a.width + pages_of(len, a.log2p) + (at - static_cast<int>(pre[lo]))] = static_cast<int32_t>(p + j);
                    a.refs[p + j] = 1;
                }
                ++at;
            }
        given += in_chunk;
    }
}

struct FreeArgs {
    int32_t* table;
    int32_t* lens;
    const uint8_t* drop;
    int32_t* refs;
    int64_t width, pages;
    int log2p;
    unsigned* status;
};

__global__ void __launch_bounds__(256) qg_free_kernel(const FreeArgs a) {
    const int b = blockIdx.x;
    if (a.drop && !a.drop[b]) return;
    const int n = pages_of(length_of(a.lens, b, a.width, a.log2p, a.status), a.log2p);
    for (int64_t j = threadIdx.x; j < a.width; j += blockDim.x) {
        if (j < n) {
            const int id = a.table[b * a.width + j];
            if (id >= 0 && id < a.pages) atomicSub(a.refs + id, 1);
            else atomicOr(a.status, kStatusBounds);
        }
        a.table[b * a.width + j] = -1;
    }
    __syncthreads();
    if (threadIdx.x == 0) a.lens[b] = 0;
}

template <class T>
T* at(uint8_t* ws, int64_t off) { return reinterpret_cast<T*>(ws + off); }

int plan_smem(const void* kern, int bytes, std::atomic<int>* done, int dev) {
    if (done[dev].load(std::memory_order_acquire)) return QG_OK;
    if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess)
        return cuda_fail(cudaGetLastError());
    done[dev].store(1, std::memory_order_release);
    return QG_OK;
}

}  // namespace

namespace {
CopyArgs copy_args(const qgkv_cache& c, const int32_t* src, const int32_t* dst, const int32_t* count, int64_t most,
                   unsigned* status) {
    CopyArgs a = {};
    a.base[0] = c.k, a.base[1] = c.v, a.scale[0] = c.k_scale, a.scale[1] = c.v_scale;
    a.layer_stride = c.layer_stride, a.page_stride = c.page_stride, a.pages = c.pages;
    a.layers = static_cast<int>(c.layers), a.heads = c.heads;
    a.bytes = c.heads * c.page_tokens * c.head_dim;
    a.src = src, a.dst = dst, a.count = count, a.most = most, a.status = status;
    return a;
}

// Eight CTAs an SM, or one for each piece there can be.
int copy_ctas(const CopyArgs& a, int sms) {
    const int64_t items = a.most * a.layers * 2 * ((a.bytes + kCopyBytes - 1) / kCopyBytes);
    return static_cast<int>(std::min<int64_t>(items, static_cast<int64_t>(sms) * 8));
}
}  // namespace

int launch_copy_pages(const qgkv_cache& c, const int32_t* src, const int32_t* dst, const int32_t* count, int64_t most,
                      unsigned* status, cudaStream_t s) {
    const CopyArgs a = copy_args(c, src, dst, count, most, status);
    const int sms = sm_count(current_device());
    if (sms <= 0) return cuda_fail(cudaGetLastError());
    qg_copy_pages_kernel<<<copy_ctas(a, sms), kCopyThreads, 0, s>>>(a);
    return launch_status();
}

int launch_fork(const qgkv_cache& c, const int32_t* table, int64_t width, const int32_t* lens, int batch,
                const int32_t* parent, int batch2, const int32_t* refs, int32_t* table2, int32_t* lens2,
                int32_t* refs2, uint8_t* ws, unsigned* status, cudaStream_t s) {
    const int dev = current_device();
    if (dev < 0) return cuda_fail(cudaGetLastError());
    static std::atomic<int> done[64];
    static std::atomic<int> done_rows[64];
    int rc = plan_smem(reinterpret_cast<const void*>(qg_fork_plan_kernel), (QGKV_MAX_BATCH + 4) * 12, done, dev);
    if (rc != QG_OK) return rc;
    rc = plan_smem(reinterpret_cast<const void*>(qg_fork_rows_kernel), (QGKV_MAX_BATCH + 4) * 12, done_rows, dev);
    if (rc != QG_OK) return rc;
    ForkArgs a = {};
    a.table = table, a.lens = lens, a.parent = parent, a.refs = refs, a.width = width, a.pages = c.pages;
    a.batch = batch, a.batch2 = batch2, a.log2p = log2_of(c.page_tokens);
    a.table2 = table2, a.lens2 = lens2, a.refs2 = refs2, a.status = status;
    a.delta = at<int32_t>(ws, kWsDelta), a.chunks = at<int32_t>(ws, kWsChunks);
    a.src = at<int32_t>(ws, kWsMovers), a.dst = at<int32_t>(ws, kWsHoles);
    a.count = at<int32_t>(ws, kWsScalars), a.counter = at<unsigned>(ws, kWsCounters) + kCntPages;
    const int chunks = static_cast<int>((c.pages + kChunk - 1) / kChunk);
    const bool merged = chunks <= kMergeChunks;
    const int smem = (batch2 + 4) * 12;
    qg_fork_rows_kernel<<<batch + batch2, merged ? kPlanThreads : 256, merged ? smem : 0, s>>>(a, merged);
    if (!merged) qg_fork_plan_kernel<<<chunks, kPlanThreads, smem, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e);
    return launch_copy_pages(c, a.src, a.dst, a.count, batch2, status, s);
}

int launch_compact(const qgkv_cache& c, const int32_t* table, int64_t width, const int32_t* lens, int batch,
                   const uint8_t* drop, const int32_t* refs, int32_t* table2, int32_t* lens2, int32_t* refs2,
                   int32_t* count, uint8_t* ws, unsigned* status, cudaStream_t s) {
    CompactArgs a = {};
    a.table = table, a.lens = lens, a.drop = drop, a.refs = refs, a.width = width, a.pages = c.pages;
    a.batch = batch, a.log2p = log2_of(c.page_tokens);
    a.table2 = table2, a.lens2 = lens2, a.refs2 = refs2, a.count = count, a.status = status;
    a.delta = at<int32_t>(ws, kWsDelta), a.now = at<int32_t>(ws, kWsRefs), a.holes = at<int32_t>(ws, kWsHoles);
    a.movers = at<int32_t>(ws, kWsMovers), a.rank = at<int32_t>(ws, kWsRank), a.chunks = at<int32_t>(ws, kWsChunks);
    a.scalars = at<int32_t>(ws, kWsScalars), a.counter = at<unsigned>(ws, kWsCounters) + kCntPages;
    const int chunks = static_cast<int>((c.pages + kChunk - 1) / kChunk);
    if (chunks <= kMergeChunks) {
        qg_compact_plan_kernel<<<drop ? batch : 1, kPlanThreads, 0, s>>>(a);
    } else {
        if (drop) qg_drop_rows_kernel<<<batch, 256, 0, s>>>(a);
        qg_compact_count_kernel<<<chunks, kPlanThreads, 0, s>>>(a);
        qg_compact_list_kernel<<<chunks, kPlanThreads, 0, s>>>(a);
    }
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return cuda_fail(e);
    const CopyArgs copy = copy_args(c, a.movers, a.holes, a.scalars + 2, c.pages, status);
    const int sms = sm_count(current_device());
    if (sms <= 0) return cuda_fail(cudaGetLastError());
    const int ref_ctas = static_cast<int>((c.pages + 4095) / 4096);
    qg_compact_move_kernel<<<batch + ref_ctas + copy_ctas(copy, sms), kCopyThreads, 0, s>>>(a, copy, ref_ctas);
    return launch_status();
}

int launch_reserve(int64_t pages, int page_tokens, int32_t* table, int64_t width, const int32_t* lens,
                   const int32_t* add, int batch, int32_t* refs, uint8_t* ws, unsigned* status, cudaStream_t s) {
    ReserveArgs a = {};
    a.table = table, a.lens = lens, a.add = add, a.refs = refs, a.width = width, a.pages = pages;
    a.batch = batch, a.log2p = log2_of(page_tokens), a.status = status;
    a.chunks = at<int32_t>(ws, kWsChunks), a.counter = at<unsigned>(ws, kWsCounters) + kCntPages;
    const int chunks = static_cast<int>((pages + kChunk - 1) / kChunk);
    qg_reserve_kernel<<<chunks, kPlanThreads, (batch + 1) * 4, s>>>(a);
    return launch_status();
}

int launch_free(int64_t pages, int page_tokens, int32_t* table, int64_t width, int32_t* lens, const uint8_t* drop,
                int batch, int32_t* refs, unsigned* status, cudaStream_t s) {
    FreeArgs a = {};
    a.table = table, a.lens = lens, a.drop = drop, a.refs = refs, a.width = width, a.pages = pages;
    a.log2p = log2_of(page_tokens), a.status = status;
    qg_free_kernel<<<batch, 256, 0, s>>>(a);
    return launch_status();
}

}  // namespace qg
