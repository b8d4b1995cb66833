// Attention over a prefix that sequences share: all rows of a group over the
// same tokens, each read once, on the tcgen05 tensor cores.
//
// Mathematics: kv_rows.cuh's, with both products transposed.  A CTA takes up to 64 (32 from 129 dims on)
// query rows (tokens x heads of a group, a multiple of 16) of one cache head and
// walks the keys in steps of 128:
//   S^T = K q^T     128 keys x rows, in tensor memory
//   e = 2^(S f - m + k), f = scale * ks,   z = e * vs as f16, in shared memory
//   O^T += V^T z    dims x rows, in tensor memory,   l += e
// A group has as many rows as its sequences have heads and tokens, from 8 to
// hundreds, the keys are always many: with the keys on the 128 rows of the MMA its
// columns follow the number of rows, and neither operand of the cache has to be
// transposed: K goes to tensor memory key by key, V to shared memory as it lies (M-major).
// A thread has one key and 16 columns: the key's scales are scalars of the thread, and what
// belongs to a query row (factor, references) comes from shared memory, four at a
// time.  References are whole numbers, shared by the four warps that hold the
// keys; they are set in a piece's first step, so that z is at most 2^6 (k = 6 less
// the order of p * vs), and move only when a z would pass 2^15: 16 columns are tried
// as if they held, one vote of the four warps decides.  Scores from 2^22 on take a
// slower way.  Two parts of z: the second is
// 2^11 times what the first leaves, with sums of its own, so that small weights keep
// their bits down to 2^-40 of a row's largest (one part: 2^-29).
//
// Bound.  The chain of a step's softmax (scores out of tensor memory, the vote, weights to shared memory): 2000 of 2800
// clocks at 64 rows of 128 dims, in a profile with the tensor pipe busy for 11 % of the time, DRAM for 14 % and 41 % of
// the issue slots.  Copies, codes and both products' operands move 190 KB of shared memory a step, 1500 clocks by
// its width, beside it.  Steps of fewer rows take as long.  832 threads leave 72 registers, at which all forms spill: 24 to
// 72 bytes of stores a thread up to 128 dims, 72 (bf16 q) to 528 (fp32) above.  Short calls are bound by the chain
// plan -> table -> codes -> first step, and by the parts that are left to join.
//
// Measured (GB300, us a layer with the rows behind the prefix; each for itself in brackets): 48 sequences of 600
// tokens behind 8200, 32 / 8 heads of 128, e4m3: bf16 43 (97), fp16 45 (105), fp32 47 (113), int8 codes 55 (149); 8 of
// them 20 (28), 128 of them 101 (237); 32 behind two prefixes of 65536, int8: 103 (575).  About 6 us to a CTA's first
// step, 1.5 a step of 64 rows, 2 behind the last.  With K as f16 in shared memory and eight softmax
// warps the first of them took 51 where it then took 46.
//
// Split.  Each unit (group, head, row block) is cut into parts, as long as lets every CTA
// have one (a piece costs as much as some steps before its first and behind its
// last), and the parts are one line, cut evenly among the CTAs.  A piece that begins a unit
// leaves its result for each row, the others in a slot of their CTA; the row
// kernel adds them to what lies behind the prefix (own_ml of a row names its group, the CTA of
// the first further piece and their number).
//
// Roles: sixteen warps for the softmax (a set of four has the keys, and 16 columns),
// four convert K, four V, one copies, one issues the MMAs.
#pragma once
#include <atomic>

#include "kv_attention.cuh"
#include "kv_tc.cuh"
#include "launch_common.cuh"

namespace qg {
namespace {

constexpr int kKeys = 128;
constexpr int kLeastSteps = 2;      // of a part
constexpr uint32_t kUnitsAhead = 2; // pieces handed to the roles ahead
constexpr uint32_t kScaleSteps = 8; // steps whose scales are held
constexpr int64_t kPrefetchBytes = int64_t(64) << 20;  // half of L2
constexpr int kMostE = 90;
constexpr int kBase = 6;             // of k: z is at most 2^6 under new references, and may grow to 2^15
constexpr int kSets = 4;             // of four softmax warps, 16 columns each
// warps by role: the softmax, then four that convert K, four that convert V, one that copies, one that issues the MMAs
constexpr int kSoftmaxWarps = 4 * kSets, kKeyWarp = kSoftmaxWarps, kValueWarp = kKeyWarp + 4, kCopyWarp = kValueWarp + 4;
constexpr int kMmaWarp = kCopyWarp + 1, kPrefixThreads = (kMmaWarp + 1) * 32;

template <int DP, int QP, int PP>
struct XShape {
    static constexpr int NMAX = prefix_rows(DP);
    static constexpr int NP = 64;                     // columns of the second product: a whole swizzle atom
    // Buffers of S^T, and of z, as shared memory has room: with three the sets of warps drift apart, and one's
    // waits are the others' time.
    static constexpr uint32_t SB = PP == 1 || DP == 64 ? 3 : 2, PB = SB == 3 ? 3 : 1;
    static constexpr int DA = DP == 256 ? 2 : 1;      // accumulators of 128 dims
    static constexpr int kQPart = NMAX * DP * 2;
    static constexpr int kPPart = kKeys * NP * 2;
    static constexpr int kOp = kKeys * DP * 2;        // V as f16
    static constexpr int RW = DP < 128 ? DP : 128;    // bytes of a raw row
    static constexpr int RT = DP / RW;                // raw tiles of an operand
    static constexpr int kRaw = kKeys * RW;
    static constexpr uint32_t kOps = DP == 256 ? 1 : 2;
    static constexpr int off_p = QP * kQPart;
    static constexpr int off_op = off_p + static_cast<int>(PB) * PP * kPPart;
    static constexpr int off_raw = off_op + static_cast<int>(kOps) * kOp;
    static constexpr int kExtra = 12 * 1024;          // what stands behind the raw slots
    static constexpr int kFit = (232448 - kExtra - off_raw) / kRaw;
    static constexpr uint32_t kRaws = kFit < 8 ? kFit : 8;          // of K, then of V
    static constexpr uint32_t kRawK = (kRaws + 1) / 2, kRawV = kRaws / 2;
    // a ring holds a step, whose scales are posted behind its copies of K
    static_assert(kRawV >= RT && kRawK >= RT, "shared memory");
    static_assert(kOps + kRawV / RT < kScaleSteps, "scales are written while they are read");
    // tensor memory: S^T, O^T (DA of NP for each part of z), K as f16 once or twice
    static constexpr int o_at = static_cast<int>(SB) * NMAX, k_at = o_at + PP * DA * NP;
    static constexpr uint32_t KB = (512 - k_at) / (DP / 2) >= 2 ? 2 : 1;
    static_assert(k_at + static_cast<int>(KB) * DP / 2 <= 512, "tensor memory");
    static constexpr int off_scale = off_raw + static_cast<int>(kRaws) * kRaw;
    static constexpr int off_cols = off_scale + static_cast<int>(kScaleSteps) * 8 * 16;
    static constexpr int off_bar = off_cols + NMAX * (7 * 4 + 8 * 4 + 8);  // Columns
    static constexpr int smem = off_bar + 512;
    static_assert(smem <= 232448 && off_cols % 16 == 0 && off_bar % 8 == 0, "shared memory");
};

struct PrefixPiece {
    int row0, nrows, h, row_first, nc, table_row, j0, j1;
    int slot;   // -1: begins its unit
    int extra;  // further pieces of a unit that this one begins, its group << 16
    int tokens; // of the prefix; < 0: no more pieces
};

// A group's units (heads x row blocks), each cut into `parts` parts of nearly equal length.
struct Units {
    int n, steps, parts, per, blocks;  // per: rows of a block
};
template <int NMAX>
__device__ __forceinline__ Units units_of(const AttnArgs& a, const SharedGroup& g) {
    Units u = {};
    if (g.tokens == 0) return u;
    const unsigned rows = static_cast<unsigned>(g.n) * a.group, most = (rows + NMAX - 1) / NMAX;
    u.per = ((rows + most - 1) / most + 15) / 16 * 16;
    u.blocks = (rows + u.per - 1) / u.per;
    u.n = u.blocks * a.c.heads;
    u.steps = static_cast<int>((static_cast<unsigned>(g.tokens) + kKeys - 1) / kKeys);
    return u;
}

// The line of all parts.  A lane has every 32nd group; a part is found by a whole warp, forward only.
template <int NMAX>
struct PartWalk {
    int b0 = -32;
    SharedGroup g;
    Units u;
    float steps, longest;              // of all units; of a part
    int base = 0, chunk = 0, upto = 0; // parts
    __device__ void load(const AttnArgs& a, int from) {
        b0 = from;
        g = SharedGroup{};
        const int b = b0 + static_cast<int>(threadIdx.x & 31);
        if (b < a.ngroups) g = shared_group(a, a.groups[b], group_before(a, b));
        u = units_of<NMAX>(a, g);
    }
    // Steps of the 32 groups loaded.  Every CTA gets the same value from the same operations.
    __device__ float sum_steps() const {
        float s = static_cast<float>(u.n) * static_cast<float>(u.steps);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(~0u, s, o);
        return s;
    }
    // Parts of at most `longest` steps, none shorter than kLeastSteps.
    __device__ int parts_of(float longest) const {
        return u.n ? max(1, min(static_cast<int>(ceilf(static_cast<float>(u.steps) / longest)), u.steps / kLeastSteps)) : 0;
    }
    // Sets the length of the parts: where all units have a CTA of their own, the shortest (by whole steps, long
    // ones by sixteenths of the mean share) with no more parts than CTAs; else a quarter of the share.
    __device__ void plan(const AttnArgs& a, int ctas) {
        const float share = steps / static_cast<float>(ctas);
        longest = fmaxf(1.f, 0.25f * share);
        if (a.ngroups > 32 || __reduce_add_sync(~0u, u.n) > ctas) return;
        const float finer = fmaxf(1.f, floorf(share * 0.0625f));
        for (float x = fmaxf(1.f, ceilf(share)); x < 4.f * share + 1.f; x += finer) {
            longest = x;
            if (__reduce_add_sync(~0u, u.n * parts_of(x)) <= ctas) return;
        }
    }
    __device__ void cut() {
        u.parts = parts_of(longest);
        upto = u.n * u.parts;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(~0u, upto, o);
            if (static_cast<int>(threadIdx.x & 31) >= o) upto += x;
        }
        chunk = __shfl_sync(~0u, upto, 31);
    }
    // The unit of part `at`, its steps and parts, and which of them it is.
    __device__ void to(const AttnArgs& a, int at, PrefixPiece& w, int& steps_of, int& parts, int& in) {
        while (at >= base + chunk && b0 + 32 < a.ngroups) {
            base += chunk;
            load(a, b0 + 32);
            cut();
        }
        const int which = min(31, __popc(__ballot_sync(~0u, upto <= at - base)));
        w.row0 = __shfl_sync(~0u, g.row0, which);
        w.nrows = __shfl_sync(~0u, g.n, which) * a.group;
        w.tokens = __shfl_sync(~0u, g.tokens, which);
        w.table_row = __shfl_sync(~0u, g.table_row, which);
        w.extra = b0 + which << 16;
        const int per = __shfl_sync(~0u, u.per, which), blocks = __shfl_sync(~0u, u.blocks, which);
        steps_of = __shfl_sync(~0u, u.steps, which), parts = __shfl_sync(~0u, u.parts, which);
        const int below = __shfl_sync(~0u, upto, which ? which - 1 : 0);
        in = at - base - (which ? below : 0);
        const int unit = in / parts;
        in -= unit * parts;
        w.h = unit / blocks;
        w.row_first = (unit - w.h * blocks) * per;
        w.nc = min(per, (w.nrows - w.row_first + 15) / 16 * 16);
    }
};

__device__ __forceinline__ void sync_warps(int id, int threads) {
    asm volatile("barrier.cta.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// Whether any of the barrier's threads says so.
__device__ __forceinline__ bool any_of(int id, int threads, bool mine) {
    uint32_t r;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\tsetp.ne.u32 q, %1, 0;\n\t"
        "barrier.cta.red.or.pred p, %2, %3, q;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(r) : "r"(static_cast<uint32_t>(mine)), "r"(id), "r"(threads) : "memory");
    return r != 0;
}

// One lane of a converged warp.
__device__ __forceinline__ bool elect_one() {
    uint32_t r;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(r));
    return r != 0;
}

__device__ __forceinline__ uint32_t hmax2_of(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Sum of each of 16 columns over the 32 lanes: lanes i and i + 16 get that of column i.
__device__ __forceinline__ float add_columns(float (&v)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = 8; w > 0; w >>= 1)
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float give = lane & w ? v[i] : v[i + w], keep = lane & w ? v[i + w] : v[i];
            v[i] = keep + __shfl_xor_sync(~0u, give, w);
        }
    return v[0] + __shfl_xor_sync(~0u, v[0], 16);
}

// Largest of each of 16 columns over the 32 lanes: lanes i and i + 16 get that of column i.
__device__ __forceinline__ float max_columns(float (&v)[16]) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int w = 8; w > 0; w >>= 1)
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float give = lane & w ? v[i] : v[i + w], keep = lane & w ? v[i + w] : v[i];
            v[i] = fmaxf(keep, __shfl_xor_sync(~0u, give, w));
        }
    return fmaxf(v[0], __shfl_xor_sync(~0u, v[0], 16));
}

// The order k of z: at most kMostE, as the sums of e = p 2^k have to stay in fp32's range.
__device__ __forceinline__ int order_z(int d) { return min(kBase - d, kMostE); }

// What belongs to the columns (query rows) of a unit, in shared memory.
template <int NMAX>
struct Columns {
    float fac[NMAX];               // factor of the scores
    float nm[NMAX];                // k less the reference
    float one[NMAX], k[NMAX];      // the same of scores that were settled (huge ones)
    float mul[NMAX];               // a factor
    float ref[NMAX];
    int refd[NMAX];
    float tops[4][NMAX];           // by warp of a set: largest scores, later sums
    float tops_v[4][NMAX];         // with the orders of vs
    int64_t orow[NMAX];            // output rows, -1 past the last
};

// The first references of 4 of the 16 columns from cb on, by each warp of a set from its own 32
// keys: a lower bound of the largest, which 2^9 above the first z leaves room for.
template <int NMAX>
__device__ __noinline__ bool first_references(Columns<NMAX>& cols, int* huge_at, uint32_t scores, int cb, bool there, float ks,
                                                 int evs, int barrier) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3;
    uint32_t s[4];
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x4.b32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(s[0]), "=r"(s[1]), "=r"(s[2]), "=r"(s[3]) : "r"(scores + cb + quarter * 4));
    tmem_loaded();
    float top[4], high[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float score = __fmul_rn(__uint_as_float(s[i]), cols.fac[cb + quarter * 4 + i] * ks);
        top[i] = there && score == score ? ceilf(score) : -INFINITY;
        high[i] = top[i] + static_cast<float>(evs);
    }
    // lane l gets column l & 3
#pragma unroll
    for (int w = 2; w > 0; w >>= 1)
#pragma unroll
        for (int i = 0; i < w; ++i) {
            const float gt = lane & w ? top[i] : top[i + w], gh = lane & w ? high[i] : high[i + w];
            top[i] = fmaxf(lane & w ? top[i + w] : top[i], __shfl_xor_sync(~0u, gt, w));
            high[i] = fmaxf(lane & w ? high[i + w] : high[i], __shfl_xor_sync(~0u, gh, w));
        }
#pragma unroll
    for (int o = 4; o < 32; o <<= 1) {
        top[0] = fmaxf(top[0], __shfl_xor_sync(~0u, top[0], o));
        high[0] = fmaxf(high[0], __shfl_xor_sync(~0u, high[0], o));
    }
    if (lane < 4) {
        const int col = cb + quarter * 4 + lane;
        const float mn = fmaxf(kNoRef, top[0]);
        const int dn = max(kNoOrder, order_of(high[0] - mn));
        cols.ref[col] = mn, cols.refd[col] = dn;
        cols.nm[col] = static_cast<float>(order_z(dn)) - mn;
        if (mn > kNoRef && fabsf(mn) >= kHugeScore) *reinterpret_cast<volatile int*>(huge_at) = 1;
    }
    sync_warps(barrier, 128);
    return *reinterpret_cast<volatile int*>(huge_at) != 0;  // the same in all four
}

// New references of the 16 columns from cb on, by the four warps of a set; mul is what the sums of e
// and z are to be multiplied by, and those of z are (n accumulators of 64 columns at `sums`).  evs: the order of the key's
// vs.  Huge scores are settled: rounded, and less their references in tensor memory.  Returns whether they are.
template <int NMAX>
__device__ __noinline__ bool new_references(Columns<NMAX>& cols, int* huge_at, uint32_t scores, int cb, bool there, float ks,
                                            int evs, int barrier, uint32_t sums, int n) {
    const int lane = threadIdx.x & 31, quarter = (threadIdx.x >> 5) & 3, key = threadIdx.x & 127;
    // Largest scores, rounded up to whole orders, and with the orders of vs; `based`: the references are taken
    // off first (huge scores, whose sums with an order do not hold it).
    auto maxima = [&](bool based) {
        uint32_t s[16];
        float t[16];
        tmem_load16(scores + cb, s);
        tmem_loaded();
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const float score = __fmul_rn(__uint_as_float(s[i]), cols.fac[cb + i] * ks);
            t[i] = there && score == score ? ceilf(score) : -INFINITY;
        }
        if (!based) {
            float u[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) u[i] = t[i];
            const float top = max_columns(u);
            if (lane < 16) cols.tops[quarter][cb + lane] = top;
        }
#pragma unroll
        for (int i = 0; i < 16; ++i)
            t[i] = fmaxf(based ? t[i] - cols.ref[cb + i] : t[i], -INFINITY) + static_cast<float>(evs);
        const float top = max_columns(t);
        if (lane < 16) cols.tops_v[quarter][cb + lane] = top;
    };
    auto largest = [](const float (&of)[4][NMAX], int col) {
        return fmaxf(fmaxf(of[0][col], of[1][col]), fmaxf(of[2][col], of[3][col]));
    };
    maxima(false);
    sync_warps(barrier, 128);
    const int col = cb + key;
    int down = 0;
    if (key < 16) {
        const float m = cols.ref[col], mn = fmaxf(m, largest(cols.tops, col));
        down = order_of(m - mn);
        cols.ref[col] = mn;
        if (mn > kNoRef && fabsf(mn) >= kHugeScore) *huge_at = 1;
    }
    sync_warps(barrier, 128);
    const bool huge = *reinterpret_cast<volatile int*>(huge_at) != 0;
    if (huge) {
        maxima(true);
        sync_warps(barrier, 128);
    }
    if (key < 16) {
        const int d = cols.refd[col];
        const float high = largest(cols.tops_v, col);
        const int dn = max(max(d + down, kNoOrder), order_of(huge ? high : high - cols.ref[col]));
        cols.mul[col] = pow2i(order_z(dn) - order_z(d) + down);
        cols.refd[col] = dn;
        cols.k[col] = static_cast<float>(order_z(dn)), cols.nm[col] = cols.k[col] - cols.ref[col];
    }
    sync_warps(barrier, 128);
    uint32_t s[16];
    for (int x = 0; x < n; ++x) {
        tmem_load16(sums + x * 64 + cb, s);
        tmem_loaded();
#pragma unroll
        for (int i = 0; i < 16; ++i) s[i] = __float_as_uint(__uint_as_float(s[i]) * cols.mul[cb + i]);
        tmem_store16(sums + x * 64 + cb, s);
    }
    if (huge) {
        tmem_load16(scores + cb, s);
        tmem_loaded();
#pragma unroll
        for (int i = 0; i < 16; ++i)
            s[i] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(s[i]), cols.fac[cb + i] * ks), cols.ref[cb + i]));
        tmem_store16(scores + cb, s);
    }
    tmem_stored();
    return huge;
}

// The rest of a wait whose phase had not ended at first: out of line, as most code that a step does not
// run, for the warps' different roles leave the instruction caches little room.
__device__ __noinline__ bool wait_on(uint64_t* bar, uint32_t parity, unsigned* status) {
    return __any_sync(~0u, !mbar_wait_bounded(bar, parity, status));
}

template <int DP, int QP, int PP, bool INT8>
__global__ void __launch_bounds__(kPrefixThreads, 1)
qg_attn_prefix_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap) {
    using F = XShape<DP, QP, PP>;
    constexpr int NMAX = F::NMAX;
    extern __shared__ __align__(1024) unsigned char smem[];
    float4* scales = reinterpret_cast<float4*>(smem + F::off_scale);  // [kScaleSteps][8]: ks, vs, there
    Columns<NMAX>& cols = *reinterpret_cast<Columns<NMAX>*>(smem + F::off_cols);
    uint64_t* kraw_full = reinterpret_cast<uint64_t*>(smem + F::off_bar);
    uint64_t* kraw_empty = kraw_full + F::kRawK;
    uint64_t* vraw_full = kraw_empty + F::kRawK;
    uint64_t* vraw_empty = vraw_full + F::kRawV;
    uint64_t* k_full = vraw_empty + F::kRawV;
    uint64_t* k_empty = k_full + F::KB;
    uint64_t* v_full = k_empty + F::KB;
    uint64_t* v_empty = v_full + F::kOps;
    uint64_t* s_full = v_empty + F::kOps;   // [SB]
    uint64_t* p_full = s_full + F::SB;      // [SB]
    uint64_t* pv_done = p_full + F::SB;     // [SB]
    uint64_t* q_full = pv_done + F::SB;
    uint64_t* sc_full = q_full + 1;         // [kScaleSteps]
    uint64_t* unit_full = sc_full + kScaleSteps;
    uint64_t* unit_empty = unit_full + kUnitsAhead;
    static_assert((2 * F::kRaws + 2 * F::KB + 2 * F::kOps + 3 * F::SB + 1 + kScaleSteps + 2 * kUnitsAhead) * 8 <= 512, "barriers");
    __shared__ PrefixPiece units[kUnitsAhead];
    __shared__ uint32_t tmem_slot;
    __shared__ int huge_set[kSets];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const KVLayer& c = a.c;
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled operands need it; the same in all threads
        if (tid == 0) atomicOr(a.status, kStatusBounds);
        return;
    }
    if (tid == 0) {
        for (uint32_t i = 0; i < F::kRawK; ++i) mbar_init(kraw_full + i, 1), mbar_init(kraw_empty + i, 4);
        for (uint32_t i = 0; i < F::kRawV; ++i) mbar_init(vraw_full + i, 1), mbar_init(vraw_empty + i, 4);
        for (uint32_t i = 0; i < F::KB; ++i) mbar_init(k_full + i, 4), mbar_init(k_empty + i, 1);
        for (uint32_t i = 0; i < F::kOps; ++i) mbar_init(v_full + i, 4), mbar_init(v_empty + i, 1);
        for (uint32_t i = 0; i < F::SB; ++i) mbar_init(s_full + i, 1), mbar_init(p_full + i, kSoftmaxWarps), mbar_init(pv_done + i, 1);
        mbar_init(q_full, kSoftmaxWarps);
        for (uint32_t i = 0; i < kScaleSteps; ++i) mbar_init(sc_full + i, 1);
        for (uint32_t i = 0; i < kUnitsAhead; ++i)
            mbar_init(unit_full + i, 1), mbar_init(unit_empty + i, kSoftmaxWarps + 8 + 1);
        fence_mbar_init();
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&tmem_slot)), "r"(512) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    // the copying warp measures the line meanwhile
    PartWalk<NMAX> walk;
    int total = 0;
    if (warp == kCopyWarp) {
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
        walk.load(a, 0);
        walk.steps = walk.sum_steps();
        for (int b = 32; b < a.ngroups; b += 32) {
            PartWalk<NMAX> next;
            next.load(a, b);
            walk.steps += next.sum_steps();
        }
        walk.plan(a, gridDim.x);
        walk.cut();
        total = walk.chunk;
        for (int b = 32; b < a.ngroups; b += 32) {
            PartWalk<NMAX> next;
            next.load(a, b);
            next.longest = walk.longest;
            next.cut();
            total += next.chunk;
        }
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;
    const uint32_t o_at = tmem + F::o_at;
    // A wait that gave up ends all further waits, copies and MMAs of its warp:
    // the kernel then runs to its end within a few wait limits.
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {  // by whole warps
        if (!dead && !__all_sync(~0u, mbar_try_wait(bar, parity & 1u))) dead = wait_on(bar, parity & 1u, a.status);
    };
    // The next piece, as the copying warp hands it to the others; false after the last.
    uint32_t turn = 0;
    PrefixPiece w;
    auto next_unit = [&]() {
        const uint32_t slot = turn % kUnitsAhead;
        wait(unit_full + slot, turn / kUnitsAhead);
        w = units[slot];
        __syncwarp();
        if (lane == 0) arrive_on(unit_empty + slot);
        ++turn;
        return !dead && w.tokens >= 0;
    };

    if (warp == kCopyWarp) {
        // ---------------------------------------------------------- copies
        const Line line(total, gridDim.x);
        int at = 0, end = 0;
        if (static_cast<int>(blockIdx.x) < line.ctas)
            at = static_cast<int>(line.first(blockIdx.x)), end = static_cast<int>(line.first(blockIdx.x + 1));
        uint32_t o = 0, g = 0;  // raw tiles of K, and of V, and steps over the life of the kernel
        uint32_t sent_k = 0, sent_v = 0;  // raw tiles whose copies were issued
        const int box = min(kKeys, 1 << c.log2p);  // tokens of a copy: a page's, as far as they are one step's
        auto copy = [&](bool v, int tile, int tok, int id, unsigned valid, uint32_t n) {
            const uint32_t slots = v ? F::kRawV : F::kRawK, slot = n % slots;
            uint64_t* full = (v ? vraw_full : kraw_full) + slot;
            if (n >= slots) wait((v ? vraw_empty : kraw_empty) + slot, n / slots - 1);
            if (dead) return;  // no arrival at a barrier whose bytes may be outstanding
            if (lane == 0) mbar_arrive_expect_tx(full, valid * 16 * F::RW);
            __syncwarp();
            if (id >= 0 && (lane & 7) * 16 % box == 0)
                tma_load_4d(smem + F::off_raw + (slot + (v ? F::kRawK : 0)) * F::kRaw + (lane & 7) * 16 * F::RW, v ? &vmap : &kmap,
                            tile * F::RW, tok, w.h, id, full);
            (v ? sent_v : sent_k) = n + 1;
        };
        for (;; ++turn) {
            const uint32_t slot = turn % kUnitsAhead;
            if (turn >= kUnitsAhead) wait(unit_empty + slot, turn / kUnitsAhead - 1);
            const bool there = !dead && at < end;
            if (there) {
                int steps, parts, in;
                walk.to(a, at, w, steps, parts, in);
                const int last = min(end - at, parts - in) + in;  // parts of one unit are one piece
                w.j0 = static_cast<int>(div64(static_cast<int64_t>(steps) * in, parts));
                w.j1 = static_cast<int>(div64(static_cast<int64_t>(steps) * last, parts));
                w.slot = in == 0 ? -1 : static_cast<int>(blockIdx.x);
                if (in == 0) w.extra |= line.of(at + parts - 1) - static_cast<int>(blockIdx.x);
                at += last - in;
            } else {
                w.tokens = -1;
            }
            if (lane == 0) {
                units[slot] = w;
                arrive_on(unit_full + slot);
            }
            __syncwarp();
            if (!there) break;
            const int32_t* table = a.table + static_cast<int64_t>(w.table_row) * a.width;
            // Lane i has the page and scales of the i-th 16 tokens of four steps; those of the next four are on
            // their way meanwhile.
            const int64_t last_tok = min(static_cast<int64_t>(w.tokens), static_cast<int64_t>(w.j1) * kKeys);
            auto pages = [&](int j) {
                const int64_t tok = static_cast<int64_t>(j) * kKeys + lane * 16;
                int id = -1;
                if (tok < last_tok) {
                    id = __ldg(table + (tok >> c.log2p));
                    if (id < 0 || id >= c.pages) {
                        id = -1;
                        atomicOr(a.status, kStatusBounds);
                    }
                }
                return id;
            };
            auto page_scales = [&](int id) {
                float2 f = make_float2(0.f, 0.f);
                if (id >= 0) {
                    const int64_t s = static_cast<int64_t>(id) * c.heads + w.h;
                    f = make_float2(__ldg(c.ks + s), __ldg(c.vs + s));
                }
                return f;
            };
            int id = pages(w.j0), id_next = -1;
            float2 f = page_scales(id), f_next = f;
            for (int j = w.j0; j < w.j1; ++j, ++g) {
                const int r = (j - w.j0) & 3;
                if (r == 0) {
                    if (j > w.j0) id = id_next, f = f_next;
                    id_next = pages(j + 4);
                }
                if (r == 2) f_next = page_scales(id_next);
                const bool mine = (lane >> 3) == r;
                const int tok = static_cast<int>((static_cast<int64_t>(j) * kKeys + (lane & 7) * 16) & ((1 << c.log2p) - 1));
                const unsigned valid = __popc(__ballot_sync(~0u, mine && id >= 0));
                for (int t = 0; t < F::RT; ++t) copy(false, t, tok, mine ? id : -1, valid, o + t);
                if (mine) scales[(g % kScaleSteps) * 8 + (lane & 7)] = make_float4(f.x, f.y, id >= 0 ? 1.f : 0.f, 0.f);
                __syncwarp();
                if (lane == 0) arrive_on(sc_full + g % kScaleSteps);
                for (int t = 0; t < F::RT; ++t) copy(true, t, tok, mine ? id : -1, valid, o + t);
                o += F::RT;
            }
        }
        if (dead) {  // the copies in flight: shared memory is theirs until they land
            for (uint32_t x = sent_k > F::kRawK ? sent_k - F::kRawK : 0; x < sent_k; ++x)
                (void)mbar_wait_bounded(kraw_full + x % F::kRawK, (x / F::kRawK) & 1u, a.status);
            for (uint32_t x = sent_v > F::kRawV ? sent_v - F::kRawV : 0; x < sent_v; ++x)
                (void)mbar_wait_bounded(vraw_full + x % F::kRawV, (x / F::kRawV) & 1u, a.status);
        }
    } else if (warp == kMmaWarp) {
        // ---------------------------------------------------------- MMAs
        // What the sequences hold behind the prefix comes to L2 meanwhile, for the launch behind this one, as far
        // as L2 keeps it: a lane a page.
        const uint32_t page_bytes = static_cast<uint32_t>(c.heads * c.dim) << c.log2p;
        int64_t room = kPrefetchBytes / (2 * static_cast<int64_t>(page_bytes) * gridDim.x);
        for (int b = blockIdx.x; b < a.batch && room > 0; b += gridDim.x) {
            const int64_t len = min(static_cast<int64_t>(max(a.lens[b], 0)), a.width << c.log2p);
            const int64_t from = max(a.skip[b], 0) >> c.log2p;
            const int64_t pages = min((len + (1 << c.log2p) - 1) >> c.log2p, from + room);
            for (int64_t x = from + lane; x < pages; x += 32) {
                const int id = a.table[b * a.width + x];
                if (id < 0 || id >= c.pages) continue;
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(c.k + id * c.page_stride), "r"(page_bytes) : "memory");
                asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(c.v + id * c.page_stride), "r"(page_bytes) : "memory");
            }
            room -= max(int64_t(0), pages - from);
        }
        __syncwarp();
        // All that the MMAs take is uniform, and so known to be, and one lane is elected: then their operands need no
        // moves between register files, which made an MMA's issue 120 clocks (16 a step: 3000 clocks a step, all of it).
        uint32_t g = 0, qs = 0;  // steps and queries taken
        const uint32_t tm = __shfl_sync(~0u, tmem, 0), sm = __shfl_sync(~0u, smem_u32(smem), 0);
        while (next_unit()) {
            const int steps = __shfl_sync(~0u, w.j1 - w.j0, 0);
            const uint32_t sdesc = f16_desc(__shfl_sync(~0u, w.nc, 0)), pdesc = f16_desc_mn(F::NP);
            constexpr int kLag = F::SB - 1;  // steps that the second products are behind the first
            wait(q_full, qs);
            for (int j = 0; j < steps + kLag; ++j) {
                if (j < steps) {
                    const uint32_t n = g + j, kb = n % F::KB, st = tm + n % F::SB * NMAX;
                    wait(k_full + kb, n / F::KB);
                    fence_after();
                    if (!dead && elect_one()) {
                        const uint32_t ka = tm + F::k_at + kb * (DP / 2);
#pragma unroll
                        for (int p = QP - 1; p >= 0; --p) {  // the small parts first: half the roundings at full size
                            const uint64_t qb = operand_desc(sm + p * F::kQPart);
#pragma unroll
                            for (int ks = 0; ks < DP / 16; ++ks)
                                mma_ts(st, ka + ks * 8, qb + (((ks >> 2) * (NMAX * 128) + (ks & 3) * 32) >> 4), sdesc,
                                       p < QP - 1 || ks > 0 ? 1u : 0u);
                        }
                        commit_to(s_full + n % F::SB);
                        commit_to(k_empty + kb);
                    }
                    __syncwarp();
                }
                if (j >= kLag) {
                    const uint32_t n = g + j - kLag, os = n % F::kOps;
                    wait(v_full + os, n / F::kOps);
                    wait(p_full + n % F::SB, n / F::SB);
                    fence_after();
                    if (!dead && elect_one()) {
#pragma unroll
                        for (int acc = 0; acc < F::DA; ++acc) {
                            const uint64_t vb = operand_desc_mn(sm + F::off_op + os * F::kOp + acc * 32768, 16384);
#pragma unroll
                            for (int p = PP - 1; p >= 0; --p) {
                                const uint64_t pb = operand_desc_mn(sm + F::off_p + ((n % F::PB) * PP + p) * F::kPPart, 16384);
#pragma unroll
                                for (int ks = 0; ks < kKeys / 16; ++ks)
                                    mma_ss(tm + F::o_at + (p * F::DA + acc) * F::NP, vb + ((ks * 2048) >> 4), pb + ((ks * 2048) >> 4),
                                           pdesc, j > kLag || ks > 0 ? 1u : 0u);
                            }
                        }
                        commit_to(pv_done + n % F::SB);
                        commit_to(v_empty + os);
                    }
                    __syncwarp();
                }
            }
            g += steps;
            ++qs;
        }
    } else if (warp >= kValueWarp) {
        // ---------------------------------------------------------- V: 8 bits -> f16 in shared memory, as it lies
        // A warp has 64 of the dims and a part of the tokens, a lane 16 dims of every eighth token: its places in the
        // swizzled rows are then the same for all of them, and the 32 lanes meet every bank equally often.
        constexpr int DB = F::RW / 64, WT = kKeys * DB / 4;  // blocks of 64 dims of a raw tile, tokens of a warp
        const int vw = warp - kValueWarp, block = vw % DB, c16 = block * 4 + (lane & 3), t7 = lane >> 2;
        const int token0 = vw / DB * WT + t7;
        const int from = token0 * F::RW + ((F::RW == 64 ? c16 ^ (t7 >> 1) : c16 ^ t7) << 4);
        const int to0 = block * 16384 + token0 * 128 + (((2 * (lane & 3)) ^ t7) << 4);
        const int to1 = block * 16384 + token0 * 128 + (((2 * (lane & 3) + 1) ^ t7) << 4);
        uint32_t r = 0, g = 0;  // raw tiles and steps
        while (next_unit()) {
            for (int j = w.j0; j < w.j1; ++j, ++g) {
                const float4* sc = scales + (g % kScaleSteps) * 8;
                wait(sc_full + g % kScaleSteps, g / kScaleSteps);
                const bool whole = __all_sync(~0u, sc[lane & 7].z != 0.f);  // no page is missing
                const uint32_t os = g % F::kOps;
#pragma unroll 1
                for (int t = 0; t < F::RT; ++t, ++r) {
                    const uint32_t rs = r % F::kRawV;
                    wait(vraw_full + rs, r / F::kRawV);
                    if (t == 0 && g >= F::kOps) wait(v_empty + os, g / F::kOps - 1);
                    const unsigned char* raw = smem + F::off_raw + (F::kRawK + rs) * F::kRaw + from;
                    unsigned char* op = smem + F::off_op + os * F::kOp + t * 32768;
#pragma unroll
                    for (int i0 = 0; i0 < WT / 8; i0 += 4) {
                        uint4 x[4];
#pragma unroll
                        for (int i = 0; i < 4; ++i) x[i] = *reinterpret_cast<const uint4*>(raw + (i0 + i) * 8 * F::RW);
                        if (!whole) {
#pragma unroll
                            for (int i = 0; i < 4; ++i)
                                if (sc[(token0 + (i0 + i) * 8) >> 4].z == 0.f) x[i] = make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            uint32_t h[8];
                            k_codes<INT8>(x[i].x, h[0], h[1]);
                            k_codes<INT8>(x[i].y, h[2], h[3]);
                            k_codes<INT8>(x[i].z, h[4], h[5]);
                            k_codes<INT8>(x[i].w, h[6], h[7]);
                            *reinterpret_cast<uint4*>(op + to0 + (i0 + i) * 1024) = make_uint4(h[0], h[1], h[2], h[3]);
                            *reinterpret_cast<uint4*>(op + to1 + (i0 + i) * 1024) = make_uint4(h[4], h[5], h[6], h[7]);
                        }
                    }
                    __syncwarp();
                    if (lane == 0 && !dead) arrive_on(vraw_empty + rs);  // a slot goes back only when its copy has landed
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) arrive_on(v_full + os);
            }
        }
    } else if (warp >= kKeyWarp) {
        // ---------------------------------------------------------- K: 8 bits -> f16 in tensor memory, a thread a key
        const int key = tid - kKeyWarp * 32;
        const int turn16 = F::RW == 64 ? (key >> 1) & 3 : key & 7;  // the copy's swizzle: no two of eight rows in a bank
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        uint32_t r = 0, g = 0;  // raw tiles and steps
        while (next_unit()) {
            for (int j = w.j0; j < w.j1; ++j, ++g) {
                wait(sc_full + g % kScaleSteps, g / kScaleSteps);
                const bool there = scales[(g % kScaleSteps) * 8 + (key >> 4)].z != 0.f, whole = __all_sync(~0u, there);
                const uint32_t kb = g % F::KB;
#pragma unroll 1
                for (int t = 0; t < F::RT; ++t, ++r) {
                    const uint32_t rs = r % F::kRawK;
                    wait(kraw_full + rs, r / F::kRawK);
                    if (t == 0 && g >= F::KB) {
                        wait(k_empty + kb, g / F::KB - 1);
                        fence_after();
                    }
                    const unsigned char* raw = smem + F::off_raw + rs * F::kRaw + key * F::RW;
#pragma unroll
                    for (int c = 0; c < F::RW / 32; ++c) {
                        uint4 x[2];
                        uint32_t h[16];
#pragma unroll
                        for (int i = 0; i < 2; ++i) x[i] = *reinterpret_cast<const uint4*>(raw + ((c * 2 + i) * 16 ^ turn16 * 16));
                        if (!whole) {
#pragma unroll
                            for (int i = 0; i < 2; ++i)
                                if (!there) x[i] = make_uint4(0, 0, 0, 0);
                        }
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            k_codes<INT8>(x[i].x, h[8 * i], h[8 * i + 1]);
                            k_codes<INT8>(x[i].y, h[8 * i + 2], h[8 * i + 3]);
                            k_codes<INT8>(x[i].z, h[8 * i + 4], h[8 * i + 5]);
                            k_codes<INT8>(x[i].w, h[8 * i + 6], h[8 * i + 7]);
                        }
                        tmem_store16(tmem + F::k_at + kb * (DP / 2) + lanes + t * (F::RW / 2) + c * 16, h);
                    }
                    __syncwarp();
                    if (lane == 0 && !dead) arrive_on(kraw_empty + rs);
                }
                tmem_stored();
                fence_before();
                __syncwarp();
                if (lane == 0) arrive_on(k_full + kb);
            }
        }
    } else {
        // ---------------------------------------------------------- softmax, a thread a key and a set's columns
        const int set = warp >> 2, quarter = warp & 3, key = quarter * 32 + lane, wid = 2 + set;
        const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16;
        uint32_t g = 0;
        for (;; ++turn) {
            const uint32_t slot = turn % kUnitsAhead;
            wait(unit_full + slot, turn / kUnitsAhead);
            // All warps go on or none: they meet at barriers below, whether their waits gave up or not.
            if (any_of(1, kSoftmaxWarps * 32, dead || units[slot].tokens < 0)) break;
            const volatile PrefixPiece& w = units[slot];
            const int nc = w.nc, j0 = w.j0, j1 = w.j1;
            {
                // ---- queries: f16 parts of q * 2^e for the rows of this warp, and what belongs to each row
                constexpr int QL = DP / 4 < 32 ? DP / 4 : 32, VL = DP / 4 / QL, QR = 32 / QL;  // lanes a row, vectors a lane
                constexpr int NB = NMAX / kSoftmaxWarps / QR;  // all reads on their way at once
                const int each = nc / kSoftmaxWarps, h = w.h, nrows = w.nrows, row_first = w.row_first;
                const int64_t row0 = w.row0;
                uint4 raw[NB][VL];
                int64_t mine = -1, my_to = -1;  // lane i: of row i
                {
                    const int r = row_first + warp * each + lane;
                    if (lane < each && r < nrows) {
                        const int i_row = static_cast<unsigned>(r) / static_cast<unsigned>(a.group), hq = h * a.group + r - i_row * a.group;
                        my_to = (row0 + i_row) * a.q_heads + hq;
                        mine = (row0 + i_row) * a.q_row + hq * a.q_head;
                    }
                    if (lane < each) cols.orow[warp * each + lane] = my_to;
                }
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    const int64_t qat = __shfl_sync(~0u, mine, i * QR + lane / QL);
#pragma unroll
                    for (int v = 0; v < VL; ++v) {
                        const int d = (v * QL + lane % QL) * 4;
                        raw[i][v] = load_q4(a.q, a.type, qat + d, qat >= 0 && d < c.dim);
                    }
                }
#pragma unroll
                for (int i = 0; i < NB; ++i) {
                    if (i * QR >= each) break;
                    const int in = i * QR + lane / QL, col = warp * each + in;
                    float amax = 0.f;
                    float4 x[VL];
#pragma unroll
                    for (int v = 0; v < VL; ++v) {
                        x[v] = q4_values(raw[i][v], a.type);
                        amax = fmaxf(fmaxf(fmaxf(amax, fabsf(x[v].x)), fmaxf(fabsf(x[v].y), fabsf(x[v].z))), fabsf(x[v].w));
                    }
#pragma unroll
                    for (int k = QL / 2; k > 0; k >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, k));
                    // 2^e with amax * 2^e in [2^14, 2^15); 1 for zero or non-finite rows
                    int e = 141 - static_cast<int>((__float_as_uint(amax) >> 23) & 255u);
                    e = amax > 0.f && amax <= 3.4028235e38f ? min(e, 120) : 0;
                    const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
                    if (in < each) {
                        if (lane % QL == 0) {
                            cols.fac[col] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
                            cols.one[col] = 1.f;
                        }
#pragma unroll
                        for (int v = 0; v < VL; ++v) {
                            const int d = (v * QL + lane % QL) * 4, ch = d >> 3;
                            // the dims in the order that k_codes gives a word's bytes
                            const float y0 = x[v].x * up, y1 = (INT8 ? x[v].z : x[v].y) * up;
                            const float y2 = (INT8 ? x[v].y : x[v].z) * up, y3 = x[v].w * up;
                            const uint2 hi = make_uint2(pack_f16x2(y0, y1), pack_f16x2(y2, y3));
                            unsigned char* dst = smem + (ch >> 3) * (NMAX * 128) + col * 128 + (((ch & 7) ^ (col & 7)) << 4) + (d & 4) * 2;
                            *reinterpret_cast<uint2*>(dst) = hi;
                            if (QP == 2)
                                *reinterpret_cast<uint2*>(dst + F::kQPart) = make_uint2(rest_f16x2(y0, y1, hi.x), rest_f16x2(y2, y3, hi.y));
                        }
                    }
                }
                if (lane == 0 && quarter == 0) huge_set[set] = 0;
                fence_proxy_async_smem();
                sync_warps(1, kSoftmaxWarps * 32);
                if (lane == 0) arrive_on(q_full);
            }
            f2 l[8];  // sums of e by column pairs
#pragma unroll
            for (int i = 0; i < 8; ++i) l[i] = {0.f, 0.f};
            const int cb = set * 16;
            const bool busy = cb < nc;  // this set has columns

            bool huge = false, next_ready = false;  // the set's scores are; the next step's scales are there
            float4 page = make_float4(0.f, 0.f, 0.f, 0.f);  // of this step, read a step ahead
            auto next_page = [&](uint32_t n, bool ready) {
                if (!ready) wait(sc_full + n % kScaleSteps, n / kScaleSteps);
                return scales[(n % kScaleSteps) * 8 + (key >> 4)];
            };
            if (busy) page = next_page(g, false);

            for (int j = j0; j < j1; ++j, ++g) {
                // Its MMAs are behind the second products of step g - 3, whose z's buffer is free then where there are three.
                wait(s_full + g % F::SB, g / F::SB);
                fence_after();
                if (busy) {
                    next_ready = j + 1 < j1 && __all_sync(~0u, mbar_try_wait(sc_full + (g + 1) % kScaleSteps, ((g + 1) / kScaleSteps) & 1u));
                    const float ks = page.x, vs = page.y;
                    const bool there = page.z != 0.f;
                    // vs < 2^evs
                    const int evs = vs > 0.f ? static_cast<int>((__float_as_uint(vs) >> 23) & 255u) - 126 : kNoOrder;
                    // pages there whose vs shows in z when e would leave its range
                    const bool plain = __all_sync(~0u, there && evs > -90);
                    const uint32_t st = tmem + g % F::SB * NMAX + lanes;
                    f2 e[8];
                    uint32_t z[8], zl[PP == 2 ? 8 : 1];
                    uint32_t s[16];
                    // e = p 2^k and z = e vs of the 16 columns under the references as they are; whether one passes them.
                    bool settled = false;
                    auto attempt = [&]() {
                        tmem_load16(st + cb, s);
                        tmem_loaded();
                        float high = -INFINITY;
                        uint32_t most = 0u;
                        const float* fac = (settled ? cols.one : cols.fac) + cb;
                        const float* nm = (settled ? cols.k : cols.nm) + cb;
                        const float by = settled ? 1.f : ks;
#pragma unroll
                        for (int q = 0; q < 4; ++q) {
                            const float4 fa = *reinterpret_cast<const float4*>(fac + 4 * q);
                            const float4 na = *reinterpret_cast<const float4*>(nm + 4 * q);
#pragma unroll
                            for (int u = 0; u < 2; ++u) {
                                const int i = 2 * q + u;
                                const f2 fq = fmul2(u ? f2{fa.z, fa.w} : f2{fa.x, fa.y}, f2{by, by});
                                e[i] = u ? f2{na.z, na.w} : f2{na.x, na.y};
                                ffma2(e[i], {__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])}, fq);
                            }
                        }
                        if (!plain) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                if (!there) e[i].x = e[i].y = -INFINITY;
                                high = fmaxf(high, fmaxf(e[i].x, e[i].y));
                            }
                        }
#pragma unroll
                        for (int i = 0; i < 8; ++i) {
                            e[i] = {exp2_fast(e[i].x), exp2_fast(e[i].y)};
                            const f2 zz = fmul2(e[i], f2{vs, vs});
                            z[i] = pack_f16x2(zz.x, zz.y);
                            if (PP == 2) {  // 2^11 times what the first part leaves
                                const f2 hi = h2_to_f2(z[i]);
                                zl[i % (PP == 2 ? 8 : 1)] = pack_f16x2((zz.x - hi.x) * 2048.f, (zz.y - hi.y) * 2048.f);
                            }
                            most = hmax2_of(most, z[i]);
                        }
                        return high > 105.f || (most & 0xFFFFu) > 0x7800u || (most >> 16) > 0x7800u;  // f16's 2^15
                    };
                    if (j == j0) huge = first_references<NMAX>(cols, huge_set + set, st, cb, there, ks, evs, wid);
#pragma unroll 1
                    for (int round = 0;; round = 1) {
                        const bool passed = attempt();
                        if (round == 1 || !any_of(wid, 128, passed || huge)) break;
                        if (j > j0) wait(pv_done + (g - 1) % F::SB, (g - 1) / F::SB);  // O stands still
                        fence_after();
                        settled = huge = new_references<NMAX>(cols, huge_set + set, st, cb, there, ks, evs, wid, o_at + lanes,
                                                       j > j0 ? PP * F::DA : 0);
                        if (j > j0) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) l[i] = fmul2(l[i], *reinterpret_cast<const f2*>(cols.mul + cb + 2 * i));
                        }
                    }
                    if (F::PB == 1 && g > 0) wait(pv_done + (g - 1) % F::SB, (g - 1) / F::SB);  // z's buffer is free
#pragma unroll
                    for (int i = 0; i < 8; ++i) fadd2(l[i], e[i]);
                    unsigned char* dst = smem + F::off_p + (g % F::PB) * PP * F::kPPart + key * 128;
                    const int ch = cb >> 3;
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        unsigned char* at = dst + (((ch + u) ^ (key & 7)) << 4);
                        *reinterpret_cast<uint4*>(at) = make_uint4(z[4 * u], z[4 * u + 1], z[4 * u + 2], z[4 * u + 3]);
                        if (PP == 2)
                            *reinterpret_cast<uint4*>(at + F::kPPart) =
                                make_uint4(zl[(4 * u) % (PP == 2 ? 8 : 1)], zl[(4 * u + 1) % (PP == 2 ? 8 : 1)],
                                           zl[(4 * u + 2) % (PP == 2 ? 8 : 1)], zl[(4 * u + 3) % (PP == 2 ? 8 : 1)]);
                    }
                    fence_proxy_async_smem();
                    fence_before();
                }
                __syncwarp();
                if (lane == 0) arrive_on(p_full + g % F::SB);
                if (busy && j + 1 < j1) page = next_page(g + 1, next_ready);
            }

            // ---- the rows' sums, then their results
            float* part = a.slots + static_cast<int64_t>(w.slot < 0 ? 0 : w.slot) * (NMAX * (DP + 2));
            const bool begins = w.slot < 0;
            if (busy) {
                float v[16];
#pragma unroll
                for (int i = 0; i < 8; ++i) v[2 * i] = l[i].x, v[2 * i + 1] = l[i].y;
                const float sum = add_columns(v);
                if (lane < 16) cols.tops[quarter][cb + lane] = sum;
                sync_warps(wid, 128);
                if (key < 16) {
                    const int col = cb + key;
                    const float sum = (cols.tops[0][col] + cols.tops[1][col]) + (cols.tops[2][col] + cols.tops[3][col]);
                    // NaN sums stay NaN; a row that saw nothing has a sum of 0
                    const bool none = sum == 0.f && cols.ref[col] == kNoRef;
                    cols.mul[col] = none ? 0.f : 1.f / sum;
                    const float m = none ? -INFINITY : cols.ref[col];
                    const float total = none ? 0.f : sum * pow2i(-order_z(cols.refd[col]));
                    if (begins) {
                        if (cols.orow[col] >= 0)
                            a.own_ml[cols.orow[col]] = make_float4(m, total, __int_as_float((static_cast<int>(blockIdx.x) + 1) | col << 16),
                                                                   __int_as_float(w.extra));
                    } else {
                        *reinterpret_cast<float2*>(part + NMAX * DP + 2 * col) = make_float2(m, total);
                    }
                }
            }
            wait(pv_done + (g - 1) % F::SB, (g - 1) / F::SB);
            fence_after();
            sync_warps(wid, 128);
            const int place = INT8 ? (lane & ~3) | ((lane & 1) << 1 | (lane & 2) >> 1) : lane;  // dims as k_codes orders them
#pragma unroll 1
            for (int acc = 0; busy && acc < F::DA; ++acc) {
                const int d = acc * 128 + quarter * 32 + place;
                if (acc * 128 + quarter * 32 >= c.dim) break;
                uint32_t v[16], vl[16];
                tmem_load16(o_at + acc * F::NP + lanes + cb, v);
                if (PP == 2) tmem_load16(o_at + (F::DA + acc) * F::NP + lanes + cb, vl);
                tmem_loaded();
                if (d < c.dim) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        float x = __uint_as_float(v[i]);
                        if (PP == 2) x = fmaf(__uint_as_float(vl[i]), 0x1p-11f, x);
                        const float f = cols.mul[cb + i];
                        const int64_t to = cols.orow[cb + i];
                        if (to >= 0) (begins ? a.own + to * c.dim : part + (cb + i) * DP)[d] = f == 0.f ? 0.f : x * f;
                    }
                }
                __syncwarp();
            }
            fence_before();
            __syncwarp();
            if (lane == 0) arrive_on(unit_empty + slot);
            sync_warps(1, kSoftmaxWarps * 32);  // all have left the columns' data
        }
    }
    fence_before();
    __syncthreads();
    if (warp == kMmaWarp) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512) : "memory");
    }
}

template <int DP, int QP, int PP, bool INT8>
int launch_one(AttnArgs& a, cudaStream_t s) {
    using F = XShape<DP, QP, PP>;
    const int dev = current_device();
    const int sms = sm_count(dev);
    if (sms <= 0) return cuda_fail(cudaGetLastError());
    const int box = std::min(kKeys, 1 << a.c.log2p);
    CUtensorMap kmap, vmap;
    if (!encode_cache(&kmap, a.c, a.c.k, F::RW, box, true) || !encode_cache(&vmap, a.c, a.c.v, F::RW, box, true))
        return cuda_fail(cudaGetLastError());
    static std::atomic<bool> done[64];
    auto kern = qg_attn_prefix_kernel<DP, QP, PP, INT8>;
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F::smem) != cudaSuccess)
            return cuda_fail(cudaGetLastError());
        done[dev].store(true, std::memory_order_release);
    }
    a.slot_rows = F::NMAX, a.slot_dims = DP;
    kern<<<std::min(sms, kMaxPrefixCtas), kPrefixThreads, F::smem, s>>>(a, kmap, vmap);
    return launch_status();
}

template <int QP, int PP, bool INT8>
int launch_typed(AttnArgs& a, cudaStream_t s) {
    if (a.c.dim <= 64) return launch_one<64, QP, PP, INT8>(a, s);
    return a.c.dim <= 128 ? launch_one<128, QP, PP, INT8>(a, s) : launch_one<256, QP, PP, INT8>(a, s);
}

}  // namespace

template <bool INT8>
int launch_prefix(AttnArgs& a, cudaStream_t s) {
    if (a.type == QGKV_F32) return launch_typed<2, 2, INT8>(a, s);
    // f16 outputs round as finely as one f16 part of p would: two
    if (a.type == QGKV_F16) return launch_typed<1, 2, INT8>(a, s);
    return launch_typed<1, 1, INT8>(a, s);
}

}  // namespace qg
