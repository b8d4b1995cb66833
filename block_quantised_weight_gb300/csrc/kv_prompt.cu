// Attention of many query rows over the 8-bit paged cache (prompts and long
// chunks) on the tcgen05 tensor cores.
//
// Mathematics: kv_rows.cuh's.  A CTA takes ROWS = 256 query rows (tokens x
// heads of a group) of one cache head as two tiles of 128 (fp32 queries: one
// tile of 128, whose q enters as two f16 parts), and walks the keys in
// steps of 128 tokens:
//   S = q K^T     q, K as f16 operands in shared memory, S in tensor memory
//   p = 2^(S * scale * ks + log2 vs + k - m),  one thread a row, over S as f16
//   O += p V      p from tensor memory, V^T from shared memory
// with l the sum of p less its block's scale.  A row's references m and u (k =
// 6 + m - u, 12 for two parts of p) are whole numbers that move only when a score
// passes them by more than 8 (2): the thread takes its 64 scores once, as if they held, and only where
// one passes goes round again and rescales its row of O in tensor memory.
//
// Bound.  4 * dim flops a score, 1 exponential: for 128 dims the tensor pipe
// and the issue slots of the softmax are near each other.  So the roles run
// beside each other: one warp finds the work and copies (TMA), four convert the 8-bit codes into
// f16 operands (K as it lies, V transposed, so that both products take
// K-major operands), one issues the MMAs, four a tile do the softmax.  The
// MMAs of one tile run while the other's softmax does; the converted operands
// serve both tiles.  Measured: prompt chunks (4812 rows in three, the longest of
// 2048, behind up to 6000 tokens, 32 / 8 heads of 128, e4m3, bf16 q) 427-455 us,
// 675-720 TFLOP/s (int8 457); fp32 q 1176 us (two parts of q and p: one tile, so
// products and softmax take turns), fp16 q 840 us (two parts of p, which spill
// 216 bytes a thread; bf16's kernel 56).  A step of 256 rows x 128 tokens takes
// about 3.4 us: the MMAs alone about half of it, the softmax about as much.
//
// Split.  Many units (row block x head): CTAs take them from a counter.  Few: the
// line of their steps is cut evenly, each CTA leaves at most two partial results
// and qg_attn_join_kernel joins them in the order of the line (4 sequences of up
// to 4100 tokens, 256 rows each: 115 us whole, 65 split).
//
// Shared memory: q 64 KB, four operand slots of 32 KB (K, V, K, V), two slots
// of raw codes of 16 KB.  Tensor memory: S (128 columns) and O (dim columns)
// of each tile.
#include <atomic>

#include "kv_attention.cuh"
#include "launch_common.cuh"

namespace qg {
namespace {

constexpr int kStepTokens = 128;
constexpr int kMaxPromptCtas = 160;  // that share the line of steps: two part slots each
// Fewer units than this many a CTA are split: 32 units 115 us whole, 65 split;
// 192 units 178 / 160, 256 units 180 / 186, 512 units 258 / 295.
constexpr int kSplitBelow = 2;
constexpr int kLeastSteps = 2;  // of a CTA's share of the line (at 4, 1000 tokens x 256 rows: 37 us for 32)
static_assert(int64_t(kMaxPromptCtas) * 2 * 256 * (128 + 2) * 4 <= kWsPartBytes, "partials exceed the workspace");
static_assert(kMaxPromptCtas * 32 <= kWsTotal - kWsSplits, "splits exceed the workspace");
constexpr uint32_t kOps = 4;       // operand slots
constexpr uint32_t kRaws = 2;      // raw slots
constexpr uint32_t kUnits = 4;   // units handed to the roles ahead
constexpr uint32_t kScales = 8;    // steps whose scales are held
constexpr uint32_t kRow8 = 1024;  // bytes of 8 operand rows of 128 bytes

template <int DP, int QP>  // QP: f16 parts of q
struct PShape {
    static constexpr int TILES = QP == 1 ? 2 : 1;
    static constexpr int ROWS = 128 * TILES;
    static constexpr int kQTile = 128 * DP * 2;
    static constexpr int kOp = kStepTokens * DP * 2;
    static constexpr int kRaw = kStepTokens * DP;
    static constexpr int off_op = TILES * QP * kQTile;
    static constexpr int off_raw = off_op + kOps * kOp;
    static constexpr int off_scale = off_raw + kRaws * kRaw;
    static constexpr int off_bar = off_scale + kScales * 8 * 16;
    static constexpr int smem = off_bar + 320;
    static constexpr int warps = TILES * 4 + 4 + 2;
    static constexpr int kCols = TILES == 2 ? 512 : 256;  // tensor memory: 256 columns a tile
    static_assert(smem <= 232448, "shared memory");
};

// K-major operand with the 128-byte swizzle: rows of 128 bytes (64 f16), 8-row
// groups kRow8 apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t saddr) {
    uint64_t d = (saddr >> 4) & 0x3FFFu;
    d |= static_cast<uint64_t>(1) << 16;
    d |= static_cast<uint64_t>((kRow8 >> 4) & 0x3FFFu) << 32;
    d |= static_cast<uint64_t>(1) << 46;
    d |= static_cast<uint64_t>(2) << 61;
    return d;
}

// kind::f16, f16 operands, both K-major, fp32 sums, 128 rows x n columns.
__host__ __device__ constexpr uint32_t f16_desc(int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (8u << 24);
}

__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(accumulate) : "memory");
}
__device__ __forceinline__ void commit_to(uint64_t* bar) {
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                 ::"r"(smem_u32(bar)) : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void arrive_on(uint64_t* bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// 32 columns of this warp's 32 lanes; the values are there after tmem_loaded().
__device__ __forceinline__ void tmem_load32(uint32_t addr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
        "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
        "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]),
          "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]),
          "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(addr));
}
__device__ __forceinline__ void tmem_loaded() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_store32(uint32_t addr, const uint32_t (&w)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
        "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
        "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};"
        ::"r"(addr), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7]),
          "r"(w[8]), "r"(w[9]), "r"(w[10]), "r"(w[11]), "r"(w[12]), "r"(w[13]), "r"(w[14]), "r"(w[15]),
          "r"(w[16]), "r"(w[17]), "r"(w[18]), "r"(w[19]), "r"(w[20]), "r"(w[21]), "r"(w[22]), "r"(w[23]),
          "r"(w[24]), "r"(w[25]), "r"(w[26]), "r"(w[27]), "r"(w[28]), "r"(w[29]), "r"(w[30]), "r"(w[31])
        : "memory");
}
__device__ __forceinline__ void tmem_stored() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// A piece of work: steps j0 .. j1 - 1 of the keys of one row block and head.
// Where that is not all its keys, the result is partial and goes to part slot
// `part`.
struct Piece {
    int b, h, row_first, n, len, row0, j0, j1, part;  // b < 0: no more; part < 0: whole
};

// A row block's place in its sequence.
template <int ROWS>
struct Block {
    int row_first, nrows, seen_least, seen_most, steps;
    __device__ static int count(int n, int group) {
        return static_cast<int>((static_cast<int64_t>(n) * group + ROWS - 1) / ROWS);
    }
    __device__ Block(int first, int n, int len, int group) : row_first(first) {
        nrows = n * group;
        const int i_last = (min(row_first + ROWS, nrows) - 1) / group;
        seen_most = max(0, len - n + i_last + 1);
        seen_least = len - n + row_first / group + 1;
        steps = (seen_most + kStepTokens - 1) / kStepTokens;
    }
};

// Finds places on the line of all units (for each sequence its row blocks from
// the last, which sees most, to the first, each for all heads), by a whole
// warp, forward only.  STEPS: the line is measured in steps (a unit without
// keys counts as one), else in units.
template <int ROWS, bool STEPS>
struct Walk {
    int b0 = -32, n, len, row0;  // of this lane's sequence, b0 + lane
    int64_t base = 0, chunk = 0, upto = 0;
    __device__ static int64_t span(const AttnArgs& a, int n, int len) {
        const int blocks = Block<ROWS>::count(n, a.group);
        int64_t sum = blocks;
        if (STEPS) {
            sum = 0;
            for (int i = 0; i < blocks; ++i) sum += max(1, Block<ROWS>(i * ROWS, n, len, a.group).steps);
        }
        return sum * a.c.heads;
    }
    // The next 32 sequences; false after the last.
    __device__ bool more(const AttnArgs& a) {
        const int lane = threadIdx.x & 31;
        b0 += 32;
        base += chunk;
        if (b0 >= a.batch) return false;
        n = len = row0 = 0;
        if (b0 + lane < a.batch) {
            const Seq sq = sequence(a, b0 + lane);
            n = sq.n, len = sq.len, row0 = a.starts[b0 + lane];
        }
        upto = span(a, n, len);
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t x = __shfl_up_sync(~0u, upto, o);
            if (lane >= o) upto += x;
        }
        chunk = __shfl_sync(~0u, upto, 31);
        return true;
    }
    // The unit at `at`; the place in the unit in `in` (STEPS).
    __device__ bool to(const AttnArgs& a, int64_t at, Piece& u, int64_t& in) {
        while (at >= base + chunk)
            if (!more(a)) return false;
        const int which = __popc(__ballot_sync(~0u, upto <= at - base));
        u.b = b0 + which;
        u.n = __shfl_sync(~0u, n, which);
        u.len = __shfl_sync(~0u, len, which);
        u.row0 = __shfl_sync(~0u, row0, which);
        const int64_t below = __shfl_sync(~0u, upto, which ? which - 1 : 0);
        in = at - base - (which ? below : 0);
        int block = Block<ROWS>::count(u.n, a.group) - 1, steps = 1;
        if (STEPS) {
            for (;; --block) {
                steps = max(1, Block<ROWS>(block * ROWS, u.n, u.len, a.group).steps);
                if (in < static_cast<int64_t>(steps) * a.c.heads) break;
                in -= static_cast<int64_t>(steps) * a.c.heads;
            }
        } else {
            const int64_t back = in / a.c.heads;
            block -= static_cast<int>(back);
            in -= back * a.c.heads;
        }
        u.row_first = block * ROWS;
        u.h = static_cast<int>(in) / steps;
        in -= static_cast<int64_t>(u.h) * steps;
        return true;
    }
};

template <int DP, int QP, int PP, bool INT8>  // PP: f16 parts of p
__global__ void __launch_bounds__(PShape<DP, QP>::warps * 32, 1)
qg_attn_prompt_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap kmap,
                      const __grid_constant__ CUtensorMap vmap, const bool may_split) {
    using F = PShape<DP, QP>;
    constexpr int TILES = F::TILES;
    extern __shared__ __align__(1024) unsigned char smem[];
    float4* scales = reinterpret_cast<float4*>(smem + F::off_scale);  // [kScales][8]: ks, vs, there, log2 vs
    uint64_t* raw_full = reinterpret_cast<uint64_t*>(smem + F::off_bar);
    uint64_t* raw_empty = raw_full + kRaws;
    uint64_t* op_full = raw_empty + kRaws;
    uint64_t* op_empty = op_full + kOps;
    uint64_t* s_full = op_empty + kOps;   // [2]
    uint64_t* p_full = s_full + 2;        // [2]
    uint64_t* q_full = p_full + 2;        // [2]
    uint64_t* o_done = q_full + 2;        // [2]
    uint64_t* t_left = o_done + 2;        // [2]
    uint64_t* sc_full = t_left + 2;       // [kScales]
    uint64_t* unit_full = sc_full + kScales;
    uint64_t* unit_empty = unit_full + kUnits;
    static_assert((2 * kRaws + 2 * kOps + 10 + kScales + 2 * kUnits) * 8 <= 320, "barriers");
    __shared__ Piece units[kUnits];
    __shared__ uint32_t tmem_slot;
    __shared__ volatile int nan_unit[8];

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const KVLayer& c = a.c;
    if ((smem_u32(smem) & 1023u) != 0) {  // the swizzled operands need it; the same in all threads
        if (tid == 0) atomicOr(a.status, kStatusBounds);
        return;
    }
    if (tid == 0) {
        for (int i = 0; i < kRaws; ++i) mbar_init(raw_full + i, 1), mbar_init(raw_empty + i, 4);
        for (int i = 0; i < kOps; ++i) mbar_init(op_full + i, 4), mbar_init(op_empty + i, 1);
        for (int i = 0; i < 2; ++i) {
            mbar_init(s_full + i, 1);
            mbar_init(p_full + i, 4);
            mbar_init(q_full + i, 4);
            mbar_init(o_done + i, 1);
            mbar_init(t_left + i, 4);
        }
        for (int i = 0; i < kScales; ++i) mbar_init(sc_full + i, 1);
        for (int i = 0; i < kUnits; ++i) mbar_init(unit_full + i, 1), mbar_init(unit_empty + i, TILES * 4 + 5);
        fence_mbar_init();
    }
    if (tid < 8) nan_unit[tid] = 0;
    if (warp == F::warps - 1) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&tmem_slot)), "r"(F::kCols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = tmem_slot;
    // A wait that gave up ends all further waits, copies and MMAs of its
    // thread: the kernel then runs to its end within a few wait limits.
    bool dead = false;
    auto wait = [&](uint64_t* bar, uint32_t parity) {  // by whole warps
        if (!dead) dead = __any_sync(~0u, !mbar_wait_bounded(bar, parity & 1u, a.status));
    };
    // The next piece, as the copying warp hands it to the others; false after
    // the last.
    uint32_t turn = 0;
    Piece w;
    auto next_unit = [&]() {
        const uint32_t slot = turn % kUnits;
        wait(unit_full + slot, turn / kUnits);
        w = units[slot];
        __syncwarp();
        if (lane == 0) arrive_on(unit_empty + slot);
        ++turn;
        return !dead && w.b >= 0;
    };

    if (warp == F::warps - 2) {
        // ---------------------------------------------------------- copies
        // Many units: the next one comes from a counter that all CTAs share, the
        // longest of a sequence first, so that the CTAs end together.  Few: the
        // line of their steps is cut evenly among the CTAs.
        Walk<F::ROWS, false> by_unit;
        Walk<F::ROWS, true> by_step;
        int64_t total = 0;
        while (by_unit.more(a)) total += by_unit.chunk;
        const int ctas = min(static_cast<int>(gridDim.x), kMaxPromptCtas);
        const bool split = may_split && total < static_cast<int64_t>(kSplitBelow) * ctas;
        by_unit = Walk<F::ROWS, false>();
        int64_t at = 0, end = 0;
        if (may_split && lane == 0 && static_cast<int>(blockIdx.x) < kMaxPromptCtas)
            a.splits[2 * blockIdx.x] = make_int4(0, 0, 0, 0);
        Line line(0, 1);
        if (split) {
            const int64_t all = total;
            total = 0;
            while (by_step.more(a)) total += by_step.chunk;
            by_step = Walk<F::ROWS, true>();
            line = Line(total, static_cast<int>(min(static_cast<int64_t>(ctas), max(all, total / kLeastSteps))));
            if (static_cast<int>(blockIdx.x) < line.ctas) at = line.first(blockIdx.x), end = line.first(blockIdx.x + 1);
        }
        uint32_t o = 0, g = 0;  // raw tiles and steps over the life of the kernel
        uint32_t sent = 0;      // raw tiles whose copies were issued
        for (;; ++turn) {
            const uint32_t slot = turn % kUnits;
            if (turn >= kUnits) wait(unit_empty + slot, turn / kUnits - 1);
            bool there = !dead;
            int64_t in = 0;
            w.part = -1, w.j0 = 0;
            if (split) {
                there = there && at < end && by_step.to(a, at, w, in);
            } else {
                unsigned u = 0;
                if (lane == 0) u = atomicAdd(a.count + kCntPrompt, 1u);
                u = __shfl_sync(~0u, u, 0);
                there = there && by_unit.to(a, u, w, in);
            }
            if (there) {
                const int steps = Block<F::ROWS>(w.row_first, w.n, w.len, a.group).steps;
                w.j1 = steps;
                if (split) {
                    const int64_t start = at - in, stop = start + max(1, steps);
                    at = min(end, stop);
                    if (in > 0 || at < stop) {
                        w.j0 = static_cast<int>(in);
                        w.j1 = static_cast<int>(at - start);
                        w.part = 2 * blockIdx.x + (in == 0 ? 1 : 0);
                        if (in == 0 && lane == 0) {  // the first part: what the join has to know
                            a.splits[2 * blockIdx.x] = make_int4(line.of(stop - 1) - static_cast<int>(blockIdx.x) + 1,
                                                                 w.h, w.row_first, 0);
                            a.splits[2 * blockIdx.x + 1] = make_int4(w.row0, w.n, 0, 0);
                        }
                    }
                }
            } else {
                w.b = -1;
            }
            if (lane == 0) {
                units[slot] = w;
                arrive_on(unit_full + slot);
            }
            __syncwarp();
            if (!there) break;
            const Block<F::ROWS> blk(w.row_first, w.n, w.len, a.group);
            // its queries on their way to L2
            for (int r = w.row_first + lane; r < min(w.row_first + F::ROWS, blk.nrows); r += 32) {
                const int i_row = r / a.group;
                const int64_t qat = (static_cast<int64_t>(w.row0) + i_row) * a.q_row + (w.h * a.group + r - i_row * a.group) * a.q_head;
                const int size = a.type == QGKV_F32 ? 4 : 2;
                for (int at = 0; at < c.dim * size; at += 128)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(static_cast<const char*>(a.q) + qat * size + at));
            }
            const int32_t* table = a.table + static_cast<int64_t>(w.b) * a.width;
            auto look = [&](int j, float4& f) {  // page of this lane's 16 tokens of step j (lanes 0-7)
                int id = -1;
                f = make_float4(0.f, 0.f, 0.f, -INFINITY);
                const int tok = j * kStepTokens + lane * 16;
                if (lane < 8 && tok < blk.seen_most) {
                    id = table[tok >> c.log2p];
                    if (id >= 0 && id < c.pages) {
                        const int64_t at = static_cast<int64_t>(id) * c.heads + w.h;
                        f.x = __ldg(c.ks + at);
                        f.y = __ldg(c.vs + at);
                        f.z = 1.f;
                        if (f.y > 0.f) f.w = log2f(f.y);
                    } else {
                        id = -1;
                        atomicOr(a.status, kStatusBounds);
                    }
                }
                return id;
            };
            float4 f;
            int id = w.j0 < w.j1 ? look(w.j0, f) : -1;
            for (int j = w.j0; j < w.j1; ++j, ++g) {
                const int tok = (j * kStepTokens + lane * 16) & ((1 << c.log2p) - 1);
                const unsigned valid = __popc(__ballot_sync(~0u, id >= 0));
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++o) {
                    const int slot = o % kRaws;
                    if (o >= kRaws) wait(raw_empty + slot, o / kRaws - 1);
                    if (kv == 0) {
                        if (lane < 8) scales[(g % kScales) * 8 + lane] = f;
                        __syncwarp();
                        if (lane == 0) arrive_on(sc_full + g % kScales);
                    }
                    if (lane == 0) mbar_arrive_expect_tx(raw_full + slot, valid * 16 * DP);
                    __syncwarp();
                    if (id >= 0 && !dead)
                        tma_load_4d(smem + F::off_raw + slot * F::kRaw + lane * 16 * DP, kv ? &vmap : &kmap, 0, tok, w.h, id,
                                    raw_full + slot);
                    if (!dead) sent = o + 1;
                }
                if (j + 1 < w.j1) id = look(j + 1, f);
            }
        }
        if (dead)  // the copies in flight: shared memory is theirs until they land
            for (uint32_t x = sent > kRaws ? sent - kRaws : 0; x < sent; ++x)
                (void)mbar_wait_bounded(raw_full + x % kRaws, (x / kRaws) & 1u, a.status);
    } else if (warp == F::warps - 1) {
        // ---------------------------------------------------------- MMAs
        uint32_t o = 0;                // operands taken
        uint32_t ps = 0, qs = 0;       // probabilities (per tile) and queries taken
        while (next_unit()) {
            const int steps = w.j1 - w.j0;
            if (steps == 0) continue;
            for (int j = 0; j <= steps; ++j) {
                const uint32_t ko = o + 2 * j, vo = ko - 1;  // K of step j, V of step j - 1
                if (j < steps) wait(op_full + ko % kOps, ko / kOps);
                if (j > 0) wait(op_full + vo % kOps, vo / kOps);
#pragma unroll
                for (int t = 0; t < TILES; ++t) {
                    const uint32_t st = tmem + t * 256, ot = st + 128;
                    if (j == 0) wait(q_full + t, qs);
                    else wait(p_full + t, (ps + j - 1));
                    fence_after();
                    if (lane == 0 && !dead) {
                        if (j > 0) {
                            const uint64_t vb = operand_desc(smem_u32(smem + F::off_op + (vo % kOps) * F::kOp));
#pragma unroll
                            for (int p = PP - 1; p >= 0; --p)
#pragma unroll
                                for (int ks = 0; ks < 8; ++ks) {
                                    const uint32_t pa = PP == 1 ? st + ks * 8 : st + (ks >> 2) * 64 + (ks & 3) * 8 + p * 32;
                                    mma_ts(ot, pa, vb + (((ks >> 2) * (DP * 128) + (ks & 3) * 32) >> 4), f16_desc(DP),
                                           j > 1 || ks > 0 || p < PP - 1 ? 1u : 0u);
                                }
                            if (j == steps) commit_to(o_done + t);
                        }
                        if (j < steps) {
                            const uint64_t kb = operand_desc(smem_u32(smem + F::off_op + (ko % kOps) * F::kOp));
#pragma unroll
                            for (int p = QP - 1; p >= 0; --p) {  // the small parts first: half the roundings at full size
                                const uint64_t qb = operand_desc(smem_u32(smem + (t * QP + p) * F::kQTile));
#pragma unroll
                                for (int ks = 0; ks < DP / 16; ++ks)
                                    mma_ss(st, qb + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4),
                                           kb + (((ks >> 2) * 16384 + (ks & 3) * 32) >> 4), f16_desc(kStepTokens),
                                           p < QP - 1 || ks > 0 ? 1u : 0u);
                            }
                            commit_to(s_full + t);
                        }
                        if (t == TILES - 1) {
                            if (j > 0) commit_to(op_empty + vo % kOps);
                            if (j < steps) commit_to(op_empty + ko % kOps);
                        }
                    }
                    __syncwarp();
                }
            }
            o += 2 * steps;
            ps += steps;
            ++qs;
        }
    } else if (warp >= TILES * 4) {
        // ---------------------------------------------------------- 8 bits -> f16 operands
        const int ct = tid - TILES * 128, cw = ct >> 5;
        uint32_t o = 0, g = 0;
        int unit = 0;
        for (; next_unit(); ++unit) {
            const Block<F::ROWS> blk(w.row_first, w.n, w.len, a.group);
            for (int j = w.j0; j < w.j1; ++j, ++g) {
                const int tok0 = j * kStepTokens;
                const bool diagonal = tok0 + kStepTokens > blk.seen_least;  // some row does not see all of it
#pragma unroll
                for (int kv = 0; kv < 2; ++kv, ++o) {
                    const int rs = o % kRaws, os = o % kOps;
                    wait(raw_full + rs, o / kRaws);
                    if (o >= kOps) wait(op_empty + os, o / kOps - 1);
                    const unsigned char* raw = smem + F::off_raw + rs * F::kRaw;
                    unsigned char* op = smem + F::off_op + os * F::kOp;
                    const float4* sc = scales + (g % kScales) * 8;
                    if (kv == 0) {
                        constexpr int C16 = DP / 16;
#pragma unroll 4
                        for (int it = 0; it < C16; ++it) {
                            const int item = it * 128 + ct, token = item / C16, c16 = item % C16;
                            uint4 x = *reinterpret_cast<const uint4*>(raw + token * DP + c16 * 16);
                            if (sc[token >> 4].z == 0.f) x = make_uint4(0, 0, 0, 0);
                            uint32_t h[8];
                            const uint32_t in[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                if (INT8) {  // dims in the order 0, 2, 1, 3 (q's too)
                                    h[2 * i] = hsub2_1152((in[i] & 0x00FF00FFu) ^ 0x64806480u);
                                    h[2 * i + 1] = hsub2_1152(((in[i] >> 8) & 0x00FF00FFu) ^ 0x64806480u);
                                } else {
                                    h[2 * i] = e4m3x2_f16x2(in[i] & 0xFFFFu);
                                    h[2 * i + 1] = e4m3x2_f16x2(in[i] >> 16);
                                }
                            }
                            // two 16-byte chunks; lanes of the second 64 dims store theirs in the other order
                            const bool flip = (c16 >> 2) & 1;
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                const bool second = (e == 1) != flip;
                                const int ch = 2 * c16 + (second ? 1 : 0);
                                *reinterpret_cast<uint4*>(op + (ch >> 3) * 16384 + token * 128 + (((ch & 7) ^ (token & 7)) << 4)) =
                                    second ? make_uint4(h[4], h[5], h[6], h[7]) : make_uint4(h[0], h[1], h[2], h[3]);
                            }
                        }
                    } else {
                        constexpr int W = DP / 4;            // words of a token
                        constexpr int per = 32 / W;          // groups of 8 tokens a warp takes at once
                        const int word = lane % W;
                        bool found = false;
#pragma unroll 1
                        for (int it = 0; it < 4 / per; ++it) {
                            const int t0 = ((it * 4 + cw) * per + lane / W) * 8;
                            const int limit = sc[t0 >> 4].z == 0.f ? 0 : blk.seen_most - tok0;
                            uint32_t x[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) {
                                x[i] = *reinterpret_cast<const uint32_t*>(raw + (t0 + i) * DP + word * 4);
                                if (t0 + i >= limit) x[i] = 0;
                            }
                            if (!INT8 && diagonal) {
                                // NaN codes must not meet the zeros of rows that do not see them
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    const uint32_t is = __vcmpeq4(x[i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                                    found |= is != 0;
                                    x[i] &= ~is;
                                }
                            }
                            uint32_t r[4][4];
#pragma unroll
                            for (int i = 0; i < 4; ++i) v_codes<INT8>(x[2 * i], x[2 * i + 1], r[i]);
                            // the order of a lane's four dims turns with the lane, so that eight lanes meet eight bank groups
                            const int spin = (lane >> 1) & 3;
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                uint32_t s0 = spin & 1 ? r[i][1] : r[i][0], s1 = spin & 1 ? r[i][2] : r[i][1];
                                uint32_t s2 = spin & 1 ? r[i][3] : r[i][2], s3 = spin & 1 ? r[i][0] : r[i][3];
                                r[i][0] = spin & 2 ? s2 : s0, r[i][1] = spin & 2 ? s3 : s1;
                                r[i][2] = spin & 2 ? s0 : s2, r[i][3] = spin & 2 ? s1 : s3;
                            }
#pragma unroll
                            for (int i = 0; i < 4; ++i) {
                                const int dim = word * 4 + ((i + spin) & 3);
                                *reinterpret_cast<uint4*>(op + (t0 >> 6) * (DP * 128) + dim * 128 +
                                                          ((((t0 >> 3) & 7) ^ (dim & 7)) << 4)) =
                                    make_uint4(r[0][i], r[1][i], r[2][i], r[3][i]);
                            }
                        }
                        if (found) nan_unit[unit & 7] = unit + 1;
                    }
                    fence_proxy_async_smem();
                    __syncwarp();
                    if (lane == 0) {
                        arrive_on(op_full + os);
                        arrive_on(raw_empty + rs);
                    }
                }
            }
        }
    } else {
        // ---------------------------------------------------------- softmax, a thread a row
        const int t = warp >> 2, trow = tid & 127;
        const uint32_t lanes = static_cast<uint32_t>((warp & 3) * 32) << 16;
        const uint32_t st = tmem + t * 256 + lanes, ot = st + 128;
        uint32_t g = 0, ss = 0, os = 0;
        int unit = 0;
        for (;; ++unit, ++turn) {
            // The piece's description stays where it is and is read again after
            // the loop over its steps, which has no registers to spare for it.
            const uint32_t slot = turn % kUnits;
            wait(unit_full + slot, turn / kUnits);
            const volatile Piece& w = units[slot];
            if (dead || w.b < 0) break;
            const int j1 = w.j1, j0 = w.j0;
            int r = w.row_first + t * 128 + trow;
            const bool live = r < w.n * a.group;
            const int limit = live ? w.len - w.n + r / a.group + 1 : 0;
            float factor = 0.f;
            const bool busy = j0 < j1;
            if (busy) {
                // ---- queries: f16 parts of q * 2^e, the sign of the scale in
                // them.  QL lanes read a row, four dims each; eight reads on
                // their way at a time.
                constexpr int QL = DP / 4, QR = 32 / QL;
                const int i_row = r / a.group;
                const int64_t mine = live ? (static_cast<int64_t>(w.row0) + i_row) * a.q_row +
                                                (w.h * a.group + r - i_row * a.group) * a.q_head : -1;
                const int d = (lane % QL) * 4;
                unsigned char* qb = smem + t * QP * F::kQTile;
#pragma unroll 1
                for (int r0 = 0; r0 < 32; r0 += 8 * QR) {
                    uint4 raw[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const int64_t at = __shfl_sync(~0u, mine, r0 + i * QR + lane / QL);
                        raw[i] = load_q4(a.q, a.type, at + d, at >= 0 && d < c.dim);
                    }
#pragma unroll
                    for (int i = 0; i < 8; ++i) {
                        const float4 x = q4_values(raw[i], a.type);
                        const int row = r0 + i * QR + lane / QL;
                        float amax = fmaxf(fmaxf(fabsf(x.x), fabsf(x.y)), fmaxf(fabsf(x.z), fabsf(x.w)));
#pragma unroll
                        for (int k = QL / 2; k > 0; k >>= 1) amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, k));
                        int e = 141 - static_cast<int>((__float_as_uint(amax) >> 23) & 255u);
                        e = amax > 0.f && amax <= 3.4028235e38f ? min(e, 120) : 0;
                        float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
                        const float f = fabsf(a.scale_log2) * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
                        for (int k = 0; k < QR; ++k) {
                            const float fk = __shfl_sync(~0u, f, k * QL);
                            if (lane == r0 + i * QR + k) factor = fk;
                        }
                        if (a.scale_log2 < 0.f) up = -up;
                        const float y0 = x.x * up, y1 = (INT8 ? x.z : x.y) * up;
                        const float y2 = (INT8 ? x.y : x.z) * up, y3 = x.w * up;
                        uint2 h = make_uint2(pack_f16x2(y0, y1), pack_f16x2(y2, y3));
                        const int tr = (warp & 3) * 32 + row, ch = d >> 3;
                        unsigned char* dst = qb + (ch >> 3) * 16384 + tr * 128 + (((ch & 7) ^ (tr & 7)) << 4) + (d & 4) * 2;
                        *reinterpret_cast<uint2*>(dst) = h;
                        if (QP == 2)
                            *reinterpret_cast<uint2*>(dst + F::kQTile) = make_uint2(rest_f16x2(y0, y1, h.x), rest_f16x2(y2, y3, h.y));
                    }
                }
                fence_proxy_async_smem();
                fence_before();
                __syncwarp();
                if (lane == 0) arrive_on(q_full + t);
            }

            // References: m of the scores, d + m of score + log2 vs.  What is
            // stored of a probability is 2^(score + log2 vs + kr), at most
            // 2^14, the largest at least 2^(kBase - 1).  One f16 part keeps its
            // 11 bits 19 binary orders or more below that, so
            // references may be passed by 8 (at 2 every fourth step went
            // round again, at 8 hardly one after a unit's first); two parts
            // keep about 2^-35 of the largest, and 2 it is.
            constexpr int kPass = PP == 1 ? 8 : 2, kBase = 14 - kPass;
            float m = kNoRef, l = 0.f, kf = kBase, kr = kBase - kNoRef;
            int d = kNoOrder;
            bool huge = false;  // of the warp: scores are first put into tensor memory less m
            for (int j = j0; j < j1; ++j, ++g, ++ss) {
                wait(sc_full + g % kScales, g / kScales);
                wait(s_full + t, ss);
                fence_after();
                const float4* sc = scales + (g % kScales) * 8;
                const int left = limit - j * kStepTokens;  // columns that the row sees
                const bool all = __all_sync(~0u, left >= kStepTokens);
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const uint32_t sh = st + half * 64;
                    uint32_t hi[32], lo[PP == 2 ? 32 : 1];
                    float lh;
#pragma unroll 1
                    for (int round = 0;; ++round) {
                        // Optimistic: with the references as they are.  A score
                        // that passes them by more than kPass sends the warp round
                        // again, once: then none does.
                        bool passed = huge && round == 0;
                        lh = 0.f;
                        uint32_t va[32], vb[32];
                        tmem_load32(sh, va);
                        tmem_loaded();
                        tmem_load32(sh + 32, vb);
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            if (q == 1) tmem_loaded();
                            const uint32_t(&v)[32] = q == 0 ? va : vb;
#pragma unroll
                            for (int s = 0; s < 2; ++s) {
                                const int grp = half * 4 + q * 2 + s;
                                const float4 f = sc[grp];
                                const float lvk = f.w + kf;
                                const bool far = lvk < -100.f;  // a block whose values count for nothing (or are 0)
                                const float add = far ? kr - kf : f.w + kr, fx = huge ? 1.f : factor * f.x;
                                const f2 fs = {fx, fx}, c2 = {add, add};
                                f2 y[8];
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    y[i] = c2;
                                    ffma2(y[i], {__uint_as_float(v[s * 16 + 2 * i]), __uint_as_float(v[s * 16 + 2 * i + 1])}, fs);
                                }
                                if (!all || f.z == 0.f) {
                                    const int seen = f.z == 0.f ? 0 : left - grp * 16;
#pragma unroll
                                    for (int i = 0; i < 8; ++i) {
                                        if (2 * i >= seen) y[i].x = -INFINITY;
                                        if (2 * i + 1 >= seen) y[i].y = -INFINITY;
                                    }
                                }
                                float top = fmaxf(y[0].x, y[0].y);
#pragma unroll
                                for (int i = 1; i < 8; ++i) top = fmaxf(top, fmaxf(y[i].x, y[i].y));
                                passed |= top > (far ? static_cast<float>(kPass) : fminf(14.f, lvk + kPass));
                                f2 sum = {0.f, 0.f};
#pragma unroll
                                for (int i = 0; i < 8; ++i) {
                                    y[i].x = exp2_fast(y[i].x);
                                    y[i].y = exp2_fast(y[i].y);
                                    fadd2(sum, y[i]);
                                    const uint32_t two = far ? 0u : pack_f16x2(y[i].x, y[i].y);
                                    hi[q * 16 + s * 8 + i] = two;
                                    if (PP == 2) lo[(q * 16 + s * 8 + i) % (PP == 2 ? 32 : 1)] = far ? 0u : rest_f16x2(y[i].x, y[i].y, two);
                                }
                                lh = fmaf(sum.x + sum.y, far ? 1.f : exp2_fast(-lvk), lh);
                            }
                        }
                        if (round == 1 || !__any_sync(~0u, passed)) break;
                        float mn = m, tops[4];
#pragma unroll
                        for (int q = 0; q < 2; ++q) {
                            tmem_load32(sh + q * 32, va);
                            tmem_loaded();
#pragma unroll
                            for (int s = 0; s < 2; ++s) {
                                const int grp = half * 4 + q * 2 + s;
                                const float4 f = sc[grp];
                                const int seen = !passed || f.z == 0.f ? 0 : left - grp * 16;
                                float top = -INFINITY;
#pragma unroll
                                for (int i = 0; i < 16; ++i)
                                    if (i < seen) top = fmaxf(top, __uint_as_float(va[s * 16 + i]));
                                if (top != -INFINITY) top = __fmul_rn(top, factor * f.x);
                                tops[q * 2 + s] = top;
                                mn = fmaxf(mn, ceilf(top));
                            }
                        }
                        const int up = order_of(m - mn);
                        int dn = max(d + up, kNoOrder);
#pragma unroll
                        for (int s = 0; s < 4; ++s)
                            dn = max(dn, order_of(ceilf(tops[s] - mn + sc[half * 4 + s].w)));
                        const int k_old = min(kBase - d, 126), k_new = min(kBase - dn, 126);
                        const int order = k_new - k_old + up;
                        const float down = pow2i(order);
                        l *= pow2i(up);
                        m = mn, d = dn;
                        huge = __any_sync(~0u, huge || (m > kNoRef && fabsf(m) >= kHugeScore));
                        kf = static_cast<float>(max(k_new, -126));
                        kr = huge ? kf : kf - m;
                        if (j > j0) {
#pragma unroll 1
                            for (int q = 0; q < DP / 32; ++q) {
                                tmem_load32(ot + q * 32, va);
                                tmem_loaded();
#pragma unroll
                                for (int i = 0; i < 32; ++i) va[i] = __float_as_uint(__uint_as_float(va[i]) * down);
                                tmem_store32(ot + q * 32, va);
                            }
                        }
                        if (half == 1) {  // the first half's probabilities are stored already
                            tmem_stored();  // and have arrived before they are read back
                            // in two factors: f16 ends at 2^-24, what is stored
                            // may come down by 2^-39 before it rounds to 0
                            const int e = max(order, -40);
                            const float da = pow2i(e >> 1), db = pow2i(e - (e >> 1));
                            const uint32_t d2a = pack_f16x2(da, da), d2b = pack_f16x2(db, db);
#pragma unroll 1
                            for (int p = 0; p < PP; ++p) {
                                tmem_load32(st + p * 32, va);
                                tmem_loaded();
#pragma unroll
                                for (int i = 0; i < 32; ++i) {
                                    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(va[i]) : "r"(va[i]), "r"(d2a));
                                    asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(va[i]) : "r"(va[i]), "r"(d2b));
                                }
                                tmem_store32(st + p * 32, va);
                            }
                        }
                        if (huge) {
#pragma unroll 1
                            for (int q = 0; q < 2; ++q) {
                                tmem_load32(sh + q * 32, va);
                                tmem_loaded();
                                const float f0 = factor * sc[half * 4 + q * 2].x, f1 = factor * sc[half * 4 + q * 2 + 1].x;
#pragma unroll
                                for (int i = 0; i < 32; ++i)
                                    va[i] = __float_as_uint(__fsub_rn(__fmul_rn(__uint_as_float(va[i]), i < 16 ? f0 : f1), m));
                                tmem_store32(sh + q * 32, va);
                            }
                        }
                        tmem_stored();
                    }
                    l += lh;
                    if (PP == 1) {
                        tmem_store32(st + half * 32, hi);
                    } else {
                        tmem_store32(st + half * 64, hi);
                        tmem_store32(st + half * 64 + 32, reinterpret_cast<const uint32_t(&)[32]>(lo));
                    }
                }
                tmem_stored();
                fence_before();
                __syncwarp();
                if (lane == 0) arrive_on(p_full + t);
            }

            // ---- the row's result
            r = w.row_first + t * 128 + trow;
            const bool there = r < w.n * a.group;
            const int i_row = r / a.group;
            const int64_t to = (static_cast<int64_t>(w.row0) + i_row) * a.q_heads + w.h * a.group + r - i_row * a.group;
            const bool none = l == 0.f && m == kNoRef;
            const int down = none ? 0 : -min(kBase - d, 126);
            const float f1 = (none ? 0.f : 1.f / l) * pow2i(down >> 1), f2v = pow2i(down - (down >> 1));
            if (busy) {
                wait(o_done + t, os);
                ++os;
                fence_after();
            }
            // The rows go out through the tile's query memory (its MMAs are
            // done), so that a row's 16-byte pieces leave together.
            const int piece = a.type == QGKV_F32 ? 4 : 8;          // values of 16 bytes
            unsigned char* stage = smem + t * QP * F::kQTile + (warp & 3) * (QP * F::kQTile / 4);
            const int row_bytes = DP * 16 / piece;
            auto stage_out = [&](int q, const uint32_t(&v)[32]) {  // 32 dims of this lane's row
                if (a.type == QGKV_F32) {
#pragma unroll
                    for (int i = 0; i < 32; i += 4)
                        *reinterpret_cast<uint4*>(stage + lane * row_bytes + (((q * 8 + i / 4) ^ (lane & 7)) << 4)) =
                            make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
                } else {
#pragma unroll
                    for (int i = 0; i < 32; i += 8) {
                        uint32_t o4[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const float lo = __uint_as_float(v[i + 2 * k]), hi = __uint_as_float(v[i + 2 * k + 1]);
                            if (a.type == QGKV_F16) o4[k] = pack_f16x2(lo, hi);
                            else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o4[k]) : "f"(hi), "f"(lo));
                        }
                        *reinterpret_cast<uint4*>(stage + lane * row_bytes + (((q * 4 + i / 8) ^ (lane & 7)) << 4)) =
                            make_uint4(o4[0], o4[1], o4[2], o4[3]);
                    }
                }
            };
            // Partial results of this warp's rows: 32 references and 32 sums, then
            // pieces of 16 bytes, lane by lane, so that each read and write is 512
            // bytes wide.
            auto part_of = [&](int slot) {
                return a.part + (static_cast<int64_t>(slot) * (TILES * 4) + warp) * (32 * (DP + 2));
            };
            const bool ends = w.part < 0;
            float* mine_part = ends ? nullptr : part_of(w.part);
#pragma unroll 1
            for (int q = 0; q < DP / 32; ++q) {
                uint32_t v[32];
                if (busy) {
                    tmem_load32(ot + q * 32, v);
                    tmem_loaded();
                }
#pragma unroll
                for (int i = 0; i < 32; ++i) v[i] = none || !busy ? 0u : __float_as_uint(__uint_as_float(v[i]) * f1 * f2v);
                if (ends) {
                    stage_out(q, v);
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i)
                        __stcg(reinterpret_cast<uint4*>(mine_part + 64 + ((q * 8 + i) * 32 + lane) * 4),
                               make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]));
                }
            }
            // Rare: NaN codes of V among tokens that not every row sees; those
            // that this row sees, in this piece's keys.
            auto nans = [&](auto put) {
                if (INT8 || !there || nan_unit[unit & 7] != unit + 1) return;
                const int from = max(max(0, w.len - w.n + w.row_first / a.group + 1) / kStepTokens, w.j0) * kStepTokens;
                for (int tok = from; tok < min(w.len - w.n + i_row + 1, w.j1 * kStepTokens); ++tok) {
                    const int id = a.table[static_cast<int64_t>(w.b) * a.width + (tok >> c.log2p)];
                    if (id < 0 || id >= c.pages) continue;
                    const uint8_t* p = c.v + id * c.page_stride + static_cast<int64_t>(w.h) * c.head_stride +
                                       (tok & ((1 << c.log2p) - 1)) * c.token_stride;
                    for (int d = 0; d < c.dim; ++d)
                        if ((p[d] & 0x7F) == 0x7F) put(d, __int_as_float(0x7FC00000));
                }
            };
            if (!ends) {
                __stcg(mine_part + lane, none ? -INFINITY : m);
                __stcg(mine_part + 32 + lane, l);
                nans([&](int d, float nan) { __stcg(mine_part + 64 + ((d >> 2) * 32 + lane) * 4 + (d & 3), nan); });
            }
            __syncwarp();
            if (ends) {
                const int pieces = DP / piece, per = 32 / pieces;  // 16-byte pieces of a row, rows at once
                const int64_t my_to = there ? to * c.dim : -1;
#pragma unroll 4
                for (int r0 = 0; r0 < 32; r0 += per) {
                    const int row = r0 + lane / pieces, ch = lane % pieces;
                    const int64_t at = __shfl_sync(~0u, my_to, row) ;
                    if (at >= 0 && ch * piece < c.dim) {
                        const uint4 x = *reinterpret_cast<const uint4*>(stage + row * row_bytes + ((ch ^ (row & 7)) << 4));
                        if (a.type == QGKV_F32) *reinterpret_cast<uint4*>(static_cast<float*>(a.out) + at + ch * 4) = x;
                        else *reinterpret_cast<uint4*>(static_cast<uint16_t*>(a.out) + at + ch * 8) = x;
                    }
                }
                __syncwarp();  // ahead of what follows
                if (there && a.lse) a.lse[to] = none ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
                nans([&](int d, float nan) {
                    if (a.type == QGKV_F32) static_cast<float*>(a.out)[to * c.dim + d] = nan;
                    else if (a.type == QGKV_F16) static_cast<__half*>(a.out)[to * c.dim + d] = __float2half_rn(nan);
                    else static_cast<__nv_bfloat16*>(a.out)[to * c.dim + d] = __float2bfloat16_rn(nan);
                });
            }
            fence_before();
            // the tile's warps have left its query memory
            __syncwarp();
            if (lane == 0) arrive_on(t_left + t);
            if (lane == 0) arrive_on(unit_empty + slot);
            wait(t_left + t, static_cast<uint32_t>(unit));
        }
    }
    fence_before();
    __syncthreads();
    if (tid == 0 && atomicAdd(a.count + kCntPrompt + 1, 1u) == gridDim.x - 1) {
        // the last CTA to end leaves the counters ready for the next call
        a.count[kCntPrompt] = 0u;
        a.count[kCntPrompt + 1] = 0u;
    }
    if (warp == F::warps - 1) {
        fence_after();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(F::kCols) : "memory");
    }
}

// Joins the parts of the units whose keys were split, in the order of the line:
// a thread takes 32 dims of a row, a CTA those of a tile's 128 rows, so that
// the parts (16 KB of them a CTA and part) come through all SMs.  In the last
// CTA to arrive joining took about 2 us a part: one sequence of 256 query rows,
// 8000 tokens 69 us (here 57), 30000 tokens 110 us (89).
template <int DP, int TILES>
__global__ void __launch_bounds__(128) qg_attn_join_kernel(const AttnArgs a) {
    const int owner = blockIdx.x, t = blockIdx.y / (DP / 32), q = blockIdx.y % (DP / 32);
    const int4 u0 = a.splits[2 * owner], u1 = a.splits[2 * owner + 1];
    const int parts = u0.x, n = u1.y;
    const int64_t row0 = u1.x;
    if (parts <= 0) return;
    if (owner + parts > kMaxPromptCtas || row0 < 0 || row0 + n > a.rows) {  // a workspace that was not zeroed
        if (threadIdx.x == 0) atomicOr(a.status, kStatusBounds);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int r = u0.z + t * 128 + threadIdx.x;
    const bool live = r < n * a.group;
    auto part_of = [&](int i) {
        const int64_t slot = 2 * (owner + i) + (i == 0 ? 1 : 0);
        return a.part + (slot * (TILES * 4) + t * 4 + warp) * (32 * (DP + 2));
    };
    float top = -INFINITY, sum = 0.f;
#pragma unroll 8
    for (int i = 0; i < parts; ++i) top = fmaxf(top, __ldcg(part_of(i) + lane));
    const float ref = top == -INFINITY ? 0.f : top;
    float acc[32];
#pragma unroll
    for (int i = 0; i < 32; ++i) acc[i] = 0.f;
#pragma unroll 4
    for (int i = 0; i < parts; ++i) {
        const float* p = part_of(i);
        float4 x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = __ldcg(reinterpret_cast<const float4*>(p + 64 + ((q * 8 + k) * 32 + lane) * 4));
        const float f = exp2_fast(__ldcg(p + lane) - ref) * __ldcg(p + 32 + lane);
        sum += f;
#pragma unroll
        for (int k = 0; k < 8; ++k) {
            acc[4 * k] = fmaf(f, x[k].x, acc[4 * k]), acc[4 * k + 1] = fmaf(f, x[k].y, acc[4 * k + 1]);
            acc[4 * k + 2] = fmaf(f, x[k].z, acc[4 * k + 2]), acc[4 * k + 3] = fmaf(f, x[k].w, acc[4 * k + 3]);
        }
    }
    if (!live) return;
    const float inv = sum == 0.f ? 0.f : 1.f / sum;
    const int i_row = r / a.group;
    const int64_t to = (row0 + i_row) * a.q_heads + u0.y * a.group + r - i_row * a.group;
#pragma unroll
    for (int k = 0; k < 8; ++k)
        if (q * 32 + k * 4 < a.c.dim)
            store_out4(a.out, a.type, to * a.c.dim + q * 32 + k * 4,
                       make_float4(acc[4 * k] * inv, acc[4 * k + 1] * inv, acc[4 * k + 2] * inv, acc[4 * k + 3] * inv));
    if (q == 0 && a.lse) a.lse[to] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
}

template <int DP, int QP, int PP, bool INT8>
int launch_one(const AttnArgs& a, cudaStream_t s) {
    using F = PShape<DP, QP>;
    const int dev = current_device();
    const int sms = sm_count(dev);
    if (sms <= 0) return cuda_fail(cudaGetLastError());
    CUtensorMap kmap, vmap;
    if (!encode_cache(&kmap, a.c, a.c.k, DP, 16, false) || !encode_cache(&vmap, a.c, a.c.v, DP, 16, false))
        return cuda_fail(cudaGetLastError());
    // Rows that fill as many units as this leave none to split, and no join to launch.
    const int ctas = std::min(sms, kMaxPromptCtas);
    const bool split = a.rows * a.group / F::ROWS * a.c.heads < static_cast<int64_t>(kSplitBelow) * ctas;
    static std::atomic<bool> done[64];
    auto kern = qg_attn_prompt_kernel<DP, QP, PP, INT8>;
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, F::smem) != cudaSuccess)
            return cuda_fail(cudaGetLastError());
        done[dev].store(true, std::memory_order_release);
    }
    kern<<<sms, F::warps * 32, F::smem, s>>>(a, kmap, vmap, split);
    if (split) qg_attn_join_kernel<DP, F::TILES><<<dim3(ctas, F::TILES * (DP / 32)), 128, 0, s>>>(a);
    return launch_status();
}

template <int QP, int PP, bool INT8>
int launch_typed(const AttnArgs& a, cudaStream_t s) {
    return a.c.dim <= 64 ? launch_one<64, QP, PP, INT8>(a, s) : launch_one<128, QP, PP, INT8>(a, s);
}

template <bool INT8>
int launch_format(const AttnArgs& a, cudaStream_t s) {
    if (a.type == QGKV_F32) return launch_typed<2, 2, INT8>(a, s);
    // f16 outputs round as finely as one f16 part of p would: two
    if (a.type == QGKV_F16) return launch_typed<1, 2, INT8>(a, s);
    return launch_typed<1, 1, INT8>(a, s);
}

}  // namespace

int launch_attn_prompt(const AttnArgs& a, bool int8, cudaStream_t s) {
    return int8 ? launch_format<true>(a, s) : launch_format<false>(a, s);
}

}  // namespace qg
