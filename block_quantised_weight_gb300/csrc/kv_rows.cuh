// Attention of few query rows over the 8-bit paged cache (decode, short
// chunks): one pass over K and V with the running maximum and sum of the
// softmax.
//
// Mathematics.  For a row r of queries and the tokens t of its sequence
//   s[t] = (scale * log2 e * ks[page]) * (q . kcode[t]),  p[t] = 2^(s[t] - m)
//   l = sum p[t],   o = sum p[t] * vs[page] * vcode[t],   out = o / l
// Codes are exact in f16.  q * 2^j (a power of two that brings the row's
// largest value to [2^14, 2^15)) and p * vs * 2^k enter the products in f16:
// 16-bit queries enter as one part, exactly (to 2^-39 of the row's largest), fp32
// ones as two, hi and lo, about 22 bits; probabilities as one part (11 bits)
// where the output is bf16, else as two.  m is at least the running maximum less
// 2 and k is chosen by a bound u on s + log2 vs (k = 12 + m - u), so that what
// reaches o is at most 2^14 and its largest part at least 2^10 (u takes the next
// whole orders of s and of vs) however the scales of the blocks differ: half a
// step of f16 there, 2^-25, is 2^-35 of the largest.  m and u are whole numbers, which makes every rescaling a power of two,
// and they move only when a score passes them by more than 2: a step costs one
// vote instead of a reduction over its tokens.  (Scores from 2^22 on cost the
// reduction in every step.)
//
// Bound.  Decode reads every code once for 4 * group flops a byte: HBM-bound
// on the stream of codes if few instructions are spent on each (about 23 bytes
// a clock and SM come in).  Short of that the batch below is bound by latency:
// twelve warps an SM, by their registers, keep 39 % of the issue slots and 62 %
// of DRAM busy.  Both products are formed transposed, tokens by
// heads (K q^T) and dims by heads (V^T p^T), so that the 16-row operand is the
// codes and the 8 columns are query rows: group sizes up to 8 fill one column
// tile, and the codes are converted once for all of them.  Each warp streams
// its own tokens through a ring in shared memory that TMA fills (one box of 16
// tokens for K and for V, whatever the order of the cache; the swizzle lets
// every read below meet each bank once), so that bytes in flight cost no
// registers and no address arithmetic.  The order of a head's dims is free in
// q . k and in the rows of o: a lane takes 16 dims of one token for K and 8 or
// 16 dims of four tokens for V, whole vectors each.  p leaves the first
// product as the transpose of what the second takes; movmatrix turns it.
//
// Measured: 48 sequences of up to 4100 tokens, 32 / 8 heads of 128, e4m3: 55-56 us,
// 5.0 TB/s (fp32 q 58, fp16 57; heads of 256 dims 57); 3 of up to 131072, int8:
// 114-121 us, 5.2-5.5 TB/s; one of 777 tokens, 32 / 4 heads of 64: 8.2 us, all of
// it latency.
//
// Split.  The tokens of all (sequence, head, row block) are one line of
// 128-token tiles, cut evenly among the CTAs whatever the lengths; a CTA that
// holds a whole (sequence, head) writes its result, the others leave
// normalised partial results in the workspace and the last to arrive at a
// counter joins them in the order of the line (bits do not depend on the
// order of arrival).
#pragma once
#include <atomic>
#include <type_traits>

#include "kv_attention.cuh"
#include "launch_common.cuh"

namespace qg {
namespace {

constexpr int kTile = 128;        // tokens of a tile: 4 warps x 32
constexpr int kThreads = 128;
constexpr int kMaxCtas = 640;     // partial slots: 2 per CTA
constexpr int kPartFloats = 2048 + 32;  // rows * dims of a partial, then its references and sums
static_assert(int64_t(kMaxCtas) * 2 * kPartFloats * 4 <= kWsPartBytes, "partials exceed the workspace");
static_assert(kMaxCtas <= kCntPages, "counters overlap");
static_assert(int64_t(kMaxCtas) * 2 * kPartFloats * 4 <= kWsSlots - kWsPart, "partials meet a prefix's results");

constexpr int kUncut = 6;    // tiles that the longest sequence may be above a CTA's share and stay whole
constexpr int kBehind = INT_MIN;  // bit of a sequence's number of rows: it lies behind a prefix
constexpr int kMasked = 0x7FABCDEF;  // a NaN that no arithmetic gives: the score of a token that a row does not see

// What the template arguments fix: DC chunks of 64 dims.
template <int DC, int MT>
struct Shape {
    static constexpr int NS = DC <= 2 ? 2 : 1;       // 16-token subtiles of one warp step
    static constexpr int RU = 8 * MT;                // query rows of a unit
    static constexpr int DP = 64 * DC;
    static constexpr int RB = DC == 1 ? 64 : 128;    // bytes of a box row
    static constexpr int NB = DC == 4 ? 2 : 1;       // boxes of a token row
    static constexpr int kBox = 16 * RB;
    static constexpr int kSub = 2 * NB * kBox;       // K and V of a subtile
    static constexpr int kStage = NS * kSub;
    static constexpr int S = DC == 1 ? 3 : 2;        // stages of a warp's ring
    static constexpr int kRing = S * kStage;         // of one warp
    static_assert(RU * DP * 4 <= kRing, "a warp's result does not fit its ring");
    // shared memory: rings, queries, references and sums, row data, barriers, sequences and their prefix sums
    static constexpr int off_q(int) { return 4 * kRing; }
    static constexpr int off_ws(int parts) { return off_q(parts) + parts * MT * 4 * DC * 32 * 8; }
    static constexpr int off_rows(int parts) { return off_ws(parts) + 2 * 4 * RU * 4; }
    static constexpr int off_bar(int parts) { return off_rows(parts) + RU * 16; }
    static constexpr int off_pre(int parts) { return off_bar(parts) + 4 * S * 8; }
};

// Adds a prefix's results to those of a row's own tokens: `top` its reference
// (-inf: no token), `sum` and the normalised dims of this lane.  The launch that wrote
// them has ended (griddepcontrol.wait).  They are that launch's where the group that they name has this row
// and the `skip` tokens of its sequence, for the launch writes every row of such a group; where a plan's entries
// disagree they can be those of a call before (kStatusBounds).
template <int XV>
__device__ __forceinline__ void join_prefix(const AttnArgs& a, int64_t to, int skip, int row_lane, float& top, float& sum, float4 (&acc)[XV]) {
    grid_dependency_wait();
    const float4 first = __ldcg(a.own_ml + to);
    const int cta = __float_as_int(first.z) & 0xFFFF, row = __float_as_int(first.z) >> 16;
    const int group = __float_as_int(first.w) >> 16;
    int more = __float_as_int(first.w) & 0xFFFF;
    bool good = cta >= 1 && more <= kMaxPrefixCtas - cta && row >= 0 && row < a.slot_rows && group >= 0 && group < a.ngroups;
    if (!good) more = 0;
    const int4 entry = a.groups[good ? group : 0], before = group_before(a, good ? group : 0);
    const int64_t stride = static_cast<int64_t>(a.slot_rows) * (a.slot_dims + 2);
    const float* parts = a.slots + (more ? cta * stride + static_cast<int64_t>(row) * a.slot_dims : 0);
    const float2* ml = reinterpret_cast<const float2*>(a.slots + (more ? cta * stride + static_cast<int64_t>(a.slot_rows) * a.slot_dims : 0)) + row;
    float best = fmaxf(top, first.x);
    float ref = best == -INFINITY ? 0.f : best;
    const float mine = exp2_fast(top - ref) * sum, theirs = exp2_fast(first.x - ref) * first.y;
    float total = mine + theirs;
    float4 o[XV];
#pragma unroll
    for (int x = 0; x < XV; ++x) {
        const int d = 4 * (row_lane + 32 * x);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
        if (d < a.c.dim) v = __ldcg(reinterpret_cast<const float4*>(a.own + to * a.c.dim + d));
        o[x] = make_float4(mine * acc[x].x + theirs * v.x, mine * acc[x].y + theirs * v.y, mine * acc[x].z + theirs * v.z,
                           mine * acc[x].w + theirs * v.w);
    }
    const SharedGroup g = shared_group(a, entry, before);
    const int64_t in = to - static_cast<int64_t>(g.row0) * a.q_heads;
    good = good && g.tokens == skip && in >= 0 && in < static_cast<int64_t>(g.n) * a.q_heads;
    if (!good && row_lane == 0) atomicOr(a.status, kStatusBounds);
    // further parts, as many at once as their reads fit
    constexpr int N = 8 / XV;
    for (int i0 = 0; i0 < more; i0 += N) {
        float2 p[N];
        float4 v[N][XV];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            p[i] = make_float2(-INFINITY, 0.f);
            if (i0 + i < more) p[i] = __ldcg(ml + (i0 + i) * (stride / 2));
#pragma unroll
            for (int x = 0; x < XV; ++x) {
                const int d = 4 * (row_lane + 32 * x);
                v[i][x] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (i0 + i < more && d < a.c.dim) v[i][x] = __ldcg(reinterpret_cast<const float4*>(parts + (i0 + i) * stride + d));
            }
        }
        float high = best;
#pragma unroll
        for (int i = 0; i < N; ++i) high = fmaxf(high, p[i].x);
        const float to_ref = high == -INFINITY ? 0.f : high, down = exp2_fast(ref - to_ref);
        best = high, ref = to_ref;
        total *= down;
#pragma unroll
        for (int x = 0; x < XV; ++x) o[x].x *= down, o[x].y *= down, o[x].z *= down, o[x].w *= down;
#pragma unroll
        for (int i = 0; i < N; ++i) {
            const float w = exp2_fast(p[i].x - ref) * p[i].y;
            total += w;
#pragma unroll
            for (int x = 0; x < XV; ++x)
                o[x].x += w * v[i][x].x, o[x].y += w * v[i][x].y, o[x].z += w * v[i][x].z, o[x].w += w * v[i][x].w;
        }
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
#pragma unroll
    for (int x = 0; x < XV; ++x) acc[x] = make_float4(o[x].x * inv, o[x].y * inv, o[x].z * inv, o[x].w * inv);
    top = best, sum = total;
}

// QP, PP: f16 parts of q and of p.  SHARED: a sequence's tokens behind those that
// its group shares; the prefix's results, of the launch before, are joined at the end.
template <int DC, int MT, int QP, int PP, bool INT8, int MINB, bool SHARED>
__global__ void __launch_bounds__(kThreads, MINB)
qg_attn_rows_kernel(const AttnArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                    int grid) {
    using F = Shape<DC, MT>;
    constexpr int NS = F::NS, RU = F::RU, DP = F::DP, S = F::S;
    constexpr int VW = DC == 1 ? 2 : 4;    // 32-bit words of one V read
    constexpr int VL = F::NB;              // V reads per token row
    extern __shared__ __align__(1024) unsigned char smem[];
    uint2* qf = reinterpret_cast<uint2*>(smem + F::off_q(QP));         // [QP][MT][4 * DC][32]
    float* ws = reinterpret_cast<float*>(smem + F::off_ws(QP));        // [4][RU] largest |q|, later references
    float* wl = ws + 4 * RU;                                             // [4][RU] sums
    int64_t* orow = reinterpret_cast<int64_t*>(smem + F::off_rows(QP));  // [RU] output rows, -1 past the last
    int* limits = reinterpret_cast<int*>(orow + RU);                      // [RU] tokens that a row sees
    int64_t* pre = reinterpret_cast<int64_t*>(smem + F::off_pre(QP));  // [batch + 1]
    int2* seqs = reinterpret_cast<int2*>(pre + a.batch + 1);              // [batch] rows (SHARED: with kBehind), length
    __shared__ int64_t warp_sum[4];
    __shared__ int warp_most[4];
    __shared__ int last_flag;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const KVLayer& c = a.c;
    // this warp's ring of stages and their barriers
    unsigned char* ring = smem + warp * F::kRing;
    uint64_t* bar = reinterpret_cast<uint64_t*>(smem + F::off_bar(QP)) + warp * S;
    if (lane == 0) {
        for (int i = 0; i < S; ++i) mbar_init(bar + i, 1);
        fence_mbar_init();
        prefetch_tensormap(&kmap);
        prefetch_tensormap(&vmap);
    }
    __syncwarp();
    unsigned issued = 0, taken = 0;  // stages over the life of the kernel
    bool dead = false;  // a wait of this lane gave up: none follows, and no copy if it is lane 0, which issues them

    // ---- the line: prefix sums of the sequences' tiles (`whole`: of their blocks for all heads)
    auto rows_of = [](int2 q) { return SHARED ? q.x & ~kBehind : q.x; };
    auto units_of = [&](int2 q, bool whole) {
        const int64_t blocks = (static_cast<int64_t>(rows_of(q)) * a.group + RU - 1) / RU;
        return blocks * c.heads * (whole ? 1 : max(1, (q.y + kTile - 1) / kTile));
    };
    auto read = [&](int b) {
        Seq s = sequence(a, b);
        if (SHARED && shared_columns(a, b, s) > 0) s.n |= kBehind;
        return make_int2(s.n, s.len);
    };
    auto measure = [&](bool known, bool whole) {
        int64_t base = 0;
        for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
            const int b = b0 + tid;
            int64_t x = 0;
            if (b < a.batch) {
                if (!known) seqs[b] = read(b);
                x = units_of(seqs[b], whole);
            }
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(~0u, x, o);
                if (lane >= o) x += y;
            }
            if (b0) __syncthreads();  // the earlier sums have been read
            if (lane == 31) warp_sum[warp] = x;
            __syncthreads();
            for (int w = 0; w < warp; ++w) x += warp_sum[w];
            if (b < a.batch) pre[b + 1] = base + x;
            base += warp_sum[0] + warp_sum[1] + warp_sum[2] + warp_sum[3];
        }
        if (tid == 0) pre[0] = 0;
        __syncthreads();
    };
    // Behind a prefix sequences are short, and beginning and joining a piece costs as
    // much as some tiles: where the longest is hardly longer than a CTA's share,
    // none is cut, and the line counts them whole (48 sequences of up to 600 tokens
    // behind 8200: 42 us for 46 cut, 192 of up to 300 behind 24 prefixes 52 for 62).
    bool uncut = false;
    if (SHARED) {
        int64_t sum = 0;
        int longest = 0;
#pragma unroll 4
        for (int b = tid; b < a.batch; b += kThreads) {
            const int2 q = read(b);
            seqs[b] = q;
            sum += units_of(q, false);
            longest = max(longest, q.y);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
        longest = __reduce_max_sync(~0u, longest);
        if (lane == 0) warp_sum[warp] = sum, warp_most[warp] = longest;
        __syncthreads();
        const Line cut(warp_sum[0] + warp_sum[1] + warp_sum[2] + warp_sum[3], grid);
        longest = max(max(warp_most[0], warp_most[1]), max(warp_most[2], warp_most[3]));
        uncut = (longest + kTile - 1) / kTile <= cut.each + kUncut;
        __syncthreads();  // the sums have been read
    }
    measure(SHARED, uncut);
    const Line line(pre[a.batch], grid);
    const int cta = blockIdx.x;
    if (cta >= line.ctas) {
        if (SHARED) grid_dependency_wait();
        return;
    }
    const int64_t u_begin = line.first(cta), u_end = line.first(cta + 1);

    int64_t u = u_begin;
    while (u < u_end) {
        // ---- which (sequence, head, row block) and which of its tiles
        int lo = 0, hi = a.batch;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (pre[mid] <= u) lo = mid; else hi = mid;
        }
        // empty sequences share their successor's prefix: take the last with pre <= u that has tiles
        const int b = lo;
        const Seq sq = {rows_of(seqs[b]), seqs[b].y};
        const int64_t row0 = a.starts ? a.starts[b] : b;
        const int32_t* row_table = a.table + static_cast<int64_t>(b) * a.width;
        const int skip = SHARED && seqs[b].x < 0 ? a.skip[b] : 0;  // as read() found: it has left them out of the length
        if (SHARED) row_table += skip >> c.log2p;
        const int tiles = max(1, (sq.len + kTile - 1) / kTile);
        const int blocks = static_cast<int>((static_cast<int64_t>(sq.n) * a.group + RU - 1) / RU);
        const int64_t in = u - pre[b];
        const int hb = static_cast<int>(SHARED && uncut ? in : div64(in, tiles));
        const int tile0 = SHARED && uncut ? 0 : static_cast<int>(in - static_cast<int64_t>(hb) * tiles);
        const int h = hb / blocks, rb = hb - h * blocks;
        const int64_t span0 = u - tile0;
        const int seg = SHARED && uncut ? tiles : static_cast<int>(min(static_cast<int64_t>(tiles - tile0), u_end - u));
        const int nrows = sq.n * a.group;
        const int row_first = rb * RU;
        // tokens that the block's last row sees
        const int i_last = min(row_first + RU, nrows) - 1;
        const int seen_most = sq.len - sq.n + i_last / a.group + 1;
        const int seen_least = sq.len - sq.n + row_first / a.group + 1;
        const int tok0 = tile0 * kTile;
        const int tok1 = min((tile0 + seg) * kTile, seen_most);
        const int full_end = min(seen_least, tok1);  // up to here every row sees every token

        // ---- the stream of this warp: steps of 16 * NS tokens, 64 * NS apart.
        // Lane i holds the page and scales of the i-th 16-token subtile, in the
        // one or the other of two sets of 32 subtiles: the copies run ahead of
        // the steps by a stage or two.
        constexpr int step_tok = 64 * NS;
        const int warp_tok = tok0 + warp * 16 * NS;
        const int steps = tok1 > warp_tok ? (tok1 - warp_tok + step_tok - 1) / step_tok : 0;
        int id_c[2];
        float ks_c[2], vs_c[2];
        auto refill = [&](int batch32) {
            const int sub = batch32 * 32 + lane;
            const int tok = warp_tok + (sub / NS) * step_tok + (sub % NS) * 16;
            int id = -1;
            float k1 = 0.f, v1 = 0.f;
            if (tok < tok1) {
                id = row_table[tok >> c.log2p];
                if (id >= 0 && id < c.pages) {
                    const int64_t at = static_cast<int64_t>(id) * c.heads + h;
                    k1 = __ldg(c.ks + at);
                    v1 = __ldg(c.vs + at);
                } else {
                    id = -1;
                    atomicOr(a.status, kStatusBounds);
                }
            }
            if (batch32 & 1) id_c[1] = id, ks_c[1] = k1, vs_c[1] = v1;
            else id_c[0] = id, ks_c[0] = k1, vs_c[0] = v1;
        };
        auto issue = [&](int it) {  // fill the next stage with step `it`
            const int odd = (it * NS >> 5) & 1;
            if ((it * NS & 31) == 0) refill(it * NS >> 5);
            const int st = issued % S;
            int id[NS];
#pragma unroll
            for (int s = 0; s < NS; ++s) id[s] = __shfl_sync(~0u, odd ? id_c[1] : id_c[0], (it * NS + s) & 31);
            if (lane == 0 && !dead) {
                unsigned bytes = 0;
#pragma unroll
                for (int s = 0; s < NS; ++s) bytes += id[s] >= 0 ? F::kSub : 0;
                mbar_arrive_expect_tx(bar + st, bytes);
#pragma unroll
                for (int s = 0; s < NS; ++s)
                    if (id[s] >= 0) {
                        const int tok = (warp_tok + it * step_tok + s * 16) & ((1 << c.log2p) - 1);
                        unsigned char* dst = ring + st * F::kStage + s * F::kSub;
#pragma unroll
                        for (int x = 0; x < F::NB; ++x) {
                            tma_load_4d(dst + x * F::kBox, &kmap, x * 128, tok, h, id[s], bar + st);
                            tma_load_4d(dst + (F::NB + x) * F::kBox, &vmap, x * 128, tok, h, id[s], bar + st);
                        }
                    }
            }
            ++issued;
            __syncwarp();
        };

        // ---- queries: the column operand, scaled by a power of two per row.
        // Warp w takes the w-th four of a lane's 16 dims; a lane prepares row g
        // of each tile of 8.
        uint4 raw[MT][DC];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int r = row_first + mt * 8 + g;
            const int i_row = r / a.group;
            const int64_t qat = (row0 + i_row) * a.q_row + (h * a.group + r - i_row * a.group) * a.q_head;
#pragma unroll
            for (int cc = 0; cc < DC; ++cc) {
                const int d0 = DC == 1 ? t * 16 : (cc >> 1) * 128 + t * 32 + (cc & 1) * 16;
                raw[mt][cc] = load_q4(a.q, a.type, qat + d0 + 4 * warp, r < nrows && d0 < c.dim);
            }
        }
        // the previous segment's users of the rings and of the arrays below are
        // done; what they wrote to the rings stays ahead of the copies
        fence_proxy_async_smem();
        __syncthreads();
        for (int it = 0; it < S && it < steps; ++it) issue(it);
        if (tid < RU) {
            const int r = row_first + tid, i_row = r / a.group;
            orow[tid] = r < nrows ? (row0 + i_row) * a.q_heads + h * a.group + r - i_row * a.group : -1;
            limits[tid] = r < nrows ? sq.len - sq.n + i_row + 1 : 0;
        }
        float4 x[MT][DC];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float amax = 0.f;
#pragma unroll
            for (int cc = 0; cc < DC; ++cc) x[mt][cc] = q4_values(raw[mt][cc], a.type);
#pragma unroll
            for (int cc = 0; cc < DC; ++cc)
                amax = fmaxf(fmaxf(fmaxf(amax, fabsf(x[mt][cc].x)), fmaxf(fabsf(x[mt][cc].y), fabsf(x[mt][cc].z))),
                             fabsf(x[mt][cc].w));
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
            if (t == 0) ws[warp * RU + mt * 8 + g] = amax;
        }
        __syncthreads();
        float fac[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const float* am = ws + mt * 8 + g;
            const float amax = fmaxf(fmaxf(am[0], am[RU]), fmaxf(am[2 * RU], am[3 * RU]));
            // 2^e with amax * 2^e in [2^14, 2^15); 1 for zero or non-finite rows
            int e = 141 - static_cast<int>((__float_as_uint(amax) >> 23) & 255u);
            e = amax > 0.f && amax <= 3.4028235e38f ? min(e, 120) : 0;
            const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
            fac[mt] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
            for (int cc = 0; cc < DC; ++cc) {
                // the dims in the order that k_codes gives a word's bytes
                const float x0 = x[mt][cc].x * up, x1 = (INT8 ? x[mt][cc].z : x[mt][cc].y) * up;
                const float x2 = (INT8 ? x[mt][cc].y : x[mt][cc].z) * up, x3 = x[mt][cc].w * up;
                uint2 f;
                f.x = pack_f16x2(x0, x1);
                f.y = pack_f16x2(x2, x3);
                qf[(mt * 4 * DC + cc * 4 + warp) * 32 + lane] = f;
                if (QP == 2) {
                    uint2 fl;
                    fl.x = rest_f16x2(x0, x1, f.x);
                    fl.y = rest_f16x2(x2, x3, f.y);
                    qf[((MT + mt) * 4 * DC + cc * 4 + warp) * 32 + lane] = fl;
                }
            }
        }
        __syncthreads();
        // the scores a lane gets are those of rows 2t and 2t + 1 of each tile
        float qfac[MT][2];
        int limit[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int r = mt * 8 + 2 * t + i;
                qfac[mt][i] = __shfl_sync(~0u, fac[mt], (2 * t + i) * 4);
                limit[mt][i] = limits[r];
            }

        float o[MT][4 * DC][4];
        float m[MT][2], pk[MT][2], l[MT][2];  // references of the scores, 2^k, sums
        int d[MT][2];                         // references of score + log2 vs, less m
        bool huge = false;                    // the same in all lanes
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[mt][i] = kNoRef;
                d[mt][i] = kNoOrder;
                pk[mt][i] = 1.f;
                l[mt][i] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 4 * DC; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[mt][j][i] = 0.f;
        }

        // lanes' byte offsets in a box: K rows g (+ 8), V rows 2t and 2t + 1 (+ 8), as the swizzle places them
        int koff[2], voff[2];
        if (DC == 1) {
            koff[0] = koff[1] = g * 64 + ((t ^ (g >> 1)) * 16);
            for (int i = 0; i < 2; ++i) voff[i] = (2 * t + i) * 64 + (((g >> 1) ^ t) * 16) + (g & 1) * 8;
        } else {
            for (int i = 0; i < 2; ++i) koff[i] = g * 128 + (((2 * t + i) ^ g) * 16);
            for (int i = 0; i < 2; ++i) voff[i] = (2 * t + i) * 128 + ((g ^ (2 * t + i)) * 16);
        }
        // One step; `full`: every row sees every token of it.
        auto step = [&](int it, auto full) {
            const int tok = warp_tok + it * step_tok;
            const unsigned char* stage = ring + (taken % S) * F::kStage;
            float ks[NS], vs[NS];
            bool there[NS];
            const int odd = (it * NS >> 5) & 1;
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int from = (it * NS + s) & 31;
                there[s] = full || __shfl_sync(~0u, odd ? id_c[1] : id_c[0], from) >= 0;
                ks[s] = __shfl_sync(~0u, odd ? ks_c[1] : ks_c[0], from);
                vs[s] = __shfl_sync(~0u, odd ? vs_c[1] : vs_c[0], from);
            }
            if (!mbar_try_wait(bar + taken % S, (taken / S) & 1) && !dead &&
                !mbar_wait_bounded(bar + taken % S, (taken / S) & 1, a.status)) {
                dead = true;
                for (unsigned x = taken; lane == 0 && x != issued; ++x)  // the copies in flight, once more
                    (void)mbar_wait_bounded(bar + x % S, (x / S) & 1, a.status);
            }
            __syncwarp();  // lanes leave the wait one by one; the products below take whole warps
            // scores: rows are tokens g and g + 8 of a subtile, columns the query rows 2t and 2t + 1
            float sc[MT][NS][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[mt][s][i] = 0.f;
            // the products with the small parts of fp32 queries have sums of their
            // own: half the roundings at a score's full size
            float low[MT][NS][4];
            if (QP == 2) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int s = 0; s < NS; ++s)
#pragma unroll
                        for (int i = 0; i < 4; ++i) low[mt][s][i] = 0.f;
            }
#pragma unroll
            for (int cc = 0; cc < DC; ++cc) {
                uint4 k4[NS][2];
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int j = 0; j < 2; ++j)
                        k4[s][j] = *reinterpret_cast<const uint4*>(stage + s * F::kSub + (cc >> 1) * F::kBox +
                                                                   j * 8 * F::RB + koff[cc & 1]);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t ka[NS][4];
#pragma unroll
                    for (int s = 0; s < NS; ++s)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint4& q4 = k4[s][j];
                            k_codes<INT8>(w == 0 ? q4.x : w == 1 ? q4.y : w == 2 ? q4.z : q4.w, ka[s][j], ka[s][j + 2]);
                        }
#pragma unroll
                    for (int p = 0; p < QP; ++p)
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            const uint2 f = qf[((p * MT + mt) * 4 * DC + cc * 4 + w) * 32 + lane];
#pragma unroll
                            for (int s = 0; s < NS; ++s)
                                mma16816(p ? low[mt][s] : sc[mt][s], ka[s][0], ka[s][1], ka[s][2], ka[s][3], f.x, f.y);
                        }
                }
            }
            if (QP == 2) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int s = 0; s < NS; ++s)
#pragma unroll
                        for (int i = 0; i < 4; ++i) sc[mt][s][i] += low[mt][s][i];
            }
            // vs < 2^evs, the same in all lanes
            int evs[NS];
#pragma unroll
            for (int s = 0; s < NS; ++s)
                evs[s] = vs[s] > 0.f ? static_cast<int>((__float_as_uint(vs[s]) >> 23) & 255u) - 126 : kNoOrder;
            if (!full) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int s = 0; s < NS; ++s)
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int mine = tok + s * 16 + g + 8 * (i >> 1);
                            if (mine >= limit[mt][i & 1] || mine >= tok1 || !there[s]) sc[mt][s][i] = __int_as_float(kMasked);
                        }
            }
            uint32_t pb[PP][MT][NS][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float y[NS][4];
                auto relative = [&](auto rounded) {  // scores less their reference
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        const float f0 = qfac[mt][0] * ks[s], f1 = qfac[mt][1] * ks[s];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const float f = i & 1 ? f1 : f0;
                            y[s][i] = rounded && huge ? __fsub_rn(__fmul_rn(sc[mt][s][i], f), m[mt][i & 1])
                                                      : fmaf(sc[mt][s][i], f, -m[mt][i & 1]);
                            if (!full && __float_as_int(sc[mt][s][i]) == kMasked) y[s][i] = -INFINITY;
                        }
                    }
                };
                relative(std::false_type());
                bool passed = huge;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        const float top = fmaxf(y[s][i], y[s][i + 2]);
                        passed |= top > fminf(2.f, static_cast<float>(2 - (evs[s] - d[mt][i])));
                    }
                if (__any_sync(~0u, passed)) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        float mn = m[mt][i], tops[NS];
#pragma unroll
                        for (int s = 0; s < NS; ++s) {
                            const float f = qfac[mt][i] * ks[s];
                            float top = -INFINITY;
#pragma unroll
                            for (int j = i; j < 4; j += 2)
                                if (full || __float_as_int(sc[mt][s][j]) != kMasked)
                                    top = fmaxf(top, __fmul_rn(sc[mt][s][j], f));
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
                            tops[s] = ceilf(top);
                            mn = fmaxf(mn, tops[s]);
                        }
                        const int down = order_of(m[mt][i] - mn);
                        int dn = max(d[mt][i] + down, kNoOrder);
#pragma unroll
                        for (int s = 0; s < NS; ++s) dn = max(dn, order_of(tops[s] - mn) + evs[s]);
                        const int k_old = min(12 - d[mt][i], kMostK), k_new = min(12 - dn, kMostK);
                        const float os = pow2i(k_new - k_old + down);
                        l[mt][i] *= pow2i(down);
#pragma unroll
                        for (int j = 0; j < 4 * DC; ++j) {
                            o[mt][j][i] *= os;
                            o[mt][j][i + 2] *= os;
                        }
                        m[mt][i] = mn;
                        d[mt][i] = dn;
                        pk[mt][i] = pow2i(max(k_new, -126));
                        huge |= mn > kNoRef && fabsf(mn) >= kHugeScore;
                    }
                    huge = __any_sync(~0u, huge);
                    relative(std::true_type());
                }
#pragma unroll
                for (int s = 0; s < NS; ++s) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = exp2_fast(y[s][i]);
                        l[mt][i & 1] += p;
                        // p first: vs * 2^k may pass the range where p is 0 (a row
                        // that saw only small scales, and here sees nothing)
                        y[s][i] = p * pk[mt][i & 1] * vs[s];
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t hi2 = pack_f16x2(y[s][2 * j], y[s][2 * j + 1]);
                        pb[0][mt][s][j] = transpose8x8(hi2);
                        if (PP == 2)
                            pb[PP - 1][mt][s][j] = transpose8x8(rest_f16x2(y[s][2 * j], y[s][2 * j + 1], hi2));
                    }
                }
            }
            // o += V^T p^T.  Row tile 2w + i: dims with bytes 4w + 2i (rows 0-7) and 4w + 2i + 1 (rows 8-15)
#pragma unroll
            for (int s = 0; s < NS; ++s)
#pragma unroll
                for (int x = 0; x < VL; ++x) {
                    uint32_t vr[4][VW];  // tokens 2t, 2t + 1, 2t + 8, 2t + 9
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        const unsigned char* p = stage + s * F::kSub + (F::NB + x) * F::kBox + (j >> 1) * 8 * F::RB + voff[j & 1];
                        if (VW == 2) {
                            const uint2 v = *reinterpret_cast<const uint2*>(p);
                            vr[j][0] = v.x, vr[j][1] = v.y;
                        } else {
                            const uint4 v = *reinterpret_cast<const uint4*>(p);
                            vr[j][0] = v.x, vr[j][1] = v.y, vr[j][VW - 2] = v.z, vr[j][VW - 1] = v.w;
                        }
                        if (!full && (!there[s] || tok + s * 16 + 2 * t + (j & 1) + 8 * (j >> 1) >= tok1)) {
#pragma unroll
                            for (int w = 0; w < VW; ++w) vr[j][w] = 0;
                        }
                    }
                    if (!INT8 && !full && sq.n > 1) {
                        // A code that is NaN where not every row sees every token:
                        // taken out of the products and set where a row sees it.
                        uint32_t any = 0;
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int w = 0; w < VW; ++w) any |= __vcmpeq4(vr[j][w] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                        if (__any_sync(~0u, any != 0)) {
#pragma unroll
                            for (int w = 0; w < VW; ++w) {
                                uint32_t is[4], c01[4], c23[4];
#pragma unroll
                                for (int j = 0; j < 4; ++j) {
                                    is[j] = __vcmpeq4(vr[j][w] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                                    vr[j][w] &= ~is[j];
                                    is[j] &= 0x38383838u;  // e4m3 1.0 where the code is NaN
                                }
                                v_codes<false>(is[0], is[1], c01);
                                v_codes<false>(is[2], is[3], c23);
#pragma unroll
                                for (int mt = 0; mt < MT; ++mt) {
                                    const int lim = limits[mt * 8 + g];
                                    const int at = tok + s * 16 + 2 * t;
                                    const uint32_t sees0 = (at < lim ? 0x3C00u : 0u) | (at + 1 < lim ? 0x3C000000u : 0u);
                                    const uint32_t sees1 = (at + 8 < lim ? 0x3C00u : 0u) | (at + 9 < lim ? 0x3C000000u : 0u);
#pragma unroll
                                    for (int i = 0; i < 2; ++i) {
                                        float cnt[4] = {0.f, 0.f, 0.f, 0.f};
                                        mma16816(cnt, c01[2 * i], c01[2 * i + 1], c23[2 * i], c23[2 * i + 1], sees0, sees1);
                                        float(&d)[4] = o[mt][x * 2 * VW + 2 * w + i];
#pragma unroll
                                        for (int j = 0; j < 4; ++j)
                                            if (cnt[j] > 0.f) d[j] = __int_as_float(0x7FC00000);
                                    }
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        uint32_t c01[4], c23[4];
                        v_codes<INT8>(vr[0][w], vr[1][w], c01);
                        v_codes<INT8>(vr[2][w], vr[3][w], c23);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                                for (int p = 0; p < PP; ++p)
                                    mma16816(o[mt][x * 2 * VW + 2 * w + i], c01[2 * i], c01[2 * i + 1], c23[2 * i],
                                             c23[2 * i + 1], pb[p][mt][s][0], pb[p][mt][s][1]);
                    }
                }
            ++taken;
            __syncwarp();  // every lane has read the stage
            if (it + S < steps) issue(it + S);
        };
        // Steps of whole tokens for every row, while all pages are there; then the rest.
        int it = 0;
        const int whole_steps = full_end > warp_tok ? (full_end - warp_tok + step_tok - 16 * NS) / step_tok : 0;
        for (; it < whole_steps; ++it) {
            int least = 0;  // negative where a page is missing
#pragma unroll
            for (int s = 0; s < NS; ++s)
                least |= __shfl_sync(~0u, (it * NS >> 5) & 1 ? id_c[1] : id_c[0], (it * NS + s) & 31);
            if (least < 0) break;
            step(it, std::true_type());
        }
        for (; it < steps; ++it) step(it, std::false_type());

        // ---- this warp's normalised result, its reference and sum
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float sum = l[mt][i];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(~0u, sum, x);
                // NaN sums stay NaN; a row that saw nothing has a sum of 0
                const bool none = sum == 0.f && m[mt][i] == kNoRef;
                const int down = none ? 0 : -min(12 - d[mt][i], kMostK);
                const float f1 = pow2i(down >> 1), f2v = pow2i(down - (down >> 1));
                const float inv = none ? 0.f : 1.f / sum;
                const int r = mt * 8 + 2 * t + i;
                if (g == 0) ws[warp * RU + r] = none ? -INFINITY : m[mt][i], wl[warp * RU + r] = sum;
                float* dst = reinterpret_cast<float*>(ring) + r * DP + g * (4 * VW);
#pragma unroll
                for (int x = 0; x < VL; ++x)
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        const float(&d0)[4] = o[mt][x * 2 * VW + 2 * w];
                        const float(&d1)[4] = o[mt][x * 2 * VW + 2 * w + 1];
                        *reinterpret_cast<float4*>(dst + x * 128 + 4 * w) =
                            make_float4(d0[i] * inv * f1 * f2v, d0[i + 2] * inv * f1 * f2v, d1[i] * inv * f1 * f2v,
                                        d1[i + 2] * inv * f1 * f2v);
                    }
            }
        __syncthreads();
        // ---- join the four warps; then either the output or a partial result.
        // LPR lanes take a row, four dims each.
        constexpr int LPR = DC == 1 ? 16 : 32, XV = DC == 4 ? 2 : 1;
        const int row_lane = lane % LPR, row_of = warp * (32 / LPR) + lane / LPR;
        const bool whole = seg == tiles;
        float* part = a.part + static_cast<int64_t>(cta * 2 + (u == u_begin ? 0 : 1)) * kPartFloats;
        constexpr int kWarpFloats = F::kRing / 4;
        const float* wo = reinterpret_cast<const float*>(smem);  // the warps' results, kWarpFloats apart
#pragma unroll
        for (int r = row_of; r < RU; r += 128 / LPR) {
            const int64_t to = orow[r];
            if (to < 0) break;
            float w[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = ws[i * RU + r];
            const float mx = fmaxf(fmaxf(w[0], w[1]), fmaxf(w[2], w[3]));
            const float ref = mx == -INFINITY ? 0.f : mx;
#pragma unroll
            for (int i = 0; i < 4; ++i) w[i] = exp2_fast(w[i] - ref) * wl[i * RU + r];  // 0 for a warp without tokens, whose result is 0
            float sum = w[0] + w[1] + w[2] + w[3], top = mx;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            float4 acc[XV];
#pragma unroll
            for (int x2 = 0; x2 < XV; ++x2) {
                const int d = 4 * (row_lane + 32 * x2);
                acc[x2] = make_float4(0.f, 0.f, 0.f, 0.f);
                if (d >= c.dim) break;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const float4 v = *reinterpret_cast<const float4*>(wo + i * kWarpFloats + r * DP + d);
                    acc[x2].x += w[i] * v.x, acc[x2].y += w[i] * v.y, acc[x2].z += w[i] * v.z, acc[x2].w += w[i] * v.w;
                }
                acc[x2].x *= inv, acc[x2].y *= inv, acc[x2].z *= inv, acc[x2].w *= inv;
            }
            if (SHARED && whole && skip) join_prefix<XV>(a, to, skip, row_lane, top, sum, acc);
#pragma unroll
            for (int x2 = 0; x2 < XV; ++x2) {
                const int d = 4 * (row_lane + 32 * x2);
                if (d >= c.dim) break;
                if (whole) store_out4(a.out, a.type, to * c.dim + d, acc[x2]);
                else *reinterpret_cast<float4*>(part + r * c.dim + d) = acc[x2];
            }
            if (row_lane == 0) {
                if (!whole) part[2048 + r] = mx, part[2048 + 16 + r] = sum;
                else if (a.lse) a.lse[to] = sum == 0.f ? -INFINITY : ((SHARED && top != -INFINITY ? top : ref) + log2f(sum)) * 0.69314718055994531f;
            }
        }
        if (!whole) {
            const int first = line.of(span0);
            const int need = line.of(span0 + tiles - 1) - first + 1;
            __threadfence();
            __syncthreads();
            if (tid == 0) {
                const unsigned old = atomicAdd(a.count + first, 1u);
                last_flag = old == static_cast<unsigned>(need - 1);
                if (last_flag) a.count[first] = 0u;
                __threadfence();
            }
            __syncthreads();
            if (last_flag) {
                // The CTAs' partials in the order of the line.  Only the first
                // of them may hold this span in its second slot.
                const float* p0 = a.part + static_cast<int64_t>(first * 2 + (line.first(first) < span0 ? 1 : 0)) * kPartFloats;
                const float* p1 = a.part + static_cast<int64_t>(first) * 2 * kPartFloats;
                auto part_of = [&](int i) { return i == 0 ? p0 : p1 + static_cast<int64_t>(i) * 2 * kPartFloats; };
                // A lane's parts of the references and sums of its rows are all on
                // their way before the first is used; then 16 parts of a row at a time.
                constexpr int RW = RU * LPR / 128;  // rows of a lane
                int64_t to[RW];
                float m0[RW], l0[RW];
#pragma unroll
                for (int i = 0; i < RW; ++i) {
                    const int r = row_of + i * (128 / LPR);
                    to[i] = orow[r];  // the lanes of a dead row take part in the shuffles
                    m0[i] = -INFINITY, l0[i] = 0.f;
                    if (to[i] >= 0 && row_lane < need) {
                        m0[i] = __ldcg(part_of(row_lane) + 2048 + r);
                        l0[i] = __ldcg(part_of(row_lane) + 2048 + 16 + r);
                    }
                }
#pragma unroll
                for (int i = 0; i < RW; ++i) {
                    const int r = row_of + i * (128 / LPR);
                    const bool live = to[i] >= 0;
                    float mx = m0[i];
                    for (int j = LPR + row_lane; live && j < need; j += LPR) mx = fmaxf(mx, __ldcg(part_of(j) + 2048 + r));
#pragma unroll
                    for (int o2 = LPR / 2; o2 > 0; o2 >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, o2));
                    const float ref = mx == -INFINITY ? 0.f : mx;
                    float4 acc[XV];
#pragma unroll
                    for (int x2 = 0; x2 < XV; ++x2) acc[x2] = make_float4(0.f, 0.f, 0.f, 0.f);
                    float sum = 0.f;
                    for (int base = 0; base < need; base += LPR) {
                        float w = m0[i], lw = l0[i];
                        if (base) {
                            const bool held = live && base + row_lane < need;
                            w = held ? __ldcg(part_of(base + row_lane) + 2048 + r) : -INFINITY;
                            lw = held ? __ldcg(part_of(base + row_lane) + 2048 + 16 + r) : 0.f;
                        }
                        w = exp2_fast(w - ref) * lw;
                        sum += w;
                        for (int j0 = 0; j0 < LPR && base + j0 < need; j0 += 16) {
#pragma unroll
                            for (int x2 = 0; x2 < XV; ++x2) {
                                const int d = 4 * (row_lane + 32 * x2);
                                float4 v[16];
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    v[j] = make_float4(0.f, 0.f, 0.f, 0.f);
                                    if (live && d < c.dim && base + j0 + j < need)
                                        v[j] = __ldcg(reinterpret_cast<const float4*>(part_of(base + j0 + j) + r * c.dim + d));
                                }
#pragma unroll
                                for (int j = 0; j < 16; ++j) {
                                    const float wj = __shfl_sync(~0u, w, j0 + j, LPR);
                                    acc[x2].x += wj * v[j].x, acc[x2].y += wj * v[j].y;
                                    acc[x2].z += wj * v[j].z, acc[x2].w += wj * v[j].w;
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int o2 = LPR / 2; o2 > 0; o2 >>= 1) sum += __shfl_xor_sync(~0u, sum, o2);
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    float join_top = mx;
#pragma unroll
                    for (int x2 = 0; x2 < XV; ++x2)
                        acc[x2].x *= inv, acc[x2].y *= inv, acc[x2].z *= inv, acc[x2].w *= inv;
                    if (SHARED && skip && live) join_prefix<XV>(a, to[i], skip, row_lane, join_top, sum, acc);
#pragma unroll
                    for (int x2 = 0; x2 < XV; ++x2) {
                        const int d = 4 * (row_lane + 32 * x2);
                        if (live && d < c.dim) store_out4(a.out, a.type, to[i] * c.dim + d, acc[x2]);
                    }
                    if (live && row_lane == 0 && a.lse)
                        a.lse[to[i]] = sum == 0.f ? -INFINITY
                                                  : ((SHARED && join_top != -INFINITY ? join_top : ref) + log2f(sum)) * 0.69314718055994531f;
                }
            }
        }
        u += SHARED && uncut ? 1 : seg;
    }
    if (SHARED) grid_dependency_wait();  // no launch behind this one meets the one before
}

template <int DC, int MT, int QP, int PP, bool INT8, int MINB, bool SHARED>
int launch_one(const AttnArgs& a, cudaStream_t s) {
    const int dev = current_device();
    const int sms = sm_count(dev);
    if (sms <= 0) return cuda_fail(cudaGetLastError());
    using F = Shape<DC, MT>;
    constexpr int fixed = F::off_pre(QP);
    static_assert(F::off_rows(QP) % 16 == 0 && F::off_bar(QP) % 8 == 0 && F::off_q(QP) % 16 == 0, "alignment");
    CUtensorMap kmap, vmap;
    if (!encode_cache(&kmap, a.c, a.c.k, F::RB, 16, true) || !encode_cache(&vmap, a.c, a.c.v, F::RB, 16, true))
        return cuda_fail(cudaGetLastError());
    const int most = fixed + (QGKV_MAX_BATCH + 1) * 16;
    static std::atomic<bool> done[64];
    auto kern = qg_attn_rows_kernel<DC, MT, QP, PP, INT8, MINB, SHARED>;
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
            return cuda_fail(cudaGetLastError());
        done[dev].store(true, std::memory_order_release);
    }
    const int grid = std::min(sms * MINB, kMaxCtas);
    const int bytes = fixed + (a.batch + 1) * 16;
    if (!SHARED) {
        kern<<<grid, kThreads, bytes, s>>>(a, kmap, vmap, grid);
        return launch_status();
    }
    // beside the launch of the prefix, as its CTAs end
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kern, a, kmap, vmap, grid) != cudaSuccess) return cuda_fail(cudaGetLastError());
    return launch_status();
}

template <int QP, int PP, bool INT8, bool SHARED>
int launch_typed(const AttnArgs& a, cudaStream_t s) {
    // 16 rows a unit read the codes half as often as 8 do, with more registers
    // and so fewer CTAs; what they gain grows with what a code costs and with the
    // rows.  8 against 16 rows a unit, us, 16 sequences of up to 4100 tokens, bf16:
    //   int8, 128 dims: 16 rows 37.6 / 41.9, 24 rows 50.5 / 46.4, 64 rows 102 / 83.6
    //   e4m3, 64 dims:  24 rows 27.3 / 28.4, 32 rows 33.3 / 31.5, 64 rows 52.2 / 45.4
    //   e4m3, 128 dims: 48 rows 58.8 / 60.0, 64 rows 70.7 / 70.3, 128 rows 124 / 111
    // 256-dim heads keep 8 for their registers.
    // int8's conversions hold more registers: two CTAs an SM instead of three
    // (long documents 114 us for 118, though 48 sequences of up to 4100 tokens 64
    // for 61; e4m3's batch 58 us for 56 with two).
    const int few = INT8 ? 16 : a.c.dim <= 64 ? 24 : 48;
    const bool wide = a.rows * a.group > few * static_cast<int64_t>(a.batch);
    if (a.c.dim <= 64) return wide ? launch_one<1, 2, QP, PP, INT8, 3, SHARED>(a, s) : launch_one<1, 1, QP, PP, INT8, 3, SHARED>(a, s);
    if (a.c.dim <= 128)
        return wide ? launch_one<2, 2, QP, PP, INT8, 2, SHARED>(a, s) : launch_one<2, 1, QP, PP, INT8, INT8 ? 2 : 3, SHARED>(a, s);
    return launch_one<4, 1, QP, PP, INT8, 2, SHARED>(a, s);
}

}  // namespace

template <bool INT8, bool SHARED>
int launch_rows(const AttnArgs& a, cudaStream_t s) {
    if (a.type == QGKV_F32) return launch_typed<2, 2, INT8, SHARED>(a, s);
    // f16 outputs round as finely as one f16 part of p would: two
    if (a.type == QGKV_F16) return launch_typed<1, 2, INT8, SHARED>(a, s);
    return launch_typed<1, 1, INT8, SHARED>(a, s);
}

}  // namespace qg
