// Attention of few query rows over the 8-bit paged cache (decode, short
// chunks): one pass over K and V with the running maximum and sum of the
// softmax.
//
// Mathematics.  For a row r of queries and the tokens t of its sequence
//   s[t] = (scale * log2 e * ks[page]) * (q . kcode[t]),  p[t] = 2^(s[t] - m)
//   l = sum p[t],   o = sum p[t] * vs[page] * vcode[t],   out = o / l
// Codes are exact in f16.  q * 2^j (a power of two that brings the row's
// largest value to [2^14, 2^15)) and p * vs * 2^k enter the products in f16:
// 16-bit queries and their probabilities as one part (q exact, p rounded to 11
// bits, below the rounding of the output), fp32 ones as two, hi and lo, about
// 22 bits.  m is at least the running maximum less 2 and k is chosen by a
// bound u on s + log2 vs (k = 12 + m - u), so that what reaches o is at most
// 2^14 and its largest part near that however the scales of the blocks
// differ.  m and u are integers, which makes every rescaling a power of two,
// and they move only when a score passes them by more than 2: a step costs one
// vote instead of a reduction over its tokens.
//
// Bound.  Decode reads every code once for 4 * group flops a byte: HBM-bound
// on the stream of codes if few instructions are spent on each (about 23 bytes
// a clock and SM come in).  Both products are formed transposed, tokens by
// heads (K q^T) and dims by heads (V^T p^T), so that the 16-row operand is the
// codes and the 8 columns are query rows: group sizes up to 8 fill one column
// tile, and the codes are converted once for all of them.  The fragments are
// laid out so that codes go from global memory to registers and into the
// tensor instruction without shared memory: the order of a head's dims is
// free in q . k and in the rows of o, so a lane takes 16 dims of one token for
// K and 8 or 16 dims of four tokens for V, each a whole vector load, each quad
// or octet a whole row segment.  p leaves the first product as the transpose
// of what the second takes; movmatrix turns it.  The loads of the next step
// are issued as soon as the registers of the current one are consumed.
//
// Split.  The tokens of all (sequence, head, row block) are one line of
// 128-token tiles, cut evenly among the CTAs whatever the lengths; a CTA that
// holds a whole (sequence, head) writes its result, the others leave
// normalised partial results in the workspace and the last to arrive at a
// counter joins them in the order of the line (bits do not depend on the
// order of arrival).
#include <atomic>
#include <type_traits>

#include "kv_attention.cuh"
#include "launch_common.cuh"

namespace qg {
namespace {

constexpr int kTile = 128;        // tokens of a tile: 4 warps x 32
constexpr int kThreads = 128;
constexpr int kMaxCtas = 1536;    // partial slots: 2 per CTA
constexpr int kPartFloats = 2048 + 32;  // rows * dims of a partial, then its log-sums
static_assert(int64_t(kMaxCtas) * 2 * kPartFloats * 4 <= kWsPartBytes, "partials exceed the workspace");
static_assert(kMaxCtas <= kCntPages, "counters overlap");

// a / b for non-negative a and positive b, in 32 bits where they fit.
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// The line of tiles cut into pieces of equal size, the first `more` one longer.
struct Line {
    int64_t each;
    int more, ctas;
    __device__ Line(int64_t total, int grid) {
        ctas = total < grid ? static_cast<int>(total) : grid;
        each = ctas ? div64(total, ctas) : 0;
        more = static_cast<int>(total - each * ctas);
    }
    __device__ int64_t first(int cta) const { return each * cta + min(cta, more); }
    __device__ int of(int64_t tile) const {
        const int64_t long_part = (each + 1) * more;
        return static_cast<int>(tile < long_part ? div64(tile, each + 1) : more + div64(tile - long_part, each));
    }
};

constexpr int kNone = -(1 << 29);  // reference of a row that has seen nothing
constexpr int kMasked = 0x7FABCDEF;  // a NaN that no arithmetic gives: the score of a token that a row does not see

// 2^k exactly; 0 below the normal range.
__device__ __forceinline__ float pow2i(int k) {
    return __uint_as_float(static_cast<uint32_t>(min(max(k, -127), 127) + 127) << 23);
}
// The least integer >= x as a reference; kNone for -inf.
__device__ __forceinline__ int ceil_ref(float x) {
    return x == -INFINITY ? kNone : static_cast<int>(ceilf(fminf(fmaxf(x, -1.0e8f), 1.0e8f)));
}

template <int DC, int MT, int PARTS, bool INT8, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) qg_attn_rows_kernel(const AttnArgs a, int grid) {
    constexpr int NS = DC <= 2 ? 2 : 1;    // 16-token subtiles of one warp step
    constexpr int RU = 8 * MT;             // query rows of a unit
    constexpr int VW = DC == 1 ? 2 : 4;    // 32-bit words of one V load
    constexpr int VL = DC == 4 ? 2 : 1;    // V loads per token row
    constexpr int DP = 64 * DC;
    extern __shared__ __align__(16) unsigned char smem[];
    uint2* qf = reinterpret_cast<uint2*>(smem);                       // [PARTS][MT][4 * DC][32]
    float* wo = reinterpret_cast<float*>(qf + PARTS * MT * 4 * DC * 32);  // [4][RU][DP]
    float* ws = wo + 4 * RU * DP;                                     // [4][RU] log-sums
    float* wt = ws + 4 * RU;                                          // [RU] and scratch
    int64_t* pre = reinterpret_cast<int64_t*>(wt + 2 * RU);           // [batch + 1]
    __shared__ int64_t warp_sum[4];
    __shared__ int last_flag;

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int g = lane >> 2, t = lane & 3;
    const KVLayer& c = a.c;

    // ---- the line: prefix sums of the sequences' tiles
    {
        int64_t base = 0;
        for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
            const int b = b0 + tid;
            int64_t u = 0;
            if (b < a.batch) {
                const Seq s = sequence(a, b);
                const int64_t blocks = (static_cast<int64_t>(s.n) * a.group + RU - 1) / RU;
                u = blocks * c.heads * max(1, (s.len + kTile - 1) / kTile);
            }
            int64_t x = u;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int64_t y = __shfl_up_sync(~0u, x, o);
                if (lane >= o) x += y;
            }
            if (lane == 31) warp_sum[warp] = x;
            __syncthreads();
            for (int w = 0; w < warp; ++w) x += warp_sum[w];
            if (b < a.batch) pre[b + 1] = base + x;
            base += warp_sum[0] + warp_sum[1] + warp_sum[2] + warp_sum[3];
            __syncthreads();
        }
        if (tid == 0) pre[0] = 0;
        __syncthreads();
    }
    const Line line(pre[a.batch], grid);
    const int cta = blockIdx.x;
    if (cta >= line.ctas) return;
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
        const Seq sq = sequence(a, b);
        const int tiles = max(1, (sq.len + kTile - 1) / kTile);
        const int blocks = static_cast<int>((static_cast<int64_t>(sq.n) * a.group + RU - 1) / RU);
        const int64_t in = u - pre[b];
        const int hb = static_cast<int>(div64(in, tiles));
        const int tile0 = static_cast<int>(in - static_cast<int64_t>(hb) * tiles);
        const int h = hb / blocks, rb = hb - h * blocks;
        const int64_t span0 = u - tile0;
        const int seg = static_cast<int>(min(static_cast<int64_t>(tiles - tile0), u_end - u));
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
        // Lane i holds the page and scales of the i-th 16-token subtile.
        constexpr int step_tok = 64 * NS;
        const int warp_tok = tok0 + warp * 16 * NS;
        const int steps = tok1 > warp_tok ? (tok1 - warp_tok + step_tok - 1) / step_tok : 0;
        const int32_t* row_table = a.table + static_cast<int64_t>(b) * a.width;
        int id_c = -1;
        float ks_c = 0.f, vs_c = 0.f;
        auto refill = [&](int batch32) {
            const int sub = batch32 * 32 + lane;
            const int tok = warp_tok + (sub / NS) * step_tok + (sub % NS) * 16;
            id_c = -1;
            ks_c = vs_c = 0.f;
            if (tok < tok1) {
                const int id = row_table[tok >> c.log2p];
                if (id >= 0 && id < c.pages) {
                    id_c = id;
                    const int64_t at = static_cast<int64_t>(id) * c.heads + h;
                    ks_c = __ldg(c.ks + at);
                    vs_c = __ldg(c.vs + at);
                } else {
                    atomicOr(a.status, kStatusBounds);
                }
            }
        };
        uint4 kr[NS][2][DC];
        uint32_t vr[NS][4][VL][VW];
        int nid[NS];
        float nks[NS], nvs[NS];
        bool nfull = false;
        // lanes past the head's dims read its last ones: their q is 0, their columns of o are not written
        const int klane = g * c.token_stride, vlane = 2 * t * c.token_stride;
        const uint8_t* kbase = c.k + static_cast<int64_t>(h) * c.head_stride;
        const uint8_t* vbase = c.v + static_cast<int64_t>(h) * c.head_stride;
        const int pmask = (1 << c.log2p) - 1;
        auto locate = [&](int it) {  // pages and scales of step `it`
            if (it > 0 && (it * NS & 31) == 0) refill(it * NS >> 5);
            const int tok = warp_tok + it * step_tok;
            nfull = tok + 16 * NS <= full_end;
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int sub = it * NS + s;
                nid[s] = __shfl_sync(~0u, id_c, sub & 31);
                nks[s] = __shfl_sync(~0u, ks_c, sub & 31);
                nvs[s] = __shfl_sync(~0u, vs_c, sub & 31);
                nfull &= nid[s] >= 0;
            }
        };
        auto load_k_as = [&](int it, auto all) {
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int tok = warp_tok + it * step_tok + s * 16;
                const uint8_t* p = kbase + nid[s] * c.page_stride + ((tok & pmask) * c.token_stride + klane);
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const uint8_t* pj = p + j * 8 * c.token_stride;
                    const bool there = all || (nid[s] >= 0 && tok + j * 8 + g < tok1);
#pragma unroll
                    for (int cc = 0; cc < DC; ++cc) {
                        if (!all) kr[s][j][cc] = make_uint4(0, 0, 0, 0);
                        if (there) kr[s][j][cc] = ldg_stream16(pj + min(cc * 64 + t * 16, c.dim - 16));
                    }
                }
            }
        };
        auto load_k = [&](int it) {
            if (nfull) load_k_as(it, std::true_type());
            else load_k_as(it, std::false_type());
        };
        auto load_v_as = [&](int it, auto all) {
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int tok = warp_tok + it * step_tok + s * 16;
                const uint8_t* p = vbase + nid[s] * c.page_stride + ((tok & pmask) * c.token_stride + vlane);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int row = (j & 1) + 8 * (j >> 1);
                    const uint8_t* pj = p + row * c.token_stride;
                    const bool there = all || (nid[s] >= 0 && tok + row + 2 * t < tok1);
#pragma unroll
                    for (int x = 0; x < VL; ++x) {
                        if (!all)
#pragma unroll
                            for (int i = 0; i < VW; ++i) vr[s][j][x][i] = 0;
                        if (there) {
                            const uint8_t* at = pj + min(x * 128 + g * (4 * VW), c.dim - 4 * VW);
                            if (VW == 2) {
                                const uint2 v = ldg_stream8(at);
                                vr[s][j][x][0] = v.x, vr[s][j][x][1] = v.y;
                            } else {
                                const uint4 v = ldg_stream16(at);
                                vr[s][j][x][0] = v.x, vr[s][j][x][1] = v.y;
                                vr[s][j][x][VW - 2] = v.z, vr[s][j][x][VW - 1] = v.w;
                            }
                        }
                    }
                }
            }
        };
        auto load_v = [&](int it) {
            if (nfull) load_v_as(it, std::true_type());
            else load_v_as(it, std::false_type());
        };
        if (steps > 0) {  // on their way while the queries are prepared
            refill(0);
            locate(0);
            load_k(0);
            load_v(0);
        }

        // ---- queries: the column operand, scaled by a power of two per row.
        // A lane prepares row g of each tile of 8; the scores it gets are
        // those of rows 2t and 2t + 1, so their factors come from the lanes
        // that prepared these.
        float qfac[MT][2], init[MT][2];
        int limit[MT][2];  // tokens that the rows see
        __syncthreads();  // the previous segment's users of qf and wo are done
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int r = row_first + mt * 8 + g;
            const bool live = r < nrows;
            const int i_row = r / a.group;
            const int64_t qat = live ? (sq.row0 + i_row) * a.q_row + (h * a.group + r - i_row * a.group) * a.q_head : 0;
            // read twice (the second time from L1): the first codes of K and V hold the registers
            auto get = [&](int cc, float(&x)[16]) {
                const int d0 = cc * 64 + t * 16;
                if (live && d0 < c.dim) {
                    load_q16(a.q, a.type, qat + d0, x);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[i] = 0.f;
                }
            };
            float amax = 0.f;
#pragma unroll 1
            for (int cc = 0; cc < DC; ++cc) {
                float x[16];
                get(cc, x);
#pragma unroll
                for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[i]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
            // 2^e with amax * 2^e in [2^14, 2^15); 1 for zero or non-finite rows
            int e = 141 - static_cast<int>((__float_as_uint(amax) >> 23) & 255u);
            e = amax > 0.f && amax <= 3.4028235e38f ? min(e, 120) : 0;
            const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
            const float fac = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23) *
                              (INT8 ? 16777216.f : 1.f);
            f2 sum = {0.f, 0.f}, sum_lo = {0.f, 0.f};
#pragma unroll 1
            for (int cc = 0; cc < DC; ++cc) {
                float x[16];
                get(cc, x);
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    // the dims in the order that k_codes gives a word's bytes
                    const float x0 = x[4 * w] * up, x1 = x[4 * w + (INT8 ? 2 : 1)] * up;
                    const float x2 = x[4 * w + (INT8 ? 1 : 2)] * up, x3 = x[4 * w + 3] * up;
                    uint2 f, fl;
                    f.x = pack_f16x2(x0, x1);
                    f.y = pack_f16x2(x2, x3);
                    if (PARTS == 2) {
                        fl.x = rest_f16x2(x0, x1, f.x);
                        fl.y = rest_f16x2(x2, x3, f.y);
                    }
                    if (INT8) {
                        fadd2(sum, h2_to_f2(f.x));
                        fadd2(sum, h2_to_f2(f.y));
                        if (PARTS == 2) {
                            fadd2(sum_lo, h2_to_f2(fl.x));
                            fadd2(sum_lo, h2_to_f2(fl.y));
                        }
                    }
                    // every warp holds the same rows: each writes a quarter of the steps
                    if (w == warp) {
                        qf[(mt * 4 * DC + cc * 4 + w) * 32 + lane] = f;
                        if (PARTS == 2) qf[((MT + mt) * 4 * DC + cc * 4 + w) * 32 + lane] = fl;
                    }
                }
            }
            float bias = (sum.x + sum.y) + (sum_lo.x + sum_lo.y);
            bias += __shfl_xor_sync(~0u, bias, 1);
            bias += __shfl_xor_sync(~0u, bias, 2);
            bias *= kCodeBias;
            const int lim = live ? sq.len - sq.n + i_row + 1 : 0;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const int src = (2 * t + i) * 4;
                qfac[mt][i] = __shfl_sync(~0u, fac, src);
                init[mt][i] = __shfl_sync(~0u, bias, src);
                limit[mt][i] = __shfl_sync(~0u, lim, src);
            }
        }
        __syncthreads();

        float o[MT][4 * DC][4];
        int m[MT][2], mu[MT][2];    // references: m of the scores, mu of score + log2 vs
        float ref[MT][2], pk[MT][2], l[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                m[mt][i] = mu[mt][i] = kNone;
                ref[mt][i] = static_cast<float>(kNone);
                pk[mt][i] = 1.f;
                l[mt][i] = 0.f;
            }
#pragma unroll
            for (int j = 0; j < 4 * DC; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[mt][j][i] = 0.f;
        }

        // One step; `full`: every row sees every token of it.
        auto step = [&](int it, auto full) {
            const int tok = warp_tok + it * step_tok;
            float ks[NS], vs[NS];
            bool there[NS];
#pragma unroll
            for (int s = 0; s < NS; ++s) ks[s] = nks[s], vs[s] = nvs[s], there[s] = nid[s] >= 0;
            // scores: rows are tokens g and g + 8 of a subtile, columns the query rows 2t and 2t + 1
            float sc[MT][NS][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[mt][s][i] = INT8 ? init[mt][i & 1] : 0.f;
#pragma unroll
            for (int cc = 0; cc < DC; ++cc) {
                if (DC == 4 && cc * 64 >= c.dim) break;  // the other DC hold more than 64 (DC - 1) dims
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t ka[NS][4];
#pragma unroll
                    for (int s = 0; s < NS; ++s)
#pragma unroll
                        for (int j = 0; j < 2; ++j) {
                            const uint4& k4 = kr[s][j][cc];
                            k_codes<INT8>(w == 0 ? k4.x : w == 1 ? k4.y : w == 2 ? k4.z : k4.w, ka[s][j], ka[s][j + 2]);
                        }
#pragma unroll
                    for (int p = 0; p < PARTS; ++p)
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) {
                            const uint2 f = qf[((p * MT + mt) * 4 * DC + cc * 4 + w) * 32 + lane];
#pragma unroll
                            for (int s = 0; s < NS; ++s)
                                mma16816(sc[mt][s], ka[s][0], ka[s][1], ka[s][2], ka[s][3], f.x, f.y);
                        }
                }
            }
            const bool more = it + 1 < steps;
            if (more) {
                locate(it + 1);
                load_k(it + 1);
            }
            // vs < 2^evs, the same in all lanes
            int evs[NS];
#pragma unroll
            for (int s = 0; s < NS; ++s)
                evs[s] = vs[s] > 0.f ? static_cast<int>((__float_as_uint(vs[s]) >> 23) & 255u) - 126 : kNone;
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
            uint32_t pb[PARTS][MT][NS][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float y[NS][4];
                auto relative = [&]() {  // scores less their reference
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        const float f0 = qfac[mt][0] * ks[s], f1 = qfac[mt][1] * ks[s];
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            y[s][i] = fmaf(sc[mt][s][i], i & 1 ? f1 : f0, -ref[mt][i & 1]);
                            if (!full && __float_as_int(sc[mt][s][i]) == kMasked) y[s][i] = -INFINITY;
                        }
                    }
                };
                relative();
                bool passed = false;
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int s = 0; s < NS; ++s) {
                        const float top = fmaxf(y[s][i], y[s][i + 2]);
                        passed |= top > fminf(2.f, static_cast<float>(2 - (evs[s] + m[mt][i] - mu[mt][i])));
                    }
                if (__any_sync(~0u, passed)) {
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        int mn = m[mt][i], un = mu[mt][i];
#pragma unroll
                        for (int s = 0; s < NS; ++s) {
                            const float f = qfac[mt][i] * ks[s];
                            float top = -INFINITY;
#pragma unroll
                            for (int j = i; j < 4; j += 2)
                                if (full || __float_as_int(sc[mt][s][j]) != kMasked) top = fmaxf(top, sc[mt][s][j] * f);
#pragma unroll
                            for (int x = 4; x < 32; x <<= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, x));
                            const int up = ceil_ref(top);
                            mn = max(mn, up);
                            un = max(un, up + evs[s]);
                        }
                        const int k_old = min(12 + m[mt][i] - mu[mt][i], 126), k_new = min(12 + mn - un, 126);
                        const float os = pow2i((k_new - mn) - (k_old - m[mt][i]));
                        l[mt][i] *= pow2i(m[mt][i] - mn);
#pragma unroll
                        for (int j = 0; j < 4 * DC; ++j) {
                            o[mt][j][i] *= os;
                            o[mt][j][i + 2] *= os;
                        }
                        m[mt][i] = mn;
                        mu[mt][i] = un;
                        ref[mt][i] = static_cast<float>(mn);
                        pk[mt][i] = pow2i(max(k_new, -126));
                    }
                    relative();
                }
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const float f0 = vs[s] * pk[mt][0], f1 = vs[s] * pk[mt][1];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float p = exp2_fast(y[s][i]);
                        l[mt][i & 1] += p;
                        y[s][i] = p * (i & 1 ? f1 : f0);
                    }
#pragma unroll
                    for (int j = 0; j < 2; ++j) {
                        const uint32_t hi2 = pack_f16x2(y[s][2 * j], y[s][2 * j + 1]);
                        pb[0][mt][s][j] = transpose8x8(hi2);
                        if (PARTS == 2)
                            pb[PARTS - 1][mt][s][j] = transpose8x8(rest_f16x2(y[s][2 * j], y[s][2 * j + 1], hi2));
                    }
                }
            }
            if (!INT8 && !full && sq.n > 1) {
                // A code of V that is NaN where not every row sees every token:
                // taken out of the products and set where a row sees it.
                uint32_t any = 0;
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
#pragma unroll
                        for (int x = 0; x < VL; ++x)
#pragma unroll
                            for (int i = 0; i < VW; ++i)
                                any |= __vcmpeq4(vr[s][j][x][i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                if (__any_sync(~0u, any != 0)) {
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const int r = row_first + mt * 8 + g;
                        const int lim = r < nrows ? sq.len - sq.n + r / a.group + 1 : 0;
#pragma unroll
                        for (int s = 0; s < NS; ++s) {
                            const int first = tok + s * 16 + 2 * t;
                            const uint32_t sees0 = (first < lim ? 0x3C00u : 0u) | (first + 1 < lim ? 0x3C000000u : 0u);
                            const uint32_t sees1 = (first + 8 < lim ? 0x3C00u : 0u) | (first + 9 < lim ? 0x3C000000u : 0u);
#pragma unroll
                            for (int x = 0; x < VL; ++x)
#pragma unroll
                                for (int w = 0; w < VW; ++w) {
                                    uint32_t is[4], c01[4], c23[4];
#pragma unroll
                                    for (int j = 0; j < 4; ++j)  // e4m3 1.0 where the code is NaN
                                        is[j] = __vcmpeq4(vr[s][j][x][w] & 0x7F7F7F7Fu, 0x7F7F7F7Fu) & 0x38383838u;
                                    v_codes<false>(is[0], is[1], c01);
                                    v_codes<false>(is[2], is[3], c23);
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
#pragma unroll
                    for (int s = 0; s < NS; ++s)
#pragma unroll
                        for (int j = 0; j < 4; ++j)
#pragma unroll
                            for (int x = 0; x < VL; ++x)
#pragma unroll
                                for (int i = 0; i < VW; ++i)
                                    vr[s][j][x][i] &= ~__vcmpeq4(vr[s][j][x][i] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                }
            }
            // o += V^T p^T.  Row tile 2w + i: dims with bytes 4w + 2i (rows 0-7) and 4w + 2i + 1 (rows 8-15)
#pragma unroll
            for (int x = 0; x < VL; ++x)
#pragma unroll
                for (int s = 0; s < NS; ++s)
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        uint32_t c01[4], c23[4];
                        v_codes<INT8>(vr[s][0][x][w], vr[s][1][x][w], c01);
                        v_codes<INT8>(vr[s][2][x][w], vr[s][3][x][w], c23);
#pragma unroll
                        for (int i = 0; i < 2; ++i)
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                                for (int p = 0; p < PARTS; ++p)
                                    mma16816(o[mt][x * 2 * VW + 2 * w + i], c01[2 * i], c01[2 * i + 1], c23[2 * i],
                                             c23[2 * i + 1], pb[p][mt][s][0], pb[p][mt][s][1]);
                    }
            if (more) load_v(it + 1);
        };
        int it = 0;
        for (; it < steps && nfull; ++it) step(it, std::true_type());
        for (; it < steps; ++it) step(it, std::false_type());

        // ---- this warp's normalised result and log-sum
#pragma unroll
        for (int mt = 0; mt < MT; ++mt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float sum = l[mt][i];
#pragma unroll
                for (int x = 4; x < 32; x <<= 1) sum += __shfl_xor_sync(~0u, sum, x);
                // NaN sums stay NaN; a row that saw nothing has a sum of 0
                const bool none = sum == 0.f && m[mt][i] == kNone;
                const int down = none ? 0 : max(-min(12 + m[mt][i] - mu[mt][i], 126), -252);
                const float f1 = pow2i(down >> 1), f2v = pow2i(down - (down >> 1));
                const float inv = none ? 0.f : 1.f / sum;
                const int r = mt * 8 + 2 * t + i;
                if (g == 0) ws[warp * RU + r] = none ? -INFINITY : static_cast<float>(m[mt][i]) + log2f(sum);
                float* dst = wo + (warp * RU + r) * DP + g * (4 * VW);
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
        // ---- join the four warps; then either the output or a partial result
        const bool whole = seg == tiles;
        const int slot = u == u_begin ? 0 : 1;
        float* part = a.part + static_cast<int64_t>(cta * 2 + slot) * kPartFloats;
        for (int r = warp; r < RU; r += 4) {
            const float s0 = ws[r], s1 = ws[RU + r], s2 = ws[2 * RU + r], s3 = ws[3 * RU + r];
            const float mx = fmaxf(fmaxf(s0, s1), fmaxf(s2, s3));
            const float ref = mx == -INFINITY ? 0.f : mx;
            const float w0 = exp2f(s0 - ref), w1 = exp2f(s1 - ref), w2 = exp2f(s2 - ref), w3 = exp2f(s3 - ref);
            const float sum = w0 + w1 + w2 + w3;
            const float inv = sum == 0.f ? 0.f : 1.f / sum;
            const float ls = sum == 0.f ? -INFINITY : ref + log2f(sum);
            const int rr = row_first + r;
            const int64_t orow = (sq.row0 + rr / a.group) * a.q_heads + h * a.group + rr % a.group;
            for (int d = lane; d < c.dim; d += 32) {
                const float* p = wo + r * DP + d;
                // a warp without tokens contributes nothing, not 0 * its contents
                float acc = 0.f;
                if (s0 != -INFINITY) acc += w0 * p[0];
                if (s1 != -INFINITY) acc += w1 * p[RU * DP];
                if (s2 != -INFINITY) acc += w2 * p[2 * RU * DP];
                if (s3 != -INFINITY) acc += w3 * p[3 * RU * DP];
                acc *= inv;
                if (!whole) part[r * c.dim + d] = acc;
                else if (rr < nrows) store_out(a.out, a.type, orow * c.dim + d, acc);
            }
            if (lane == 0) {
                if (!whole) part[2048 + r] = ls;
                else if (rr < nrows && a.lse) a.lse[orow] = ls * 0.69314718055994531f;
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
                // the CTAs' partials in the order of the line
                auto slot_of = [&](int cc) {
                    return a.part + static_cast<int64_t>(cc * 2 + (line.first(cc) >= span0 ? 0 : 1)) * kPartFloats;
                };
                for (int r = warp; r < RU; r += 4) {
                    const int rr = row_first + r;
                    if (rr >= nrows) break;
                    float mx = -INFINITY;
                    for (int i = lane; i < need; i += 32) mx = fmaxf(mx, __ldcg(slot_of(first + i) + 2048 + r));
#pragma unroll
                    for (int x = 16; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, x));
                    const float ref = mx == -INFINITY ? 0.f : mx;
                    float acc[2 * DC];
#pragma unroll
                    for (int x = 0; x < 2 * DC; ++x) acc[x] = 0.f;
                    float sum = 0.f;
#pragma unroll 4
                    for (int i = 0; i < need; ++i) {
                        const float* p = slot_of(first + i);
                        const float ls = __ldcg(p + 2048 + r);
                        const float w = exp2f(ls - ref);
                        sum += w;
                        if (ls == -INFINITY) continue;
#pragma unroll
                        for (int x = 0; x < 2 * DC; ++x)
                            if (x * 32 + lane < c.dim) acc[x] += w * __ldcg(p + r * c.dim + x * 32 + lane);
                    }
                    const float inv = sum == 0.f ? 0.f : 1.f / sum;
                    const int64_t orow = (sq.row0 + rr / a.group) * a.q_heads + h * a.group + rr % a.group;
#pragma unroll
                    for (int x = 0; x < 2 * DC; ++x)
                        if (x * 32 + lane < c.dim)
                            store_out(a.out, a.type, orow * c.dim + x * 32 + lane, acc[x] * inv);
                    if (lane == 0 && a.lse)
                        a.lse[orow] = sum == 0.f ? -INFINITY : (ref + log2f(sum)) * 0.69314718055994531f;
                }
            }
        }
        u += seg;
    }
}

template <int DC, int MT, int PARTS, bool INT8, int MINB>
int launch_one(const AttnArgs& a, cudaStream_t s) {
    const int dev = current_device();
    const int sms = sm_count(dev);
    if (sms <= 0) return cuda_fail(cudaGetLastError());
    constexpr int RU = 8 * MT, DP = 64 * DC;
    const int fixed = PARTS * MT * 4 * DC * 32 * 8 + 4 * RU * DP * 4 + 6 * RU * 4;
    const int most = fixed + (QGKV_MAX_BATCH + 1) * 8;
    static std::atomic<bool> done[64];
    auto kern = qg_attn_rows_kernel<DC, MT, PARTS, INT8, MINB>;
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
            return cuda_fail(cudaGetLastError());
        done[dev].store(true, std::memory_order_release);
    }
    const int grid = sms * MINB < kMaxCtas ? sms * MINB : kMaxCtas;
    kern<<<grid, kThreads, fixed + (a.batch + 1) * 8, s>>>(a, grid);
    return launch_status();
}

template <int PARTS, bool INT8>
int launch_typed(const AttnArgs& a, cudaStream_t s) {
    // 16 rows a unit where the mean sequence has more than 8 (the codes are
    // then read half as often); 256-dim heads keep 8 for their registers
    const bool wide = a.rows * a.group > 8 * static_cast<int64_t>(a.batch);
    if (a.c.dim <= 64) return wide ? launch_one<1, 2, PARTS, INT8, 4>(a, s) : launch_one<1, 1, PARTS, INT8, 3>(a, s);
    if (a.c.dim <= 128) return wide ? launch_one<2, 2, PARTS, INT8, 2>(a, s) : launch_one<2, 1, PARTS, INT8, 2>(a, s);
    return launch_one<4, 1, PARTS, INT8, 2>(a, s);
}

}  // namespace

int launch_attn_rows(const AttnArgs& a, bool int8, cudaStream_t s) {
    if (a.type == QGKV_F32) return int8 ? launch_typed<2, true>(a, s) : launch_typed<2, false>(a, s);
    return int8 ? launch_typed<1, true>(a, s) : launch_typed<1, false>(a, s);
}

}  // namespace qg
