// Attention of few query rows over the 8-bit paged cache (decode, short
// chunks): one pass over K and V with the running maximum and sum of the
// softmax.
//
// Mathematics.  For a row r of queries and the tokens t of its sequence
//   s[t] = (scale * log2 e * ks[page]) * (q . kcode[t]),  p[t] = 2^(s[t] - m)
//   l = sum p[t],   o = sum p[t] * vs[page] * vcode[t],   out = o / l
// with m at or above the running maximum.  Codes are exact in f16.  q * 2^j (a
// power of two that brings the row's largest value to [2^14, 2^15)) and
// p * vs * 2^(14 + m - u) enter the products as two f16 parts, hi and lo,
// about 22 bits: the 16 rows of the tensor instruction are 8 query rows
// twice, hi in rows 0-7 and lo in rows 8-15, and the two halves of the sums
// are added in fp32.  With the group sizes of grouped-query heads (8 and
// below) the lo parts take rows that would stay empty.  u bounds s + log2 vs
// over the tokens seen, so that what reaches o is at most 2^14 and its
// largest part near that, however the scales of the blocks differ; m and u
// are integers, which makes every rescaling a power of two.
//
// Bound.  Decode reads every code once for 4 * group flops a byte: HBM-bound
// on the stream of codes.  The fragments are laid out so that codes go from
// global memory to registers and into the tensor instruction without shared
// memory: the order of a head's dims is free in q . k (q is permuted the same
// way) and in the columns of o, the order of tokens is free in the sum, so a
// lane takes 16 dims of one token for K and 8 or 16 dims of four tokens for
// V, each a whole vector load, each quad or octet a whole row segment.  The
// loads of the next tile are issued as soon as the registers of the current
// one are consumed.
//
// Split.  The tokens of all (sequence, head, row block) are one line of
// 128-token tiles, cut evenly among the CTAs whatever the lengths; a CTA that
// holds a whole (sequence, head) writes its result, the others leave
// normalised partial results in the workspace and the last to arrive at a
// counter joins them in the order of the line (bits do not depend on the
// order of arrival).
#include <atomic>

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

constexpr int kNone = -(1 << 29);  // reference of a row that has seen nothing

// 2^k exactly; 0 below the normal range.
__device__ __forceinline__ float pow2i(int k) {
    return __uint_as_float(static_cast<uint32_t>(min(max(k, -127), 127) + 127) << 23);
}
// x * 2^k, -252 <= k <= 252, in two exact steps.
__device__ __forceinline__ float times_pow2(float x, int k) {
    k = max(k, -252);
    return x * pow2i(k >> 1) * pow2i(k - (k >> 1));
}
// The least integer >= x as a reference; kNone for -inf.
__device__ __forceinline__ int ceil_ref(float x) {
    return x == -INFINITY ? kNone : static_cast<int>(ceilf(fminf(fmaxf(x, -1.0e8f), 1.0e8f)));
}

template <int DC, int MT, bool INT8, int MINB>
__global__ void __launch_bounds__(kThreads, MINB) qg_attn_rows_kernel(const AttnArgs a, int grid) {
    constexpr int NS = DC <= 2 ? 2 : 1;    // 16-token subtiles of one warp step
    constexpr int RU = 8 * MT;             // query rows of a unit
    constexpr int VW = DC == 1 ? 2 : 4;    // 32-bit words of one V load
    constexpr int VL = DC == 4 ? 2 : 1;    // V loads per token row
    constexpr int DP = 64 * DC;
    extern __shared__ __align__(16) unsigned char smem[];
    uint4* qf = reinterpret_cast<uint4*>(smem);                       // [MT][4 * DC][32]
    float* wo = reinterpret_cast<float*>(qf + MT * 4 * DC * 32);      // [4][RU][DP]
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
    const int64_t total = pre[a.batch];
    const int64_t G = total < grid ? total : grid;
    const int64_t cta = blockIdx.x;
    if (cta >= G) return;
    const int64_t u_begin = total * cta / G, u_end = total * (cta + 1) / G;

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
        const int tile0 = static_cast<int>(in % tiles);
        const int hb = static_cast<int>(in / tiles);
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

        // ---- queries: fragments of hi and lo parts, scaled by a power of two per row
        float qfac[MT];
        __syncthreads();  // the previous segment's users of qf and wo are done
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int r = row_first + mt * 8 + g;
            const bool live = r < nrows;
            const int64_t qat = live ? (sq.row0 + r / a.group) * a.q_row + (h * a.group + r % a.group) * a.q_head : 0;
            float amax = 0.f;
            float x[DC][16];
#pragma unroll
            for (int cc = 0; cc < DC; ++cc) {
                const int d0 = cc * 64 + t * 16;
                if (live && d0 < c.dim) {
                    load_q16(a.q, a.type, qat + d0, x[cc]);
                } else {
#pragma unroll
                    for (int i = 0; i < 16; ++i) x[cc][i] = 0.f;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) amax = fmaxf(amax, fabsf(x[cc][i]));
            }
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 1));
            amax = fmaxf(amax, __shfl_xor_sync(~0u, amax, 2));
            // 2^e with amax * 2^e in [2^14, 2^15); 1 for zero or non-finite rows
            int e = 141 - static_cast<int>((__float_as_uint(amax) >> 23) & 255u);
            e = amax > 0.f && amax <= 3.4028235e38f ? min(e, 120) : 0;
            const float up = __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
            qfac[mt] = a.scale_log2 * __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
            // every warp holds the same rows: each writes a quarter of the steps
#pragma unroll
            for (int cc = 0; cc < DC; ++cc)
#pragma unroll
                for (int w = 0; w < 4; ++w)
                    if (w == warp) {
                        uint4 f;
                        f.x = pack_f16x2(x[cc][4 * w] * up, x[cc][4 * w + 1] * up);
                        f.z = pack_f16x2(x[cc][4 * w + 2] * up, x[cc][4 * w + 3] * up);
                        f.y = rest_f16x2(x[cc][4 * w] * up, x[cc][4 * w + 1] * up, f.x);
                        f.w = rest_f16x2(x[cc][4 * w + 2] * up, x[cc][4 * w + 3] * up, f.z);
                        qf[(mt * 4 * DC + cc * 4 + w) * 32 + lane] = f;
                    }
        }
        __syncthreads();
        int limit[MT];  // tokens that this lane's row sees
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            const int r = row_first + mt * 8 + g;
            limit[mt] = r < nrows ? sq.len - sq.n + r / a.group + 1 : 0;
        }

        float o[MT][8 * DC][4];
        int m[MT], mu[MT];  // references of l and of o, powers of two
        float l[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            m[mt] = mu[mt] = kNone;
            l[mt] = 0.f;
#pragma unroll
            for (int j = 0; j < 8 * DC; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) o[mt][j][i] = 0.f;
        }

        // ---- the stream of this warp: steps of 16 * NS tokens, 4 * 16 * NS apart
        const int step_tok = 64 * NS;
        const int warp_tok = tok0 + warp * 16 * NS;
        const int32_t* row_table = a.table + static_cast<int64_t>(b) * a.width;
        int id_c = -1;         // page of subtile (batch of 32) + lane
        float ks_c = 0.f, vs_c = 0.f;
        int have = -1;         // which batch of 32 subtiles the lanes hold
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
            have = batch32;
        };

        uint4 kr[NS][2][DC];
        uint32_t vr[NS][4][VL][VW];
        int nid[NS];
        float nks[NS], nvs[NS];
        auto locate = [&](int it) {  // pages and scales of step `it`
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int sub = it * NS + s;
                if ((sub >> 5) != have) refill(sub >> 5);
                nid[s] = __shfl_sync(~0u, id_c, sub & 31);
                nks[s] = __shfl_sync(~0u, ks_c, sub & 31);
                nvs[s] = __shfl_sync(~0u, vs_c, sub & 31);
            }
        };
        const uint8_t* kbase = c.k + static_cast<int64_t>(h) * c.head_stride;
        const uint8_t* vbase = c.v + static_cast<int64_t>(h) * c.head_stride;
        const int pmask = (1 << c.log2p) - 1;
        auto load_k = [&](int it) {
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int tok = warp_tok + it * step_tok + s * 16;
                const uint8_t* p = kbase + nid[s] * c.page_stride + t * 16;
#pragma unroll
                for (int j = 0; j < 2; ++j) {
                    const int mine = tok + j * 8 + g;
#pragma unroll
                    for (int cc = 0; cc < DC; ++cc) {
                        kr[s][j][cc] = make_uint4(0, 0, 0, 0);
                        if (nid[s] >= 0 && mine < tok1 && cc * 64 + t * 16 < c.dim)
                            kr[s][j][cc] = ldg_stream16(p + (mine & pmask) * c.token_stride + cc * 64);
                    }
                }
            }
        };
        auto load_v = [&](int it) {
#pragma unroll
            for (int s = 0; s < NS; ++s) {
                const int tok = warp_tok + it * step_tok + s * 16;
                const uint8_t* p = vbase + nid[s] * c.page_stride + g * (4 * VW);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const int mine = tok + (j & 1) + 2 * t + 8 * (j >> 1);
#pragma unroll
                    for (int x = 0; x < VL; ++x) {
#pragma unroll
                        for (int i = 0; i < VW; ++i) vr[s][j][x][i] = 0;
                        if (nid[s] >= 0 && mine < tok1 && x * 128 + g * (4 * VW) < c.dim) {
                            const uint8_t* at = p + (mine & pmask) * c.token_stride + x * 128;
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

        const int steps = tok1 > warp_tok ? (tok1 - warp_tok + step_tok - 1) / step_tok : 0;
        if (steps > 0) {
            locate(0);
            load_k(0);
            load_v(0);
        }
        for (int it = 0; it < steps; ++it) {
            const int tok = warp_tok + it * step_tok;
            float ks[NS], vs[NS];
            bool there[NS];
#pragma unroll
            for (int s = 0; s < NS; ++s) ks[s] = nks[s], vs[s] = nvs[s], there[s] = nid[s] >= 0;
            // scores: S[mt][token tile] = (hi; lo) rows of q . k
            float sc[MT][2 * NS][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int j = 0; j < 2 * NS; ++j)
#pragma unroll
                    for (int i = 0; i < 4; ++i) sc[mt][j][i] = 0.f;
#pragma unroll
            for (int cc = 0; cc < DC; ++cc) {
                if (cc * 64 >= c.dim) break;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    uint32_t b0[2 * NS], b1[2 * NS];
#pragma unroll
                    for (int j = 0; j < 2 * NS; ++j) {
                        const uint4& k4 = kr[j >> 1][j & 1][cc];
                        codes4_f16<INT8>(w == 0 ? k4.x : w == 1 ? k4.y : w == 2 ? k4.z : k4.w, b0[j], b1[j]);
                    }
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) {
                        const uint4 f = qf[(mt * 4 * DC + cc * 4 + w) * 32 + lane];
#pragma unroll
                        for (int j = 0; j < 2 * NS; ++j) mma16816(sc[mt][j], f.x, f.y, f.z, f.w, b0[j], b1[j]);
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
            const bool full = tok + 16 * NS <= seen_least && there[0] && there[NS - 1];
            bool odd_v = false;  // a code of V that is NaN where not every row sees every token
            if (!full && !INT8 && sq.n > 1) {
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
                odd_v = __any_sync(~0u, any != 0);
            }
            uint32_t pa[MT][NS][4];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float x[2 * NS][2];
                int mn = m[mt], un = mu[mt];
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    float mx = -INFINITY;
#pragma unroll
                    for (int j = 2 * s; j < 2 * s + 2; ++j)
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            float y = (sc[mt][j][i] + sc[mt][j][i + 2]) * (qfac[mt] * ks[s]);
                            if (!full) {
                                const int mine = tok + j * 8 + 2 * t + i;
                                if (mine >= limit[mt] || mine >= tok1 || !there[s]) y = -INFINITY;
                            }
                            x[j][i] = y;
                            mx = fmaxf(mx, y);
                        }
                    mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 1));
                    mx = fmaxf(mx, __shfl_xor_sync(~0u, mx, 2));
                    const int up = ceil_ref(mx);
                    mn = max(mn, up);
                    un = max(un, up + evs[s]);
                }
                l[mt] *= pow2i(m[mt] - mn);
                const float os = pow2i(mu[mt] - un);
                m[mt] = mn;
                mu[mt] = un;
                const float ref = static_cast<float>(mn);
#pragma unroll
                for (int s = 0; s < NS; ++s) {
                    const float f = times_pow2(vs[s], min(14 + mn - un, 126));
#pragma unroll
                    for (int j = 2 * s; j < 2 * s + 2; ++j) {
#pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            x[j][i] = exp2_fast(x[j][i] - ref);
                            l[mt] += x[j][i];
                            x[j][i] *= f;
                        }
                        const uint32_t hi2 = pack_f16x2(x[j][0], x[j][1]);
                        pa[mt][s][(j & 1) * 2] = hi2;
                        pa[mt][s][(j & 1) * 2 + 1] = rest_f16x2(x[j][0], x[j][1], hi2);
                    }
                }
                if (__any_sync(~0u, os != 1.f)) {
#pragma unroll
                    for (int j = 0; j < 8 * DC; ++j)
#pragma unroll
                        for (int i = 0; i < 4; ++i) o[mt][j][i] *= os;
                }
            }
            // o += p v.  Column tile 4w + i holds dims {lane group * width + 4w + i}
#pragma unroll
            for (int x = 0; x < VL; ++x) {
#pragma unroll
                for (int s = 0; s < NS; ++s) {
#pragma unroll
                    for (int w = 0; w < VW; ++w) {
                        uint32_t r0 = vr[s][0][x][w], r1 = vr[s][1][x][w], r2 = vr[s][2][x][w], r3 = vr[s][3][x][w];
                        if (odd_v) {  // NaN codes: kept out of the products, set where a row sees them
                            uint32_t n[4] = {r0, r1, r2, r3};
                            uint32_t is[4];
#pragma unroll
                            for (int j = 0; j < 4; ++j) {
                                is[j] = __vcmpeq4(n[j] & 0x7F7F7F7Fu, 0x7F7F7F7Fu);
                                n[j] &= ~is[j];
                                is[j] &= 0x38383838u;  // e4m3 1.0
                            }
                            r0 = n[0], r1 = n[1], r2 = n[2], r3 = n[3];
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                uint32_t sees[2];
#pragma unroll
                                for (int j = 0; j < 2; ++j) {
                                    const int mine = tok + s * 16 + j * 8 + 2 * t;
                                    sees[j] = (mine < limit[mt] ? 0x3C00u : 0u) |
                                              (mine + 1 < limit[mt] ? 0x3C000000u : 0u);
                                }
#pragma unroll
                                for (int i = 0; i < 4; ++i) {
                                    const uint32_t sel = i < 2 ? 0x5140u : 0x7362u;
                                    uint32_t p0 = prmt(is[0], is[1], sel), p1 = prmt(is[2], is[3], sel);
                                    if (i & 1) p0 >>= 16, p1 >>= 16;
                                    float cnt[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma16816(cnt, sees[0], 0u, sees[1], 0u, e4m3x2_f16x2(p0 & 0xFFFFu),
                                             e4m3x2_f16x2(p1 & 0xFFFFu));
                                    float(&d)[4] = o[mt][x * 16 + 4 * w + i];
                                    if (cnt[0] > 0.f) d[0] = __int_as_float(0x7FC00000);
                                    if (cnt[1] > 0.f) d[1] = __int_as_float(0x7FC00000);
                                }
                            }
                        }
#pragma unroll
                        for (int half = 0; half < 2; ++half) {
                            const uint32_t sel = half == 0 ? 0x5140u : 0x7362u;
                            uint32_t x0, x1, y0, y1;
                            codes4_f16<INT8>(prmt(r0, r1, sel), x0, x1);
                            codes4_f16<INT8>(prmt(r2, r3, sel), y0, y1);
#pragma unroll
                            for (int mt = 0; mt < MT; ++mt) {
                                const uint32_t(&p)[4] = pa[mt][s];
                                mma16816(o[mt][x * 16 + 4 * w + 2 * half], p[0], p[1], p[2], p[3], x0, y0);
                                mma16816(o[mt][x * 16 + 4 * w + 2 * half + 1], p[0], p[1], p[2], p[3], x1, y1);
                            }
                        }
                    }
                }
            }
            if (more) load_v(it + 1);
        }

        // ---- this warp's normalised result and log-sum
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            l[mt] += __shfl_xor_sync(~0u, l[mt], 1);
            l[mt] += __shfl_xor_sync(~0u, l[mt], 2);
            // NaN sums stay NaN; a row that saw nothing has l = 0
            const bool none = l[mt] == 0.f && m[mt] == kNone;
            const int down = min(max(mu[mt] - m[mt] - 14, -252), 252);
            const float f1 = pow2i(down >> 1), f2v = pow2i(down - (down >> 1));
            const float inv = none ? 0.f : 1.f / l[mt];
            if (t == 0) ws[warp * RU + mt * 8 + g] = none ? -INFINITY : static_cast<float>(m[mt]) + log2f(l[mt]);
            float* dst = wo + (warp * RU + mt * 8 + g) * DP;
#pragma unroll
            for (int j = 0; j < 8 * DC; ++j) {
                // column n of tile j is dim (n * 4 VW + j % (4 VW)) of its 32 VW-wide part
                const int part = j / (4 * VW), in_part = j % (4 * VW);
                const int d = part * (32 * VW) + 2 * t * (4 * VW) + in_part;
                dst[d] = (o[mt][j][0] + o[mt][j][2]) * inv * f1 * f2v;
                dst[d + 4 * VW] = (o[mt][j][1] + o[mt][j][3]) * inv * f1 * f2v;
            }
        }
        __syncthreads();
        // ---- join the four warps; then either the output or a partial result
        const bool whole = seg == tiles;
        const int slot = u == u_begin ? 0 : 1;
        float* part = a.part + (cta * 2 + slot) * kPartFloats;
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
            const int64_t first = ((span0 + 1) * G - 1) / total, lastc = ((span0 + tiles) * G - 1) / total;
            const int need = static_cast<int>(lastc - first + 1);
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
                auto slot_of = [&](int64_t cc) {
                    return a.part + (cc * 2 + (total * cc / G >= span0 ? 0 : 1)) * kPartFloats;
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

template <int DC, int MT, bool INT8, int MINB>
int launch_one(const AttnArgs& a, cudaStream_t s) {
    const int dev = current_device();
    const int sms = sm_count(dev);
    if (sms <= 0) return cuda_fail(cudaGetLastError());
    constexpr int RU = 8 * MT, DP = 64 * DC;
    const int fixed = MT * 4 * DC * 32 * 16 + 4 * RU * DP * 4 + 6 * RU * 4;
    const int most = fixed + (QGKV_MAX_BATCH + 1) * 8;
    static std::atomic<bool> done[64];
    auto kern = qg_attn_rows_kernel<DC, MT, INT8, MINB>;
    if (!done[dev].load(std::memory_order_acquire)) {
        if (cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, most) != cudaSuccess)
            return cuda_fail(cudaGetLastError());
        done[dev].store(true, std::memory_order_release);
    }
    const int grid = sms * MINB < kMaxCtas ? sms * MINB : kMaxCtas;
    kern<<<grid, kThreads, fixed + (a.batch + 1) * 8, s>>>(a, grid);
    return launch_status();
}

template <bool INT8>
int launch_typed(const AttnArgs& a, cudaStream_t s) {
    // 16 rows a unit where the mean sequence has more than 8 (the codes are
    // then read half as often); 256-dim heads keep 8 for their registers
    const bool wide = a.rows * a.group > 8 * static_cast<int64_t>(a.batch);
    if (a.c.dim <= 64) return wide ? launch_one<1, 2, INT8, 3>(a, s) : launch_one<1, 1, INT8, 4>(a, s);
    if (a.c.dim <= 128) return wide ? launch_one<2, 2, INT8, 2>(a, s) : launch_one<2, 1, INT8, 3>(a, s);
    return launch_one<4, 1, INT8, 2>(a, s);
}

}  // namespace

int launch_attn_rows(const AttnArgs& a, bool int8, cudaStream_t s) {
    return int8 ? launch_typed<true>(a, s) : launch_typed<false>(a, s);
}

}  // namespace qg
