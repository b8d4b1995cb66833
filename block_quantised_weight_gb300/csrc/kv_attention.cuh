// Arguments and launchers of the attention over the 8-bit paged cache.
#pragma once
#include "kv_common.cuh"

namespace qg {

struct AttnArgs {
    KVLayer c;
    const void* q;
    void* out;
    float* lse;
    int64_t q_row, q_head;  // elements
    int type, q_heads, group;
    const int32_t* table;
    int64_t width;
    const int32_t* lens;
    const int32_t* starts;
    int batch;
    int64_t rows;
    float scale_log2;  // softmax scale * log2(e)
    float* part;
    int4* splits;
    unsigned* count;
    unsigned* status;
    // A shared prefix: the plan's groups and tokens, and the prefix's results (kv_prefix.cuh)
    const int4* groups;
    const int32_t* skip;
    int ngroups;
    float* own;      // [rows][q_heads][dim], normalised, of a row's first piece
    float4* own_ml;  // [rows][q_heads] its reference and sum, the CTA of the next and their row, their number and its group
    float* slots;    // [CTA][slot_rows][slot_dims], then [slot_rows] references and sums, of further pieces
    int slot_rows, slot_dims;
};

// Number of rows and length of sequence b.  A length beyond the table is cut
// to it, rows outside the tensor are none (kStatusBounds).
struct Seq {
    int n, len;
};
__device__ __forceinline__ Seq sequence(const AttnArgs& a, int b) {
    Seq s = {1, a.lens[b]};
    if (a.starts) {
        const int64_t r0 = a.starts[b], r1 = a.starts[b + 1];
        s.n = static_cast<int>(r1 - r0);
        if (r0 < 0 || r1 < r0 || r1 > a.rows) {
            atomicOr(a.status, kStatusBounds);
            s.n = 0;
        }
    }
    const int64_t most = a.width << a.c.log2p;
    if (s.len < 0 || s.len > most) {
        atomicOr(a.status, kStatusBounds);
        s.len = s.len < 0 ? 0 : static_cast<int>(most);
    }
    return s;
}

// Entries of a plan that do not fit the call count as nothing shared (kStatusBounds).
// A group: n rows from row0 on, whose tokens a table row has.  Groups' rows rise: one that begins among those of
// the group before counts as nothing shared, so that two groups never write the results of one row.
struct SharedGroup {
    int row0, n, tokens, table_row;
};
__device__ __forceinline__ bool group_fits(const AttnArgs& a, int4 g) {  // first row, rows, tokens, first sequence
    return g.x >= 0 && g.y >= 0 && static_cast<int64_t>(g.x) + g.y <= a.rows && g.z >= 0 && g.z <= a.width << a.c.log2p &&
           (g.z & ((1 << a.c.log2p) - 1)) == 0 && (g.z == 0 || (g.w >= 0 && g.w < a.batch));
}
__device__ __forceinline__ int4 group_before(const AttnArgs& a, int b) { return b > 0 ? a.groups[b - 1] : make_int4(0, 0, 0, 0); }
__device__ __forceinline__ SharedGroup shared_group(const AttnArgs& a, int4 g, int4 before) {
    const bool good = group_fits(a, g) && (g.y == 0 || !group_fits(a, before) || g.x >= before.x + before.y);
    if (!good) atomicOr(a.status, kStatusBounds);
    return good && g.y > 0 && g.z > 0 ? SharedGroup{g.x, g.y, g.z, g.w} : SharedGroup{0, 0, 0, 0};
}
// Whole columns of its table that a sequence of n rows and len tokens (cut to the table) shares by a plan's entry
// `skip`, which its first row sees; -1 where the entry does not fit it.
__host__ __device__ constexpr int columns_shared(int skip, int n, int len, int log2p) {
    return skip == 0 || n == 0 ? 0 : skip < 0 || skip > len - n + 1 || (skip & ((1 << log2p) - 1)) ? -1 : skip >> log2p;
}
// What sequence b reads behind the tokens that it shares: less of its length, the columns of its table behind those
// returned.  An entry that does not fit is as none (kStatusBounds).
__device__ __forceinline__ int shared_columns(const AttnArgs& a, int b, Seq& s) {
    const int columns = columns_shared(a.skip[b], s.n, s.len, a.c.log2p);
    if (columns < 0) atomicOr(a.status, kStatusBounds);
    if (columns <= 0) return 0;
    s.len -= columns << a.c.log2p;
    return columns;
}

// a / b for non-negative a and positive b, in 32 bits where they fit.
__device__ __forceinline__ int64_t div64(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
    return a / b;
}

// A line of tiles (or steps) cut into pieces of equal size, the first `more` one longer.
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

// References of the running softmax.  m of a row is a whole number held as a
// float, so that it follows scores of any size, kNoRef before the row's first
// token; d, the reference of score + log2 vs, is held less m, at least kNoOrder (no
// value but zeros yet).
constexpr float kNoRef = -3.402823466e38f;
constexpr int kMostK = 124;  // of k: p * 2^k stays finite, p being 4 at most
constexpr int kNoOrder = -1000;
// From here on a score's rounding (2^-24 of it) is no small part of a binary
// order: the scores of a warp that has met one are rounded before the reference
// is taken off, so that equal scores get equal weights.
constexpr float kHugeScore = 0x1p22f;

// 2^k exactly; 0 below the normal range.
__device__ __forceinline__ float pow2i(int k) {
    return __uint_as_float(static_cast<uint32_t>(min(max(k, -127), 127) + 127) << 23);
}
// A difference of binary orders (at most a few hundred) as an integer; -inf is far below all.
__device__ __forceinline__ int order_of(float x) { return static_cast<int>(fmaxf(x, -4000.f)); }

// Four consecutive output values.
__device__ __forceinline__ void store_out4(void* out, int type, int64_t at, float4 x) {
    if (type == QGKV_F32) {
        *reinterpret_cast<float4*>(static_cast<float*>(out) + at) = x;
    } else if (type == QGKV_F16) {
        *reinterpret_cast<uint2*>(static_cast<__half*>(out) + at) = make_uint2(pack_f16x2(x.x, x.y), pack_f16x2(x.z, x.w));
    } else {
        uint32_t lo, hi;
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(lo) : "f"(x.y), "f"(x.x));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(hi) : "f"(x.w), "f"(x.z));
        *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(out) + at) = make_uint2(lo, hi);
    }
}

// Four consecutive query values as they lie (16-bit types in x and y); to
// values with q4_values once they are there, so that reads of several vectors
// do not wait for one another.
__device__ __forceinline__ uint4 load_q4(const void* q, int type, int64_t at, bool there) {
    uint4 r = make_uint4(0u, 0u, 0u, 0u);
    if (type == QGKV_F32) {
        if (there) r = __ldg(reinterpret_cast<const uint4*>(static_cast<const float*>(q) + at));
    } else if (there) {
        const uint2 v = __ldg(reinterpret_cast<const uint2*>(static_cast<const uint16_t*>(q) + at));
        r.x = v.x, r.y = v.y;
    }
    return r;
}
__device__ __forceinline__ float4 q4_values(uint4 v, int type) {
    if (type == QGKV_F32)
        return make_float4(__uint_as_float(v.x), __uint_as_float(v.y), __uint_as_float(v.z), __uint_as_float(v.w));
    if (type == QGKV_F16) {
        const f2 a = h2_to_f2(v.x), b = h2_to_f2(v.y);
        return make_float4(a.x, a.y, b.x, b.y);
    }
    return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u), __uint_as_float(v.y << 16),
                       __uint_as_float(v.y & 0xFFFF0000u));
}

int launch_attn_rows(const AttnArgs& a, bool int8, cudaStream_t s);
int launch_attn_rows_shared(const AttnArgs& a, bool int8, cudaStream_t s);
// Query rows of a unit of the prefix (kv_prefix.cuh).
constexpr int kMaxPrefixCtas = 160;
__host__ __device__ constexpr int prefix_rows(int dp) { return dp == 256 ? 32 : 64; }
static_assert(int64_t(kMaxPrefixCtas) * 64 * (128 + 2) * 4 <= kWsOwn - kWsSlots &&
              int64_t(kMaxPrefixCtas) * 32 * (256 + 2) * 4 <= kWsOwn - kWsSlots, "slots exceed the workspace");
// Bytes of the results kept for each of `rows` rows.
inline int64_t own_bytes(int64_t rows, int q_heads, int dim) { return rows * q_heads * (dim * int64_t(4) + 16); }
int launch_attn_prefix(AttnArgs& a, bool int8, cudaStream_t s);
// K or V of one layer as [pages][heads][page_tokens][dim], boxes of box_tokens x box_bytes; `swizzle`: 64- or
// 128-byte rows, so that reads down a column of a box meet no bank twice.  Bytes past the dims arrive as 0.
bool encode_cache(CUtensorMap* map, const KVLayer& c, const uint8_t* base, int box_bytes, int box_tokens, bool swizzle);
int launch_attn_prompt(const AttnArgs& a, bool int8, cudaStream_t s);

}  // namespace qg
