// C-ABI entry points declared in include/qgkv.h: every argument is checked on
// the host before anything is launched.
#include <cstdint>

#include "kv_attention.cuh"
#include "launch.h"
#include "launch_common.cuh"
#include "qgkv_launch.h"

namespace {

bool off16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) != 0; }
bool off4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) != 0; }

bool meets(const void* a, int64_t abytes, const void* b, int64_t bbytes) {
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a), b0 = reinterpret_cast<uintptr_t>(b);
    return a0 < b0 + static_cast<uintptr_t>(bbytes) && b0 < a0 + static_cast<uintptr_t>(abytes);
}

int type_bytes(int type) { return type == QGKV_F32 ? 4 : type == QGKV_F16 || type == QGKV_BF16 ? 2 : 0; }

bool page_size_ok(int p) { return p == 16 || p == 32 || p == 64 || p == 128 || p == 256; }

constexpr int64_t kMost = int64_t(1) << 31;

int check_cache(const qgkv_cache* c, int64_t layer) {
    if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale) return QG_EINVAL;
    if (c->format != QGKV_E4M3 && c->format != QGKV_INT8) return QG_EINVAL;
    if (c->order != QGKV_HND && c->order != QGKV_NHD) return QG_EINVAL;
    if (c->layers < 1 || c->layers > 4096 || layer < 0 || layer >= c->layers) return QG_EINVAL;
    if (c->pages < 1 || c->pages > QGKV_MAX_PAGES || c->heads < 1 || c->heads > 1024) return QG_EINVAL;
    if (!page_size_ok(c->page_tokens) || c->head_dim < 16 || c->head_dim > 256 || c->head_dim % 16) return QG_EINVAL;
    const int64_t bytes = static_cast<int64_t>(c->heads) * c->page_tokens * c->head_dim;
    if (c->page_stride < bytes || (c->layers > 1 && c->layer_stride < bytes)) return QG_EINVAL;
    if (c->page_stride >= (int64_t(1) << 40) || c->layer_stride > (int64_t(1) << 50) || c->layer_stride < 0)
        return QG_EINVAL;
    if (off16(c->k) || off16(c->v) || off4(c->k_scale) || off4(c->v_scale) || c->page_stride % 16 ||
        c->layer_stride % 16)
        return QG_EALIGN;
    return QG_OK;
}

int check_batch(const int32_t* table, int64_t width, const int32_t* lens, int batch) {
    if (!table || !lens || batch < 1 || batch > QGKV_MAX_BATCH || width < 1 || width > QGKV_MAX_PAGES) return QG_EINVAL;
    if (off4(table) || off4(lens)) return QG_EALIGN;
    return QG_OK;
}

int check_workspace(const void* ws, int64_t bytes) {
    if (!ws) return QG_EINVAL;
    if (bytes < qg::kWsTotal) return QG_ESCRATCH;
    if (reinterpret_cast<uintptr_t>(ws) & 255u) return QG_EALIGN;
    return QG_OK;
}

// Rows of `heads` x dim values: strides that hold them, in whole 16 bytes.  No
// rows need no memory (an empty tensor's address is null).
int check_rows(const void* p, int type, int64_t rows, int heads, int dim, int64_t row_stride, int64_t head_stride) {
    const int size = type_bytes(type);
    if ((!p && rows) || !size || rows < 0 || rows > kMost) return QG_EINVAL;
    if (row_stride < dim || head_stride < dim || row_stride > kMost || head_stride > kMost) return QG_EINVAL;
    if (off16(p) || row_stride * size % 16 || head_stride * size % 16) return QG_EALIGN;
    (void)heads;
    return QG_OK;
}

// Outputs of the table operations: none meets another or an input.
struct Piece {
    const void* p;
    int64_t bytes;
};
bool any_meet(const Piece* outs, int nouts, const Piece* ins, int nins) {
    for (int i = 0; i < nouts; ++i) {
        for (int j = 0; j < nins; ++j)
            if (ins[j].p && meets(outs[i].p, outs[i].bytes, ins[j].p, ins[j].bytes)) return true;
        for (int j = i + 1; j < nouts; ++j)
            if (meets(outs[i].p, outs[i].bytes, outs[j].p, outs[j].bytes)) return true;
    }
    return false;
}

int64_t cache_bytes(const qgkv_cache* c) {
    return (c->layers - 1) * c->layer_stride + (c->pages - 1) * c->page_stride +
           static_cast<int64_t>(c->heads) * c->page_tokens * c->head_dim;
}

// The checks of both attentions; fills `a`.  *done: there is nothing to launch.
int prepare_attention(const qgkv_cache* cache, int64_t layer, const void* q, void* out, float* lse, int type,
                      int64_t rows, int q_heads, int64_t row_stride, int64_t head_stride, const int32_t* table,
                      int64_t table_width, const int32_t* lens, const int32_t* starts, int batch, float scale,
                      void* workspace, int64_t workspace_bytes, Piece plan, qg::AttnArgs& a, bool* done) {
    *done = true;
    int rc = check_cache(cache, layer);
    if (rc != QG_OK) return rc;
    if ((rc = check_batch(table, table_width, lens, batch)) != QG_OK) return rc;
    if (q_heads < 1 || q_heads % cache->heads || q_heads > 65536) return QG_EINVAL;
    if ((!out && rows) || !(scale > -3.0e38f && scale < 3.0e38f)) return QG_EINVAL;
    if ((rc = check_rows(q, type, rows, q_heads, cache->head_dim, row_stride, head_stride)) != QG_OK) return rc;
    if (!starts && rows != batch) return QG_EINVAL;
    // the kernels count the query rows of a cache head (tokens x heads of a group) in 32 bits
    if (rows * (q_heads / cache->heads) > kMost - 512) return QG_EINVAL;
    if (off16(out) || off4(lse) || off4(starts)) return QG_EALIGN;
    if ((rc = check_workspace(workspace, workspace_bytes)) != QG_OK) return rc;
    if (rows == 0) return QG_OK;
    const int64_t size = type_bytes(type);
    const int64_t in = ((rows - 1) * row_stride + (q_heads - 1) * head_stride + cache->head_dim) * size;
    const int64_t written = rows * q_heads * cache->head_dim * size, held = cache_bytes(cache);
    if (meets(out, written, q, in) || meets(out, written, cache->k, held) || meets(out, written, cache->v, held) ||
        (lse && (meets(lse, rows * q_heads * 4, out, written) || meets(lse, rows * q_heads * 4, q, in))))
        return QG_EALIAS;
    if (plan.p && (meets(out, written, plan.p, plan.bytes) || (lse && meets(lse, rows * q_heads * 4, plan.p, plan.bytes))))
        return QG_EALIAS;
    unsigned* st = qg::status_ptr();
    if (!st) return qg::cuda_fail(cudaGetLastError());
    a = {};
    a.c = qg::layer_of(*cache, layer);
    a.q = q, a.out = out, a.lse = lse, a.q_row = row_stride, a.q_head = head_stride, a.type = type;
    a.q_heads = q_heads, a.group = q_heads / cache->heads;
    a.table = table, a.width = table_width, a.lens = lens, a.starts = starts, a.batch = batch, a.rows = rows;
    a.scale_log2 = scale * 1.4426950408889634f;
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.part = reinterpret_cast<float*>(ws + qg::kWsPart);
    a.splits = reinterpret_cast<int4*>(ws + qg::kWsSplits);
    a.count = reinterpret_cast<unsigned*>(ws + qg::kWsCounters) + qg::kCntAttn;
    a.status = st;
    *done = false;
    return QG_OK;
}

bool many_rows(const qg::AttnArgs& a) {
    // The tcgen05 kernel takes as long for one query row (token x head of a
    // group) a sequence as for 256, the row kernel's time grows with them.  Row
    // kernel / tcgen05 kernel, us, e4m3, 32 / 8 heads of 128, by query rows a
    // sequence (the same for each of a call):
    //   16 sequences of up to 4100 tokens: bf16 96 rows 128 / 113, 128 rows 161 /
    //   113, 256 rows 297 / 121; fp32 64 rows 111 / 141, 128 rows 198 / 144, 256
    //   rows 368 / 255; f16 (two parts of p for two tiles) 128 rows 175 / 177, 256
    //   rows 326 / 187
    //   48 of up to 1000: bf16 64 rows 122 / 98, 128 rows 223 / 101; f16 128 rows
    //   238 / 166
    //   few row blocks, whose keys are split, bf16: 4 of up to 4100: 128 rows 56 /
    //   56, 256 rows 92 / 59; one of 1000: 128 rows 18 / 30, 256 rows 27 / 31; of
    //   8000: 128 rows 40 / 60, 256 rows 59 / 61; of 30000: 128 rows 93 / 90, 256
    //   rows 161 / 95
    // The border is late for f16 batches and for few but long sequences, by up to
    // 1.4 times.  The mean over a call decides for all of it: a prompt among many
    // single tokens goes the way of the single tokens, or they its.
    const int sms = qg::sm_count(qg::current_device());
    const int few = a.type == QGKV_F16 || 2 * static_cast<int64_t>(a.batch) * a.c.heads < sms ? 256 : 128;
    return a.rows * a.group >= static_cast<int64_t>(few) * a.batch && a.starts && a.c.dim <= 128;
}

int launch_attention(const qg::AttnArgs& a, bool int8, cudaStream_t stream) {
    return many_rows(a) ? qg::launch_attn_prompt(a, int8, stream) : qg::launch_attn_rows(a, int8, stream);
}

// The pages that sequences read beside the first, at most by the table's width, have to be
// worth a second kernel and the join (more than a plan saves where there are several groups, each of which
// reads its prefix once).  Shared / each for itself, us:
//   4 beams of 820 tokens, 4 heads of 64 (1.3 MB): 13.6 / 8.2
//   4 of 1080, 8 heads of 128 (6.7 MB): 15.0 / 10.8;  8 groups of 4 of 1060, 4 heads of 64 (17 MB): 15.7 / 14.2
//   4 of 4160, 8 heads of 128 (26 MB): 16.3 / 18.2;  48 of 1320 (130 MB): 26 / 27;  48 of 8800 (850 MB): 42 / 97
// Widths are all that the host knows: behind a table much wider than its
// sequences a small plan is followed all the same.  And of the groups it knows their number: one large group
// beside many of one sequence does not share (the header says how to pass them).  Nor does the prefix kernel read as
// fast as the row kernel, for a step takes it as long for few rows as for 64: with 16 groups
// behind up to 6000 tokens, bf16, of 2 / 3 / 4 / 6 sequences, shared 57 / 57 / 65 / 70, each for itself 35 / 47 / 58 /
// 81 (8 heads of 64), 67 / 69 / 78 / 85 and 47 / 63 / 77 / 109 (of 128), 77 / 78 / 81 / 94 and 51 / 66 / 84 / 116 (4 of 256).
constexpr double kLeastSaved = 16 << 20;
constexpr int kLeastMembers = 4;  // sequences of a call to each group
bool worth_sharing(const qg::AttnArgs& a, int ngroups) {
    if (a.batch < static_cast<int64_t>(kLeastMembers) * ngroups) return false;
    const double most = 2.0 * (a.batch - 1) * a.width * (int64_t(1) << a.c.log2p) * a.c.heads * a.c.dim;
    return most >= kLeastSaved && !many_rows(a);
}

}  // namespace

extern "C" {

int64_t qgkv_workspace_bytes(void) { return qg::kWsTotal; }

int qgkv_append(const qgkv_cache* cache, int64_t layer, const void* k, const void* v, int type, int64_t rows,
                int64_t row_stride, int64_t head_stride, const int32_t* table, int64_t table_width,
                const int32_t* lens, const int32_t* starts, int batch, cudaStream_t stream) {
    int rc = check_cache(cache, layer);
    if (rc != QG_OK) return rc;
    if ((rc = check_batch(table, table_width, lens, batch)) != QG_OK) return rc;
    if ((rc = check_rows(k, type, rows, cache->heads, cache->head_dim, row_stride, head_stride)) != QG_OK) return rc;
    if ((rc = check_rows(v, type, rows, cache->heads, cache->head_dim, row_stride, head_stride)) != QG_OK) return rc;
    if (!starts && rows != batch) return QG_EINVAL;
    if (off4(starts)) return QG_EALIGN;
    if (rows == 0) return QG_OK;
    const int64_t in = ((rows - 1) * row_stride + (cache->heads - 1) * head_stride + cache->head_dim) * type_bytes(type);
    const int64_t held = cache_bytes(cache);
    if (meets(k, in, cache->k, held) || meets(k, in, cache->v, held) || meets(v, in, cache->k, held) ||
        meets(v, in, cache->v, held))
        return QG_EALIAS;
    unsigned* st = qg::status_ptr();
    if (!st) return qg::cuda_fail(cudaGetLastError());
    return qg::launch_append(*cache, layer, k, v, type, rows, row_stride, head_stride, table, table_width, lens, starts,
                             batch, st, stream);
}

int qgkv_append_rotary(const qgkv_cache* cache, int64_t layer, const void* q, const void* k, const void* v, int type,
                       int64_t rows, int q_heads, int64_t q_row, int64_t q_head, int64_t kv_row, int64_t kv_head,
                       const float* rope, int64_t positions, int turned, int pairs, void* q_out, const int32_t* table,
                       int64_t table_width, const int32_t* lens, const int32_t* starts, int batch,
                       cudaStream_t stream) {
    int rc = check_cache(cache, layer);
    if (rc != QG_OK) return rc;
    if ((rc = check_batch(table, table_width, lens, batch)) != QG_OK) return rc;
    const int dim = cache->head_dim;
    if (!rope || positions < 1 || positions > kMost || turned < 16 || turned > dim || turned % 16) return QG_EINVAL;
    if (pairs != QGKV_INTERLEAVED && pairs != QGKV_HALVES) return QG_EINVAL;
    if ((rc = check_rows(k, type, rows, cache->heads, dim, kv_row, kv_head)) != QG_OK) return rc;
    if ((rc = check_rows(v, type, rows, cache->heads, dim, kv_row, kv_head)) != QG_OK) return rc;
    if (q) {
        if (q_heads < 1 || q_heads > 65536 || (!q_out && rows)) return QG_EINVAL;
        if ((rc = check_rows(q, type, rows, q_heads, dim, q_row, q_head)) != QG_OK) return rc;
    }
    if (!starts && rows != batch) return QG_EINVAL;
    if (off4(starts) || off16(rope) || (q && off16(q_out))) return QG_EALIGN;
    if (rows == 0) return QG_OK;
    const int64_t size = type_bytes(type), held = cache_bytes(cache);
    const int64_t kv_in = ((rows - 1) * kv_row + (cache->heads - 1) * kv_head + dim) * size;
    const int64_t angles = positions * turned * 4, numbers = batch * table_width * 4;
    const Piece ins[] = {{k, kv_in}, {v, kv_in}, {rope, angles}, {table, numbers}, {lens, batch * int64_t(4)},
                         {starts, starts ? (batch + 1) * int64_t(4) : 0}};
    const Piece codes[] = {{cache->k, held}, {cache->v, held}};
    for (const Piece& c : codes)
        for (const Piece& in : ins)
            if (in.p && meets(c.p, c.bytes, in.p, in.bytes)) return QG_EALIAS;
    if (q) {
        const int64_t q_in = ((rows - 1) * q_row + (q_heads - 1) * q_head + dim) * size;
        const Piece out = {q_out, rows * q_heads * dim * size};
        if (any_meet(&out, 1, ins, 6) || any_meet(&out, 1, codes, 2) || meets(q, q_in, cache->k, held) ||
            meets(q, q_in, cache->v, held))
            return QG_EALIAS;
        const bool itself = q_out == q && (q_head == dim || q_heads == 1) && (q_row == q_heads * int64_t(dim) || rows == 1);
        if (!itself && meets(q_out, out.bytes, q, q_in)) return QG_EALIAS;
    }
    unsigned* st = qg::status_ptr();
    if (!st) return qg::cuda_fail(cudaGetLastError());
    return qg::launch_append_rotary(*cache, layer, q, k, v, type, rows, q_heads, q_row, q_head, kv_row, kv_head, rope,
                                    positions, turned, pairs, q_out, table, table_width, lens, starts, batch, st,
                                    stream);
}

int qgkv_attention(const qgkv_cache* cache, int64_t layer, const void* q, void* out, float* lse, int type,
                   int64_t rows, int q_heads, int64_t row_stride, int64_t head_stride, const int32_t* table,
                   int64_t table_width, const int32_t* lens, const int32_t* starts, int batch, float scale,
                   void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
    qg::AttnArgs a;
    bool done;
    const int rc = prepare_attention(cache, layer, q, out, lse, type, rows, q_heads, row_stride, head_stride, table,
                                     table_width, lens, starts, batch, scale, workspace, workspace_bytes, {nullptr, 0},
                                     a, &done);
    return rc != QG_OK || done ? rc : launch_attention(a, cache->format == QGKV_INT8, stream);
}

int qgkv_share(int64_t pages, int page_tokens, const int32_t* table, int64_t table_width, const int32_t* lens,
               const int32_t* starts, int64_t rows, int batch, const int32_t* groups, int ngroups, int32_t* plan,
               cudaStream_t stream) {
    const int rc = check_batch(table, table_width, lens, batch);
    if (rc != QG_OK) return rc;
    if (pages < 1 || pages > QGKV_MAX_PAGES || !page_size_ok(page_tokens) || rows < 0 || rows > kMost) return QG_EINVAL;
    if (!groups || ngroups < 1 || ngroups > QGKV_MAX_BATCH || !plan || (!starts && rows != batch)) return QG_EINVAL;
    if (table_width * page_tokens > kMost - page_tokens) return QG_EINVAL;  // tokens are counted in 32 bits
    if (off4(starts) || off4(groups) || off16(plan)) return QG_EALIGN;
    const Piece ins[] = {{table, batch * table_width * 4}, {lens, batch * 4}, {starts, (batch + 1) * 4},
                         {groups, (ngroups + 1) * 4}};
    const Piece to = {plan, (4 * ngroups + batch) * 4};
    if (any_meet(&to, 1, ins, 4)) return QG_EALIAS;
    unsigned* st = qg::status_ptr();
    if (!st) return qg::cuda_fail(cudaGetLastError());
    return qg::launch_share(pages, page_tokens, table, table_width, lens, starts, rows, batch, groups, ngroups, plan, st,
                            stream);
}

int qgkv_attention_shared(const qgkv_cache* cache, int64_t layer, const void* q, void* out, float* lse, int type,
                          int64_t rows, int q_heads, int64_t row_stride, int64_t head_stride, const int32_t* table,
                          int64_t table_width, const int32_t* lens, const int32_t* starts, int batch,
                          const int32_t* plan, int ngroups, float scale, void* workspace, int64_t workspace_bytes,
                          cudaStream_t stream) {
    if (!plan || ngroups < 1 || ngroups > QGKV_MAX_BATCH) return QG_EINVAL;
    if (off16(plan)) return QG_EALIGN;
    qg::AttnArgs a;
    bool done;
    const int rc = prepare_attention(cache, layer, q, out, lse, type, rows, q_heads, row_stride, head_stride, table,
                                     table_width, lens, starts, batch, scale, workspace, workspace_bytes,
                                     {plan, (4 * int64_t(ngroups) + batch) * 4}, a, &done);
    if (rc != QG_OK || done) return rc;
    const bool int8 = cache->format == QGKV_INT8;
    if (!worth_sharing(a, ngroups) || qg::own_bytes(rows, q_heads, cache->head_dim) > qg::kWsSplits - qg::kWsOwn)
        return launch_attention(a, int8, stream);
    uint8_t* ws = static_cast<uint8_t*>(workspace);
    a.groups = reinterpret_cast<const int4*>(plan);
    a.skip = plan + 4 * int64_t(ngroups);
    a.ngroups = ngroups;
    a.own_ml = reinterpret_cast<float4*>(ws + qg::kWsOwn);
    a.own = reinterpret_cast<float*>(a.own_ml + rows * q_heads);
    a.slots = reinterpret_cast<float*>(ws + qg::kWsSlots);
    const int launched = qg::launch_attn_prefix(a, int8, stream);
    return launched != QG_OK ? launched : qg::launch_attn_rows_shared(a, int8, stream);
}

int qgkv_copy_pages(const qgkv_cache* cache, const int32_t* src, const int32_t* dst, const int32_t* count,
                    int64_t most, cudaStream_t stream) {
    const int rc = check_cache(cache, 0);
    if (rc != QG_OK) return rc;
    if (most < 0 || most > QGKV_MAX_PAGES || (most && (!src || !dst))) return QG_EINVAL;
    if (off4(src) || off4(dst) || off4(count)) return QG_EALIGN;
    if (most == 0) return QG_OK;
    unsigned* st = qg::status_ptr();
    if (!st) return qg::cuda_fail(cudaGetLastError());
    return qg::launch_copy_pages(*cache, src, dst, count, most, st, stream);
}

int qgkv_fork(const qgkv_cache* cache, const int32_t* table, int64_t table_width, const int32_t* lens, int batch,
              const int32_t* parent, int batch2, const int32_t* refs, int32_t* table2, int32_t* lens2, int32_t* refs2,
              void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
    int rc = check_cache(cache, 0);
    if (rc != QG_OK) return rc;
    if ((rc = check_batch(table, table_width, lens, batch)) != QG_OK) return rc;
    if (!parent || !refs || !table2 || !lens2 || !refs2 || batch2 < 1 || batch2 > QGKV_MAX_BATCH) return QG_EINVAL;
    if (off16(refs) || off16(refs2) || off4(parent) || off4(table2) || off4(lens2)) return QG_EALIGN;
    if ((rc = check_workspace(workspace, workspace_bytes)) != QG_OK) return rc;
    const Piece ins[] = {{table, batch * table_width * 4}, {lens, batch * 4}, {parent, batch2 * 4}, {refs, cache->pages * 4}};
    const Piece outs[] = {{table2, batch2 * table_width * 4}, {lens2, batch2 * 4}, {refs2, cache->pages * 4}};
    if (any_meet(outs, 3, ins, 4)) return QG_EALIAS;
    unsigned* st = qg::status_ptr();
    if (!st) return qg::cuda_fail(cudaGetLastError());
    return qg::launch_fork(*cache, table, table_width, lens, batch, parent, batch2, refs, table2, lens2, refs2,
                           static_cast<uint8_t*>(workspace), st, stream);
}

int qgkv_compact(const qgkv_cache* cache, const int32_t* table, int64_t table_width, const int32_t* lens, int batch,
                 const uint8_t* drop, const int32_t* refs, int32_t* table2, int32_t* lens2, int32_t* refs2,
                 int32_t* count, void* workspace, int64_t workspace_bytes, cudaStream_t stream) {
    int rc = check_cache(cache, 0);
    if (rc != QG_OK) return rc;
    if ((rc = check_batch(table, table_width, lens, batch)) != QG_OK) return rc;
    if (!refs || !table2 || !lens2 || !refs2 || !count) return QG_EINVAL;
    if (off16(refs) || off16(refs2) || off4(table2) || off4(lens2) || off4(count)) return QG_EALIGN;
    if ((rc = check_workspace(workspace, workspace_bytes)) != QG_OK) return rc;
    const Piece ins[] = {{table, batch * table_width * 4}, {lens, batch * 4}, {drop, batch}, {refs, cache->pages * 4}};
    const Piece outs[] = {{table2, batch * table_width * 4}, {lens2, batch * 4}, {refs2, cache->pages * 4}, {count, 4}};
    if (any_meet(outs, 4, ins, 4)) return QG_EALIAS;
    unsigned* st = qg::status_ptr();
    if (!st) return qg::cuda_fail(cudaGetLastError());
    return qg::launch_compact(*cache, table, table_width, lens, batch, drop, refs, table2, lens2, refs2, count,
                              static_cast<uint8_t*>(workspace), st, stream);
}

int qgkv_reserve(int64_t pages, int page_tokens, int32_t* table, int64_t table_width, const int32_t* lens,
                 const int32_t* add, int batch, int32_t* refs, void* workspace, int64_t workspace_bytes,
                 cudaStream_t stream) {
    int rc = check_batch(table, table_width, lens, batch);
    if (rc != QG_OK) return rc;
    if (pages < 1 || pages > QGKV_MAX_PAGES || !page_size_ok(page_tokens) || !refs) return QG_EINVAL;
    if (off16(refs) || off4(add)) return QG_EALIGN;
    if ((rc = check_workspace(workspace, workspace_bytes)) != QG_OK) return rc;
    const Piece ins[] = {{lens, batch * 4}, {add, batch * 4}};
    const Piece outs[] = {{table, batch * table_width * 4}, {refs, pages * 4}};
    if (any_meet(outs, 2, ins, 2)) return QG_EALIAS;
    unsigned* st = qg::status_ptr();
    if (!st) return qg::cuda_fail(cudaGetLastError());
    return qg::launch_reserve(pages, page_tokens, table, table_width, lens, add, batch, refs,
                              static_cast<uint8_t*>(workspace), st, stream);
}

int qgkv_free(int64_t pages, int page_tokens, int32_t* table, int64_t table_width, int32_t* lens, const uint8_t* drop,
              int batch, int32_t* refs, cudaStream_t stream) {
    const int rc = check_batch(table, table_width, lens, batch);
    if (rc != QG_OK) return rc;
    if (pages < 1 || pages > QGKV_MAX_PAGES || !page_size_ok(page_tokens) || !refs) return QG_EINVAL;
    if (off4(refs)) return QG_EALIGN;
    const Piece ins[] = {{drop, batch}};
    const Piece outs[] = {{table, batch * table_width * 4}, {lens, batch * 4}, {refs, pages * 4}};
    if (any_meet(outs, 3, ins, 1)) return QG_EALIAS;
    unsigned* st = qg::status_ptr();
    if (!st) return qg::cuda_fail(cudaGetLastError());
    return qg::launch_free(pages, page_tokens, table, table_width, lens, drop, batch, refs, st, stream);
}

int qgbeam_select(const void* logits, int type, const float* cum, int requests, int beams, int64_t vocab,
                  int64_t row_stride, int keep, float* scores, int32_t* tokens, int32_t* parents, void* workspace,
                  int64_t workspace_bytes, cudaStream_t stream) {
    const int size = type_bytes(type);
    if (!logits || !cum || !scores || !tokens || !parents || !size) return QG_EINVAL;
    if (requests < 1 || requests > QGKV_MAX_BATCH || beams < 1 || beams > QGKV_MAX_BEAMS) return QG_EINVAL;
    if (vocab < 1 || vocab >= kMost - 4096 || row_stride < vocab || row_stride > kMost) return QG_EINVAL;
    if (keep < 1 || keep > QGKV_MAX_KEEP || keep > beams * vocab) return QG_EINVAL;
    if ((reinterpret_cast<uintptr_t>(logits) & static_cast<uintptr_t>(size - 1)) || off4(cum) || off4(scores) ||
        off4(tokens) || off4(parents))
        return QG_EALIGN;
    int rc = check_workspace(workspace, workspace_bytes);
    if (rc != QG_OK) return rc;
    const int64_t rows = static_cast<int64_t>(requests) * beams, n = static_cast<int64_t>(requests) * keep * 4;
    const Piece ins[] = {{logits, ((rows - 1) * row_stride + vocab) * size}, {cum, rows * 4}};
    const Piece outs[] = {{scores, n}, {tokens, n}, {parents, n}};
    if (any_meet(outs, 3, ins, 2)) return QG_EALIAS;
    if (!qg::status_ptr()) return qg::cuda_fail(cudaGetLastError());
    return qg::launch_beam_select(logits, type, cum, requests, beams, vocab, row_stride, keep, scores, tokens, parents,
                                  static_cast<uint8_t*>(workspace), stream);
}

int qglogits_adjust(const void* logits, int type, int64_t rows, int64_t vocab, int64_t row_stride, void* out,
                    int out_type, int64_t out_stride, const int32_t* history, int64_t width, const int32_t* lens,
                    const int32_t* prompt_lens, const float* repetition, const float* presence, const float* frequency,
                    const int32_t* bias_tokens, const float* bias, int biases, const float* temperature,
                    const uint32_t* mask, int64_t mask_words, int masks, const int32_t* mask_rows,
                    cudaStream_t stream) {
    const int64_t size = type_bytes(type), out_size = type_bytes(out_type);
    if (!size || !(out_type == type || out_type == QGKV_F32)) return QG_EINVAL;
    if (rows < 0 || rows > QGKV_MAX_BATCH * QGKV_MAX_BEAMS || vocab < 1 || vocab >= kMost - 4096) return QG_EINVAL;
    if (rows && (!logits || !out)) return QG_EINVAL;
    if (row_stride < vocab || row_stride > kMost || out_stride < vocab || out_stride > kMost) return QG_EINVAL;
    if (rows == 0) return QG_OK;
    if (history) {
        if (!lens || width < 1 || width > QGKV_MAX_HISTORY) return QG_EINVAL;
    } else if (lens || prompt_lens || repetition || presence || frequency) {
        return QG_EINVAL;
    }
    if (biases < 0 || biases > QGKV_MAX_BIASES || (biases && (!bias_tokens || !bias)) || (!biases && (bias_tokens || bias)))
        return QG_EINVAL;
    if (mask) {
        if (masks < 1 || mask_words < (vocab + 31) / 32 || mask_words > kMost || (!mask_rows && masks < rows)) return QG_EINVAL;
    } else if (mask_rows) {
        return QG_EINVAL;
    }
    if ((reinterpret_cast<uintptr_t>(logits) & static_cast<uintptr_t>(size - 1)) ||
        (reinterpret_cast<uintptr_t>(out) & static_cast<uintptr_t>(out_size - 1)) || off4(history) || off4(lens) ||
        off4(prompt_lens) || off4(repetition) || off4(presence) || off4(frequency) || off4(bias_tokens) || off4(bias) ||
        off4(temperature) || off4(mask) || off4(mask_rows))
        return QG_EALIGN;
    const int64_t words = rows * 4;
    const Piece ins[] = {{history, rows * width * 4}, {lens, words}, {prompt_lens, words}, {repetition, words},
                         {presence, words}, {frequency, words}, {bias_tokens, words * biases}, {bias, words * biases},
                         {temperature, words}, {mask, masks * mask_words * 4}, {mask_rows, words}};
    const Piece to = {out, ((rows - 1) * out_stride + vocab) * out_size};
    if (any_meet(&to, 1, ins, 11)) return QG_EALIAS;
    const bool itself = out == logits && out_type == type && (out_stride == row_stride || rows == 1);
    if (!itself && meets(out, to.bytes, logits, ((rows - 1) * row_stride + vocab) * size)) return QG_EALIAS;
    unsigned* st = qg::status_ptr();
    if (!st) return qg::cuda_fail(cudaGetLastError());
    return qg::launch_logits_adjust(logits, type, rows, vocab, row_stride, out, out_type, out_stride, history, width,
                                    lens, prompt_lens, repetition, presence, frequency, bias_tokens, bias, biases,
                                    temperature, mask, mask_words, masks, mask_rows, st, stream);
}

}  // extern "C"
