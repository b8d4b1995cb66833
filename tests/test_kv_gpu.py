"""GPU tests of the decode-state operators (include/qgkv.h) against plain
implementations in 64 bits.

Attention tolerance.  With A = sum p |v| of an output, S the largest
scale * sum |q k| of its row and L its tokens: q and p of fp32 queries enter as
two f16 parts (relative 2^-22 each), 16-bit q exactly, p of bf16 queries as one
f16 part (2^-11), the scores' fp32 sums and scaling are off by at most
4 S 2^-22 (which changes p by that factor), 2^x by 2^-22, and sums of L / 64
steps plus joins by (16 + L / 64) 2^-22 of A; the output's own rounding adds
eps / 2.  A weight p * scale far below the row's largest, W, is cut at f16's
smallest step, 2^-39 W, which counts only where the large weights meet codes of
zero: L 2^-38 W times the largest code.  Everything else (codes, scales, tables, pages, selected tokens) is
compared bit for bit.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_quantised_weight_gb300 import build, qgemv  # noqa: E402

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


@pytest.fixture(scope="module")
def kv():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    from block_quantised_weight_gb300 import qgkv
    return qgkv


@pytest.fixture(scope="module")
def ws(kv):
    return kv.KVWorkspace("cuda")


@pytest.fixture(autouse=True)
def status_clean(kv):
    yield
    torch.cuda.synchronize()
    assert qgemv.qg_device_status() == qgemv.QG_OK


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def values(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).double()


def make(kv, lens, heads, dim, page, fmt, order, seed=0, layers=2, spare=3, width=None):
    """A cache with random codes and scales (every page, held or not) and a table of shuffled pages."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    need = [(n + page - 1) // page for n in lens]
    pages = sum(need) + spare
    cache = kv.KVCache.allocate(layers, pages, heads, page, dim, fmt, order)
    for c in (cache.k, cache.v):
        r = torch.randint(0, 256, c.shape, device="cuda", generator=g, dtype=torch.uint8)
        if fmt == "e4m3":
            r[(r & 0x7F) == 0x7F] = 0x3A
        else:
            r[r == 128] = 127
        c.copy_(r)
    for s in (cache.k_scale, cache.v_scale):
        s.copy_(torch.exp2(torch.randint(-9, -4, s.shape, device="cuda", generator=g).float()) *
                (1 if fmt == "e4m3" else 1.37))
    if fmt == "int8":
        cache.k_scale *= 0.5
    perm = torch.randperm(pages, generator=torch.Generator().manual_seed(seed)).tolist()
    width = width or max(max(need), 1)
    table = np.full((len(lens), width), -1, np.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = perm[at:at + n]
        at += n
    return cache, i32(table.tolist()), i32(lens)


def gather(cache, layer, table, b, n, which):
    """[n, heads, dim] of sequence b in 64 bits."""
    ids = table[b, :(n + cache.page_tokens - 1) // cache.page_tokens].long()
    c = values((cache.k if which == "k" else cache.v)[layer][ids].contiguous(), cache.fmt)
    s = (cache.k_scale if which == "k" else cache.v_scale)[layer][ids].double()
    if cache.order == "hnd":
        c = c.transpose(1, 2)
    return (c * s[:, None, :, None]).flatten(0, 1)[:n]


def attention_ref(cache, layer, q, table, lens, starts, scale):
    """out, lse, A and S of every row, in 64 bits."""
    hq = q.shape[1]
    group = hq // cache.heads
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    absum = torch.zeros_like(out)
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device="cuda")
    smax = torch.zeros_like(lse)
    floor = torch.zeros_like(lse)
    for b, n in enumerate(lens):
        r0, r1 = starts[b], starts[b + 1]
        if n == 0 or r0 == r1:
            continue
        k = gather(cache, layer, table, b, n, "k").repeat_interleave(group, 1)
        v = gather(cache, layer, table, b, n, "v").repeat_interleave(group, 1)
        x = q[r0:r1].double()
        s = torch.einsum("rhd,thd->rht", x, k) * scale
        hidden = torch.arange(n, device="cuda")[None, :] > (n - (r1 - r0) + torch.arange(r1 - r0, device="cuda"))[:, None]
        s.masked_fill_(hidden[:, None, :], -math.inf)
        l = torch.logsumexp(s, -1)
        p = torch.where(torch.isneginf(s), 0.0, torch.exp(s - l[..., None]))
        vz = torch.nan_to_num(v)
        out[r0:r1] = torch.einsum("rht,thd->rhd", p, vz)
        absum[r0:r1] = torch.einsum("rht,thd->rhd", p, vz.abs())
        lse[r0:r1] = l
        vs = cache.v_scale[layer][table[b, :(n + cache.page_tokens - 1) // cache.page_tokens].long()].double()
        vs = vs.repeat_interleave(cache.page_tokens, 0)[:n].repeat_interleave(group, 1)
        floor[r0:r1] = (p * vs.T[None]).amax(-1) * n * 2.0 ** -38 * (448 if cache.fmt == "e4m3" else 127)
        smax[r0:r1] = abs(scale) * torch.einsum("rhd,thd->rht", x.abs(), k.abs()).amax(-1)
    return out, lse, absum, smax, floor


def close(out, lse, ref, most, dtype, one_part=False):
    want, wl, absum, smax, floor = ref
    steps = (16 + most / 64) * 2.0 ** -22
    rel = 4 * smax * 2.0 ** -22 + steps
    tol = absum * (rel[..., None] + (2.0 ** -11 if one_part else 0.0)) + floor[..., None] + 1e-30
    tol = tol + want.abs() * (1.01 * torch.finfo(dtype).eps / 2)
    if dtype == torch.float16:
        tol = tol + 2.0 ** -25
    err = (out.double() - want).abs()
    assert torch.isfinite(out).all()
    assert (err <= tol).all(), f"worst {float((err / tol).max()):.3f} of the tolerance"
    if lse is not None:
        assert torch.equal(torch.isneginf(lse), torch.isneginf(wl))
        ok = ~torch.isneginf(wl)
        assert ((lse.double() - wl).abs()[ok] <= (rel + wl.abs() * 2.0 ** -22 + 2.0 ** -22)[ok]).all()


def starts_of(rows):
    s = [0]
    for n in rows:
        s.append(s[-1] + n)
    return s


def check_attention(kv, ws, lens, rows, hq, heads, dim, page, fmt, order, dtype, seed=0, scale=None, layer=1):
    cache, table, ln = make(kv, lens, heads, dim, page, fmt, order, seed)
    st = starts_of(rows)
    q = torch.randn((st[-1], hq, dim), device="cuda", generator=torch.Generator(device="cuda").manual_seed(seed)) \
        .to(DT[dtype])
    starts = None if all(r == 1 for r in rows) else i32(st)
    out, lse = kv.kv_attention(cache, layer, q, table, ln, starts=starts, scale=scale, return_lse=True, workspace=ws)
    again = kv.kv_attention(cache, layer, q, table, ln, starts=starts, scale=scale, workspace=ws)
    ref = attention_ref(cache, layer, q, table, lens, st, scale or 1 / math.sqrt(dim))
    close(out, lse, ref, max(lens), DT[dtype], one_part=dtype == "bf16")
    assert torch.equal(out, again)  # the same bits whoever joins the parts


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("lens", [[1], [15], [16], [17], [129], [1000], [3, 0, 257, 64, 1]], ids=str)
@pytest.mark.parametrize("dim, hq, heads", [(64, 32, 4), (128, 8, 8), (80, 6, 2)])
def test_attention_one_token(kv, ws, lens, fmt, dim, hq, heads):
    check_attention(kv, ws, lens, [1] * len(lens), hq, heads, dim, 16, fmt, "hnd", "f32")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [16, 64, 96, 128, 144, 256])
@pytest.mark.parametrize("group", [1, 3, 8, 12, 17])
def test_attention_heads_and_dims(kv, ws, dim, group, dtype):
    check_attention(kv, ws, [70, 333, 2], [1, 1, 1], 2 * group, 2, dim, 32, "e4m3", "nhd", dtype, seed=group)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("order", ["hnd", "nhd"])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attention_pages(kv, ws, page, order, fmt):
    check_attention(kv, ws, [page - 1, page, page + 1, 5 * page + 3], [1] * 4, 8, 2, 64, page, fmt, order, "bf16", seed=page)


@pytest.mark.parametrize("rows", [[2], [5, 1, 3], [17, 0, 40], [100, 130]], ids=str)
@pytest.mark.parametrize("dim, dtype", [(64, "f32"), (128, "bf16"), (256, "f16"), (96, "f32")])
@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attention_several_rows(kv, ws, rows, dim, dtype, fmt):
    lens = [r + x for r, x in zip(rows, (0, 77, 300))]
    check_attention(kv, ws, lens, rows, 12, 4, dim, 32, fmt, "hnd", dtype)


@pytest.mark.parametrize("rows", [1, 3, 40, 300])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_int8_small_codes(kv, ws, rows, dtype):
    """Small codes and queries of one sign: the scores are exact to their own size, not to that of 128 * sum(q)."""
    n, dim = 700, 128
    cache, table, ln = make(kv, [n], 2, dim, 32, "int8", "hnd", seed=21)
    g = torch.Generator(device="cuda").manual_seed(22)
    cache.k.copy_(torch.randint(-2, 3, cache.k.shape, device="cuda", generator=g).to(torch.int8).view(torch.uint8))
    cache.k_scale.fill_(1.0)
    q = (1.0 + 0.5 * torch.rand((rows, 4, dim), device="cuda", generator=g)).to(DT[dtype])
    out, lse = kv.kv_attention(cache, 0, q, table, ln, starts=i32([0, rows]), return_lse=True, workspace=ws)
    ref = attention_ref(cache, 0, q, table, [n], [0, rows], 1 / math.sqrt(dim))
    close(out, lse, ref, n, DT[dtype], one_part=dtype == "bf16")


def test_attention_rows_that_see_nothing(kv, ws):
    """More rows than tokens: the first rows' masks leave nothing; also empty sequences among full ones."""
    for lens, rows in (([2, 0, 0], [5, 3, 0]), ([0], [1]), ([0, 90, 0, 1], [1, 1, 1, 1]), ([30], [200])):
        check_attention(kv, ws, lens, rows, 4, 2, 64, 16, "e4m3", "hnd", "f32")


@pytest.mark.parametrize("lens, rows", [
    ([300], [300]), ([1000, 513, 64], [257, 513, 1]), ([129, 0, 700, 128], [128, 0, 5, 128]), ([2100], [130]),
    ([40, 50], [200, 64]), ([128, 256], [128, 256]),
], ids=str)
@pytest.mark.parametrize("group, dim, page, order, dtype, fmt", [
    (1, 64, 16, "hnd", "f32", "e4m3"), (4, 128, 64, "hnd", "bf16", "e4m3"), (8, 64, 32, "nhd", "f16", "int8"),
    (3, 128, 128, "nhd", "f32", "int8"), (12, 96, 16, "hnd", "bf16", "int8"), (2, 80, 256, "hnd", "f32", "e4m3"),
    (5, 16, 16, "nhd", "f16", "e4m3"), (1, 128, 16, "hnd", "f16", "e4m3"),
])
def test_attention_prompts(kv, ws, lens, rows, group, dim, page, order, dtype, fmt):
    """Many rows a sequence: whole blocks of rows, parts of them, rows before the first token."""
    check_attention(kv, ws, lens, rows, 2 * group, 2, dim, page, fmt, order, dtype, seed=group)


def test_attention_prompts_of_many_sequences(kv, ws):
    g = np.random.default_rng(7)
    rows = [int(x) for x in g.integers(30, 400, 60)]
    lens = [r + int(x) for r, x in zip(rows, g.integers(0, 300, 60))]
    check_attention(kv, ws, lens, rows, 8, 4, 64, 32, "e4m3", "hnd", "bf16", seed=60)


@pytest.mark.parametrize("lens, rows", [
    ([20011], [150]), ([9000, 40, 0, 2500, 3], [150, 200, 0, 1500, 90]), ([5000], [5000]), ([640, 700], [64, 64]),
], ids=str)
@pytest.mark.parametrize("heads, group, dim, page, dtype, fmt", [
    (1, 4, 128, 64, "bf16", "e4m3"), (2, 2, 64, 16, "f32", "int8"), (3, 3, 96, 32, "f16", "e4m3"), (8, 1, 128, 128, "f32", "e4m3"),
])
def test_attention_prompts_of_few_blocks(kv, ws, lens, rows, heads, group, dim, page, dtype, fmt):
    """Fewer row blocks than there is room for: their keys are split and the parts joined."""
    check_attention(kv, ws, lens, rows, heads * group, heads, dim, page, fmt, "hnd", dtype, seed=heads)


def test_attention_prompt_nan_codes_of_split_keys(kv, ws):
    """NaN codes of V that only later rows see, in several parts of the keys."""
    lens, rows = [3000], [1500]
    cache, table, ln = make(kv, lens, 2, 64, 16, "e4m3", "hnd", seed=8)
    q = torch.randn((1500, 4, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(9))
    marks = ((1503, 0, 5), (2100, 1, 63), (2101, 0, 6), (2999, 1, 7), (40, 1, 9))
    for tok, head, dim in marks:
        cache.v[1, table[0, tok // 16].long(), head, tok % 16, dim] = 0xFF
    out = kv.kv_attention(cache, 1, q, table, ln, starts=i32([0, 1500]), workspace=ws)
    want = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    for tok, head, dim in marks:
        want[max(0, tok - 1500):, 2 * head:2 * head + 2, dim] = True
    assert torch.equal(torch.isnan(out), want)


def test_attention_prompt_negative_scale(kv, ws):
    check_attention(kv, ws, [200], [150], 4, 2, 64, 16, "int8", "hnd", "f32", scale=-0.1)
    check_attention(kv, ws, [200], [1], 4, 2, 64, 16, "int8", "hnd", "f32", scale=-0.1)


@pytest.mark.parametrize("dtype, orders", [("f32", 20), ("f32", 26), ("f32", 30), ("f16", 26), ("f16", 30), ("bf16", 26)])
@pytest.mark.parametrize("at", [3, 100, 200])
@pytest.mark.parametrize("first", [0, 64, 128, 192])
@pytest.mark.parametrize("group", [1, 4])
def test_attention_prompt_one_large_score(kv, ws, dtype, orders, at, first, group):
    """One token `orders` binary orders above the others, whose values are zero: what 64 of the others carry stays.

    A weight is stored as p' = p * 2^11 (bf16: 2^5) or more, in f16, with two roundings of parts by up to three
    halves of a 2^-24 step each: off by at most 3 * 2^-36 (bf16 3 * 2^-30) of the largest, for each of 64 tokens.
    """
    n, rows, dim = 256, 64, 64
    e4 = lambda x: torch.tensor(float(x)).to(torch.float8_e4m3fn).view(torch.uint8).item()  # noqa: E731
    cache = kv.KVCache.allocate(1, 20, 1, 16, dim, "e4m3", "hnd")
    for c in (cache.k, cache.v):
        c.zero_()
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    k = torch.zeros((n, dim), dtype=torch.uint8, device="cuda")
    v = torch.zeros_like(k)
    v[first:first + 64] = e4(1.0)
    v[at] = 0
    k[at, 0] = e4(orders)
    cache.k[0, :16, 0] = k.view(16, 16, dim)
    cache.v[0, :16, 0] = v.view(16, 16, dim)
    q = torch.zeros((rows, group, dim), device="cuda")
    q[:, :, 0] = math.log(2)
    q = q.to(DT[dtype])
    table = i32([list(range(16))])
    out = kv.kv_attention(cache, 0, q, table, i32([n]), starts=i32([0, rows]), scale=1.0, workspace=ws)
    want, _, absum, smax, _ = attention_ref(cache, 0, q, table, [n], [0, rows], 1.0)
    rel = 4 * smax[..., None] * 2.0 ** -22 + 20 * 2.0 ** -22 + (2.0 ** -11 if dtype == "bf16" else 0.0)
    tol = absum * rel + 64 * 3 * 2.0 ** (-30 if dtype == "bf16" else -36)
    tol = tol + want.abs() * (1.01 * torch.finfo(DT[dtype]).eps / 2) + (2.0 ** -25 if dtype == "f16" else 0.0)
    err = (out.double() - want).abs()
    assert (err <= tol).all(), f"worst {float((err / tol).max()):.3f} of the tolerance"


def test_attention_prompt_masked_tokens_do_not_reach(kv, ws):
    """NaN codes behind the length and in tokens that only later rows see; a missing page."""
    lens, rows = [300], [140]
    cache, table, ln = make(kv, lens, 2, 64, 16, "e4m3", "hnd", seed=3)
    st = starts_of(rows)
    q = torch.randn((140, 4, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(4))
    ref = attention_ref(cache, 0, q, table, lens, st, 0.125)
    last = table[0, 18].long()
    for c in (cache.k, cache.v):
        c[0, last, :, 300 - 288:] = 0x7F
    held = set(table[0].tolist())
    for p in range(cache.pages):
        if p not in held:
            cache.k[0, p] = 0x7F
            cache.v[0, p] = 0xFF
    out, lse = kv.kv_attention(cache, 0, q, table, ln, starts=i32(st), return_lse=True, workspace=ws)
    close(out, lse, ref, 300, torch.float32)
    for tok, head, dim in ((260, 1, 5), (299, 0, 63), (130, 0, 7)):  # rows from tok - 160 on see it
        cache.v[0, table[0, tok // 16].long(), head, tok % 16, dim] = 0x7F
    out = kv.kv_attention(cache, 0, q, table, ln, starts=i32(st), workspace=ws)
    want = torch.zeros(out.shape, dtype=torch.bool, device="cuda")
    want[100:, 2:, 5] = True
    want[139:, :2, 63] = True
    want[:, :2, 7] = True
    assert torch.equal(torch.isnan(out), want)
    assert ((out.double() - ref[0]).abs()[~want] <= (ref[2] * 1e-4)[~want]).all()
    cache.k[0, table[0, 17].long(), 0, 3, 9] = 0xFF  # position 275: rows from 115 on of the first group
    out = kv.kv_attention(cache, 0, q, table, ln, starts=i32(st), workspace=ws)
    assert torch.isnan(out[115:, :2]).all() and torch.isfinite(out[:115, 2:, :5]).all()
    assert not torch.isnan(out[:115, :2, 8:60]).any()


def test_attention_prompt_bad_page_is_reported_and_masked(kv, ws):
    lens, rows = [200], [90]
    cache, table, ln = make(kv, lens, 2, 64, 16, "int8", "hnd", seed=4)
    q = torch.randn((90, 4, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    for wrong in (-1, cache.pages):
        t = table.clone()
        t[0, 2] = wrong
        out = kv.kv_attention(cache, 0, q, t, ln, starts=i32([0, 90]), workspace=ws)
        assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS
        keep = [i for i in range(table.shape[1]) if i != 2]
        ref = attention_ref(cache, 0, q, table[:, keep].contiguous(), [200 - 16], [0, 90], 0.125)
        close(out, None, ref, 200, torch.float32)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_attention_prompt_bad_page_of_many_rows(kv, ws, fmt):
    """The same with enough rows for the prompt kernel and keys in several parts."""
    cache, table, ln = make(kv, [700], 2, 64, 16, fmt, "hnd", seed=6)
    q = torch.randn((300, 4, 64), device="cuda", generator=torch.Generator(device="cuda").manual_seed(7))
    for wrong in (-1, cache.pages):
        t = table.clone()
        t[0, 2] = wrong
        out = kv.kv_attention(cache, 0, q, t, ln, starts=i32([0, 300]), workspace=ws)
        assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS
        keep = [i for i in range(table.shape[1]) if i != 2]
        ref = attention_ref(cache, 0, q, table[:, keep].contiguous(), [700 - 16], [0, 300], 0.125)
        close(out, None, ref, 700, torch.float32)


@pytest.mark.parametrize("batch, context", [(1, 40000), (2, 9001), (70, 300), (300, 40)])
def test_attention_splits(kv, ws, batch, context):
    """Few long sequences (parts joined through the workspace) and many short ones."""
    lens = [max(1, context - 7 * b) for b in range(batch)]
    check_attention(kv, ws, lens, [1] * batch, 8, 2, 64, 64, "int8", "hnd", "f32", seed=batch)


def test_attention_long_offsets(kv, ws):
    """Pages whose byte offsets pass 32 bits: a page stride far larger than the page."""
    dim, page, heads, pages, gap = 64, 16, 2, 9, 1 << 29
    hold = [torch.zeros(pages * gap, dtype=torch.uint8, device="cuda") for _ in range(2)]
    g = torch.Generator(device="cuda").manual_seed(5)
    parts = []
    for h in hold:
        x = h.as_strided((1, pages, heads, page, dim), (pages * gap, gap, page * dim, dim, 1))
        x.copy_(torch.randint(0, 120, x.shape, device="cuda", generator=g, dtype=torch.uint8))
        parts.append(x)
    s = torch.full((1, pages, heads), 0.01, device="cuda")
    cache = kv.KVCache(parts[0], s, parts[1], s.clone(), "int8", "hnd")
    n = pages * page - 3
    table = i32([list(range(pages - 1, -1, -1))])
    q = torch.randn((1, 4, dim), device="cuda", generator=g)
    out, lse = kv.kv_attention(cache, 0, q, table, i32([n]), return_lse=True, workspace=ws)
    close(out, lse, attention_ref(cache, 0, q, table, [n], [0, 1], 1 / 8), n, torch.float32)
    x = torch.randn((1, heads, dim), device="cuda", generator=g)
    kv.kv_append(cache, 0, x, x, table, i32([n - 1]))
    got = gather(cache, 0, table, 0, n, "k")[n - 1]
    assert ((got - x[0].double()).abs() <= cache.k_scale[0, table[0, (n - 1) // page], :, None].double() * 0.501).all()


def test_attention_strided_queries_and_lse_off(kv, ws):
    cache, table, lens = make(kv, [50, 61], 2, 64, 16, "e4m3", "hnd")
    big = torch.randn((2, 3, 8, 64), device="cuda")
    q = big[:, 1]
    out = torch.full((2, 8, 64), 7.0, device="cuda")
    got = kv.kv_attention(cache, 0, q, table, lens, out=out, workspace=ws)
    assert got is out
    close(out, None, attention_ref(cache, 0, q, table, [50, 61], [0, 1, 2], 1 / 8), 61, torch.float32)


def test_attention_masked_tokens_do_not_reach(kv, ws):
    """NaN codes and NaN scales behind the length, and NaN codes in tokens that only later rows see."""
    lens, rows = [37], [6]
    cache, table, ln = make(kv, lens, 2, 64, 16, "e4m3", "hnd", seed=3)
    st = starts_of(rows)
    q = torch.randn((6, 4, 64), device="cuda")
    ref = attention_ref(cache, 0, q, table, lens, st, 0.125)
    for c in (cache.k, cache.v):
        c[0, table[0, 2].long(), :, 37 - 32:] = 0x7F         # behind the length, in its last page
    held = set(table[0].tolist())
    for p in range(cache.pages):
        if p not in held:
            cache.k[0, p] = 0x7F
            cache.v[0, p] = 0xFF
            cache.k_scale[0, p] = math.nan
            cache.v_scale[0, p] = math.inf
    out, lse = kv.kv_attention(cache, 0, q, table, ln, starts=i32(st), return_lse=True, workspace=ws)
    close(out, lse, ref, 37, torch.float32)
    # V of the token that rows 3, 4 and 5 see (position 34) in head 1, dim 5
    cache.v[0, table[0, 2].long(), 1, 34 - 32, 5] = 0x7F
    out = kv.kv_attention(cache, 0, q, table, ln, starts=i32(st), workspace=ws)
    bad = torch.isnan(out)
    want = torch.zeros_like(bad)
    want[3:, 2:, 5] = True
    assert torch.equal(bad, want)
    ok = ~want
    assert ((out.double() - ref[0]).abs()[ok] <= (ref[2] * 1e-4)[ok]).all()
    # K of position 35: rows 4 and 5 of the first head's group become NaN, the others keep their values
    cache.k[0, table[0, 2].long(), 0, 35 - 32, 9] = 0xFF
    out = kv.kv_attention(cache, 0, q, table, ln, starts=i32(st), workspace=ws)
    assert torch.isnan(out[4:, :2]).all() and torch.isfinite(out[:4, :2]).all()


def test_attention_scales_of_all_sizes(kv, ws):
    """Blocks whose scales differ by 2^60, blocks of zeros (scale 0), and a query of large values."""
    torch.manual_seed(11)
    lens = [200]
    cache, table, ln = make(kv, lens, 2, 64, 16, "e4m3", "hnd", seed=9)
    cache.v_scale[0, table[0, ::2].long()] *= 2.0 ** 40
    cache.v_scale[0, table[0, 1::3].long()] *= 2.0 ** -20
    cache.v_scale[0, table[0, 4].long()] = 0.0
    cache.k_scale[0, table[0, 5].long()] = 0.0
    q = torch.randn((1, 8, 64), device="cuda") * torch.exp2(torch.arange(8, device="cuda") * 12.0 - 60)[None, :, None]
    scale = 1e-4
    out, lse = kv.kv_attention(cache, 0, q, table, ln, scale=scale, return_lse=True, workspace=ws)
    close(out, lse, attention_ref(cache, 0, q, table, lens, [0, 1], scale), 200, torch.float32)


def test_attention_non_finite_query(kv, ws):
    cache, table, ln = make(kv, [40, 40], 1, 64, 16, "int8", "hnd", seed=2)
    q = torch.randn((2, 3, 64), device="cuda")
    q[0, 1, 7] = math.nan
    ref = attention_ref(cache, 0, torch.nan_to_num(q), table, [40, 40], [0, 1, 2], 0.125)
    out = kv.kv_attention(cache, 0, q, table, ln, workspace=ws)
    assert torch.isnan(out[0, 1]).all()
    ok = [(0, 0), (0, 2), (1, 0), (1, 1), (1, 2)]
    for r, h in ok:
        assert ((out[r, h].double() - ref[0][r, h]).abs() <= ref[2][r, h] * 1e-4).all()


def test_attention_bad_page_is_reported_and_masked(kv, ws):
    lens = [90]
    cache, table, ln = make(kv, lens, 2, 64, 16, "e4m3", "hnd", seed=4)
    q = torch.randn((1, 4, 64), device="cuda")
    for wrong in (-1, cache.pages, 2 ** 31 - 1):
        t = table.clone()
        t[0, 2] = wrong
        out = kv.kv_attention(cache, 0, q, t, ln, workspace=ws)
        assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS
        # the tokens of that page count as masked: the same as without them
        keep = [0, 1, 3, 4, 5]
        ref = attention_ref(cache, 0, q, table[:, keep].contiguous(), [90 - 16], [0, 1], 0.125)
        close(out, None, ref, 90, torch.float32)
    out = kv.kv_attention(cache, 0, q, table, i32([7 * 16 + 1]), workspace=ws)  # longer than the table
    assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS


def test_attention_other_stream_and_graph(kv, ws):
    """On a stream of its own with its own workspace, and replayed from a graph with other lengths."""
    cache, table, ln = make(kv, [100, 100], 2, 64, 16, "e4m3", "hnd", seed=8)
    q = torch.randn((2, 8, 64), device="cuda")
    side, own = torch.cuda.Stream(), kv.KVWorkspace("cuda")
    torch.cuda.synchronize()
    out = kv.kv_attention(cache, 0, q, table, ln, workspace=own, stream=side)
    side.synchronize()
    close(out, None, attention_ref(cache, 0, q, table, [100, 100], [0, 1, 2], 0.125), 100, torch.float32)
    buf = torch.empty_like(q)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kv.kv_attention(cache, 0, q, table, ln, out=buf, workspace=own)
    for lens in ([3, 100], [64, 0]):
        ln.copy_(i32(lens))
        graph.replay()
        torch.cuda.synchronize()
        close(buf, None, attention_ref(cache, 0, q, table, lens, [0, 1, 2], 0.125), 100, torch.float32)


# ---------------------------------------------------------------- append

def e4m3_round(x):
    """Nearest e4m3 value of a float64 array, ties to even, saturating."""
    with np.errstate(invalid="ignore"):
        e = np.frexp(np.abs(np.where(np.isfinite(x), x, 0.0)))[1] - 1
        step = np.ldexp(1.0, np.maximum(e, -6) - 3)
        y = np.rint(np.clip(x, -1e9, 1e9) / step) * step
        return np.clip(y, -448, 448)


def append_ref(codes, scale, off, x, fmt):
    """One block in float64 with the fp32 roundings of the definition: codes [P, D] (values), x [n, D]."""
    f32 = np.float32
    a = np.abs(np.where(np.isfinite(x), x, 0)).max(initial=0.0)
    if a == 0:
        need = f32(0)
    elif fmt == "int8":
        need = f32(f32(a) / f32(127))
    else:
        e = -126
        while a > 448.0 * 2.0 ** e:
            e += 1
        need = f32(2.0 ** e)
    old = scale if off else f32(0)
    new = max(old, need)
    out = codes.copy()
    if off and new > old:
        f = f32(old / new)
        y = (out[:off].astype(f32) * f).astype(np.float64)
        out[:off] = np.rint(y) if fmt == "int8" else e4m3_round(y)
    for i in range(len(x)):
        with np.errstate(all="ignore"):
            y = (x[i].astype(f32) / new).astype(np.float64) if new > 0 else np.where(np.isfinite(x[i]), 0.0, x[i])
        if fmt == "int8":
            out[off + i] = np.where(np.isnan(y), 0, np.rint(np.clip(y, -127, 127)))
        else:
            out[off + i] = np.where(np.isnan(y), np.nan, e4m3_round(y))
    return out, new


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("order", ["hnd", "nhd"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("lens, rows", [([0], [1]), ([15, 16, 17, 40], [1, 1, 1, 1]), ([0, 5, 31, 64], [70, 0, 33, 1]),
                                        ([47], [16])], ids=str)
def test_append(kv, fmt, order, dtype, lens, rows):
    heads, dim, page = 3, 80, 16
    after = [a + b for a, b in zip(lens, rows)]
    cache, table, _ = make(kv, after, heads, dim, page, fmt, order, seed=sum(after))
    st = starts_of(rows)
    g = torch.Generator(device="cuda").manual_seed(1)
    kvt = torch.randn((st[-1], 2, heads, dim), device="cuda", generator=g) * \
        torch.exp2(torch.randint(-6, 6, (st[-1], 2, heads, 1), device="cuda", generator=g).float())
    kvt = kvt.to(DT[dtype])
    k, v = kvt[:, 0], kvt[:, 1]
    before = [(values(c.clone(), fmt).cpu().numpy(), s.cpu().numpy().copy()) for c, s in
              ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    kv.kv_append(cache, 1, k, v, table, i32(lens), starts=None if all(r == 1 for r in rows) else i32(st))
    for (codes, scale), c, s, x in zip(before, (cache.k, cache.v), (cache.k_scale, cache.v_scale), (k, v)):
        x = x.float().cpu().numpy().astype(np.float64)
        view = codes[1] if order == "hnd" else codes[1].transpose(0, 2, 1, 3)
        for b in range(len(lens)):
            at = lens[b]
            while at < after[b]:
                pid, off = int(table[b, at // page]), at % page
                n = min(page - off, after[b] - at)
                r = st[b] + at - lens[b]
                for h in range(heads):
                    view[pid, h], scale[1, pid, h] = append_ref(view[pid, h], scale[1, pid, h], off, x[r:r + n, h], fmt)
                at += n
        assert np.array_equal(s.cpu().numpy(), scale)
        assert np.array_equal(values(c, fmt).cpu().numpy(), codes)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_append_special_values(kv, fmt):
    """Zeros, infinities, NaN, the smallest and largest magnitudes; blocks of nothing else."""
    rows = [[0.0] * 16, [math.inf, -math.inf, math.nan, 1.0] * 4, [math.nan] * 16, [1e-45] * 15 + [0.0],
            [3.4e38] * 15 + [-1.0], [448.0] * 16, [449.0] + [2.0 ** -9] * 15, [1e-38, 2e-38] * 8, [127.0, 63.5] * 8]
    x = torch.tensor(rows, dtype=torch.float32, device="cuda").view(len(rows), 1, 16)
    cache, table, ln = make(kv, [1] * len(rows), 1, 16, 16, fmt, "hnd", seed=1)
    kv.kv_append(cache, 0, x, x, table, torch.zeros_like(ln))
    for i, r in enumerate(rows):
        pid = int(table[i, 0])
        want, s = append_ref(np.zeros((16, 16)), np.float32(0), 0, np.array([r], np.float32).astype(np.float64), fmt)
        got = values(cache.k[0, pid, 0, 0].contiguous(), fmt).cpu().numpy()
        assert np.float32(cache.k_scale[0, pid, 0].item()) == s, i
        assert np.array_equal(got, want[0], equal_nan=True), i


def test_append_bad_pages_write_nothing(kv):
    cache, table, ln = make(kv, [10, 10], 2, 64, 16, "e4m3", "hnd")
    k0 = cache.k.clone()
    x = torch.randn((2, 2, 64), device="cuda")
    for t, n in ((i32([[-1], [cache.pages]]), i32([3, 4])), (table, i32([16, -1]))):
        kv.kv_append(cache, 0, x, x, t, n)
        assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS
        assert torch.equal(cache.k, k0)


# ---------------------------------------------------------------- pages

def filled(kv, layers, pages, heads, page, dim, seed=0):
    cache = kv.KVCache.allocate(layers, pages, heads, page, dim, "int8", "hnd")
    g = torch.Generator(device="cuda").manual_seed(seed)
    for c in (cache.k, cache.v):
        c.copy_(torch.randint(0, 256, c.shape, device="cuda", generator=g, dtype=torch.uint8))
    for s in (cache.k_scale, cache.v_scale):
        s.copy_(torch.rand(s.shape, device="cuda", generator=g))
    return cache


def state(cache):
    return [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]


def moved(before, src, dst):
    out = [x.clone() for x in before]
    for x, y in zip(out, before):
        for s, d in zip(src, dst):
            x[:, d] = y[:, s]
    return out


def same_state(cache, want):
    return all(torch.equal(a, b) for a, b in zip((cache.k, cache.v, cache.k_scale, cache.v_scale), want))


@pytest.mark.parametrize("heads, page, dim", [(1, 16, 16), (3, 32, 80), (8, 128, 128)])
def test_copy_pages(kv, heads, page, dim):
    cache = filled(kv, 3, 20, heads, page, dim)
    was = state(cache)
    src, dst = [5, 5, 19, 0], [1, 2, 3, 18]
    kv.kv_copy_pages(cache, i32(src), i32(dst), count=i32([3]))
    assert same_state(cache, moved(was, src[:3], dst[:3]))
    kv.kv_copy_pages(cache, i32(src), i32(dst))
    assert same_state(cache, moved(was, src, dst))
    kv.kv_copy_pages(cache, i32([3, 4]), i32([20, -1]))
    assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS
    assert same_state(cache, moved(was, src, dst))


def fork_ref(table, lens, parent, refs, page):
    table2 = np.full((len(parent), table.shape[1]), -1, np.int32)
    refs2 = refs.copy()
    need = [(n + page - 1) // page for n in lens]
    for b in range(len(lens)):
        for j in range(need[b]):
            refs2[table[b, j]] -= 1
    for i, p in enumerate(parent):
        table2[i, :need[p]] = table[p, :need[p]]
        for j in range(need[p]):
            refs2[table[p, j]] += 1
    lens2 = np.array([lens[p] for p in parent], np.int32)
    tails = [int(table2[i, lens2[i] // page]) if lens2[i] % page else -1 for i in range(len(parent))]
    pairs, missing = [], 0
    start = refs2.copy()
    free = [p for p in range(len(refs)) if refs2[p] == 0]
    for i, t in enumerate(tails):
        if t < 0:
            continue
        outside = start[t] > tails.count(t)
        if outside or t in tails[:i]:
            refs2[t] -= 1
            if free:
                d = free.pop(0)
                refs2[d] = 1
                pairs.append((t, d))
            else:
                d, missing = -1, missing + 1
            table2[i, lens2[i] // page] = d
    return table2, lens2, refs2, pairs, missing


def counts(table, lens, page, pages):
    refs = np.zeros(pages, np.int32)
    for b, n in enumerate(lens):
        for j in range((n + page - 1) // page):
            refs[table[b, j]] += 1
    return refs


@pytest.mark.parametrize("lens, parent", [
    ([1], [0, 0, 0]), ([32], [0, 0]), ([33, 7, 64, 0], [1, 1, 3, 0, 0, 2]), ([10, 20, 30], [2, 2, 2]), ([50], [0]),
    ([5, 6], [1]), ([0, 0], [1, 0, 0]),
], ids=str)
@pytest.mark.parametrize("outside", [False, True])
def test_fork(kv, ws, lens, parent, outside):
    page, pages = 16, 40
    cache = filled(kv, 2, pages, 2, page, 64)
    perm = np.random.default_rng(3).permutation(pages)
    table = np.full((len(lens), 6), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        need = (n + page - 1) // page
        table[b, :need] = perm[at:at + need]
        at += need
    refs = counts(table, lens, page, pages)
    if outside:  # a sequence of another table holds every page too
        refs[refs > 0] += 1
    want = fork_ref(table, lens, parent, refs, page)
    was = state(cache)
    t2, l2, r2 = kv.kv_fork(cache, i32(table.tolist()), i32(lens), i32(parent), i32(refs.tolist()), workspace=ws)
    assert np.array_equal(t2.cpu().numpy(), want[0])
    assert np.array_equal(l2.cpu().numpy(), want[1])
    assert np.array_equal(r2.cpu().numpy(), want[2])
    assert same_state(cache, moved(was, [s for s, _ in want[3]], [d for _, d in want[3]]))


@pytest.mark.parametrize("pages", [4097, 9000, 17001])
def test_fork_many(kv, ws, pages):
    """Two generations over several counting chunks; the free pages lie far apart."""
    page = 16
    rng = np.random.default_rng(pages)
    cache = filled(kv, 1, pages, 1, page, 16)
    lens = [int(x) for x in rng.integers(0, 200, 300)]
    perm = rng.permutation(pages)
    table = np.full((300, 13), -1, np.int32)
    at = 0
    for b, n in enumerate(lens):
        need = (n + page - 1) // page
        table[b, :need] = perm[at:at + need]
        at += need
    refs = counts(table, lens, page, pages)
    refs[np.setdiff1d(np.arange(pages), perm[:at])[:-150]] = 1  # all but 150 of the others are held elsewhere
    t, l, r = i32(table.tolist()), i32(lens), i32(refs.tolist())
    for gen in range(2):
        parent = [int(x) for x in rng.integers(0, len(lens), 300)]
        want = fork_ref(table, lens, parent, refs, page)
        assert want[4] == 0
        was = state(cache)
        t, l, r = kv.kv_fork(cache, t, l, i32(parent), r, workspace=ws)
        table, lens, refs = want[0], [int(x) for x in want[1]], want[2]
        assert np.array_equal(t.cpu().numpy(), table) and np.array_equal(r.cpu().numpy(), refs)
        assert same_state(cache, moved(was, [s for s, _ in want[3]], [d for _, d in want[3]]))


def test_fork_without_free_pages(kv, ws):
    page, pages = 16, 3
    cache = filled(kv, 1, pages, 1, page, 16)
    table = np.array([[0, 1], [2, -1]], np.int32)
    lens = [20, 3]
    refs = counts(table, lens, page, pages)
    want = fork_ref(table, lens, [0, 0, 0, 1], refs, page)
    assert want[4] == 2
    t2, l2, r2 = kv.kv_fork(cache, i32(table.tolist()), i32(lens), i32([0, 0, 0, 1]), i32(refs.tolist()), workspace=ws)
    assert qgemv.qg_device_status() == qgemv.QG_EPAGES
    assert np.array_equal(t2.cpu().numpy(), want[0]) and np.array_equal(r2.cpu().numpy(), want[2])
    kv.kv_fork(cache, i32(table.tolist()), i32(lens), i32([0, 2, -1]), i32(refs.tolist()), workspace=ws)  # no such parent
    assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS


def compact_ref(table, lens, drop, refs, page):
    refs = refs.copy()
    table = table.copy()
    lens = list(lens)
    for b in range(len(lens)):
        need = (lens[b] + page - 1) // page
        if drop[b]:
            for j in range(need):
                refs[table[b, j]] -= 1
            lens[b], need = 0, 0
        table[b, need:] = -1
    n = int((refs > 0).sum())
    src = [p for p in range(n, len(refs)) if refs[p] > 0]
    dst = [p for p in range(n) if refs[p] <= 0]
    to = np.arange(len(refs))
    to[src] = dst
    refs2 = np.zeros_like(refs)
    for p in range(len(refs)):
        if refs[p] > 0:
            refs2[to[p]] = refs[p]
    return np.where(table >= 0, to[table], -1), np.array(lens), refs2, n, src, dst


@pytest.mark.parametrize("pages", [5, 64, 4096, 4100, 12289, 20483])
@pytest.mark.parametrize("share", [0.0, 0.5, 1.0])
def test_compact(kv, ws, pages, share):
    page = 16
    rng = np.random.default_rng(pages)
    cache = filled(kv, 2, pages, 1, page, 16)
    batch = min(200, max(2, pages // 8))
    lens, table, at = [], np.full((batch, 30), -1, np.int32), 0
    perm = rng.permutation(pages)
    for b in range(batch):
        need = int(rng.integers(0, 31))
        need = min(need, pages - at)
        table[b, :need] = perm[at:at + need]
        lens.append(max(0, need * page - int(rng.integers(0, page))))
        at += need
    refs = counts(table, lens, page, pages)
    drop = rng.random(batch) < share
    want = compact_ref(table, lens, drop, refs, page)
    was = state(cache)
    d = None if share == 0 else torch.from_numpy(drop).cuda()
    t2, l2, r2, n = kv.kv_compact(cache, i32(table.tolist()), i32(lens), i32(refs.tolist()), drop=d, workspace=ws)
    assert int(n) == want[3]
    assert np.array_equal(t2.cpu().numpy(), want[0]) and np.array_equal(l2.cpu().numpy(), want[1])
    assert np.array_equal(r2.cpu().numpy(), want[2])
    assert same_state(cache, moved(was, want[4], want[5]))


@pytest.mark.parametrize("pages", [30, 4200])
def test_reserve_and_free(kv, ws, pages):
    page = 16
    cache = filled(kv, 1, pages, 1, page, 16)
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[1::3] = 1
    refs[:pages - 28] = 1
    table, lens = i32([[-1] * 5] * 4), i32([0, 0, 0, 0])
    held = []
    for add in ([0, 1, 16, 17], [1, 15, 1, 15], [16, 1, 0, 16]):
        want_refs = refs.cpu().numpy()
        free = [p for p in range(pages) if want_refs[p] == 0]
        want = table.cpu().numpy()
        for b in range(4):
            n = int(lens[b])
            for j in range((n + page - 1) // page, (n + add[b] + page - 1) // page):
                want[b, j] = free.pop(0)
                want_refs[want[b, j]] = 1
        kv.kv_reserve(cache, table, lens, refs, add=i32(add), workspace=ws)
        assert np.array_equal(table.cpu().numpy(), want) and np.array_equal(refs.cpu().numpy(), want_refs)
        lens += i32(add)
        held.append(table.clone())
    kv.kv_reserve(cache, table, lens, refs, workspace=ws)  # one token each
    before = refs.clone()
    drop = torch.tensor([True, False, False, True], device="cuda")
    ids = torch.cat([table[0, :(int(lens[0]) + 15) // page], table[3, :(int(lens[3]) + 15) // page]]).long()
    kv.kv_free(cache, table, lens, refs, drop=drop)
    before[ids] -= 1
    assert torch.equal(refs, before)
    assert lens.tolist()[0] == 0 and lens.tolist()[3] == 0 and (table[0] == -1).all() and (table[1, 0] >= 0)


def test_reserve_short(kv, ws):
    """Too few pages: sequences in order, one that does not fit gets none."""
    cache = filled(kv, 1, 6, 1, 16, 16)
    refs = torch.zeros(6, dtype=torch.int32, device="cuda")
    refs[2] = 1
    table, lens = i32([[-1] * 8] * 3), i32([0, 0, 0])
    kv.kv_reserve(cache, table, lens, refs, add=i32([32, 70, 48]), workspace=ws)
    assert qgemv.qg_device_status() == qgemv.QG_EPAGES
    assert table[:, :4].tolist() == [[0, 1, -1, -1], [-1] * 4, [3, 4, 5, -1]]
    assert refs.tolist() == [1] * 6
    kv.kv_reserve(cache, table, i32([32, 0, 120]), refs, add=i32([0, 0, 9]), workspace=ws)  # past the table
    assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS


# ---------------------------------------------------------------- beam selection

def beam_ref(x, cum, keep):
    """Scores in 64 bits, (score, flat index) order."""
    requests, beams = cum.shape
    x = x.double().cpu().numpy()
    c = cum.double().cpu().numpy().reshape(-1)
    vocab = x.shape[1]
    score = np.full(x.shape, -np.inf)
    for r in range(len(x)):
        m = x[r].max()
        if np.isfinite(m) and not np.isnan(x[r]).any() and c[r] < np.inf:
            score[r] = c[r] + (x[r] - (m + np.log(np.exp(x[r] - m).sum())))
    score = score.reshape(requests, beams * vocab)
    order = np.argsort(-score, axis=1, kind="stable")[:, :keep]
    rows = np.arange(requests)[:, None] * beams
    return np.take_along_axis(score, order, 1), order % vocab, rows + order // vocab


def check_beam(kv, ws, x, cum, keep):
    s, t, p = kv.beam_select(x, cum, keep, workspace=ws)
    ws_, wt, wp = beam_ref(x, cum, keep)
    assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(p.cpu().numpy(), wp)
    got = s.double().cpu().numpy()
    fin = np.isfinite(ws_)
    assert np.array_equal(fin, np.isfinite(got))
    # lse in fp32 parts (2^-21 relative of the sum, so absolute in the log) and the score's own rounding
    assert (np.abs(got - ws_)[fin] <= 2.0 ** -20 + np.abs(ws_[fin]) * 2.0 ** -24).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("requests, beams, vocab, keep", [
    (1, 1, 1, 1), (1, 1, 5, 5), (2, 3, 7, 21), (1, 4, 32000, 8), (5, 2, 2047, 4), (3, 8, 2049, 16), (2, 1, 50001, 128),
    (1, 64, 3001, 128), (40, 4, 12345, 8),
])
def test_beam(kv, ws, dtype, requests, beams, vocab, keep):
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = (torch.randn((requests * beams, vocab), device="cuda", generator=g) * 3).to(DT[dtype])
    cum = -torch.rand((requests, beams), device="cuda", generator=g) * 3
    check_beam(kv, ws, x, cum, keep)


@pytest.mark.parametrize("vocab", [700, 32001])
def test_beam_ties_and_orders(kv, ws, vocab):
    """Equal logits everywhere, identical beams, rising and falling rows: of equal scores the lowest index."""
    x = torch.zeros((4, vocab), device="cuda")
    check_beam(kv, ws, x, torch.zeros((1, 4), device="cuda"), 16)
    up = torch.arange(vocab, device="cuda").float() * 1e-3
    for row in (up, up.flip(0), torch.round(up)):
        check_beam(kv, ws, torch.stack([row, row, row, row]), torch.zeros((2, 2), device="cuda"), 128)


def test_beam_masked_and_bad_rows(kv, ws):
    vocab = 5000
    x = torch.randn((8, vocab), device="cuda")
    x[0, :] = -math.inf                      # nothing but masked tokens
    x[1, 7:] = -math.inf                     # fewer tokens than are kept
    x[2, 100] = math.nan
    x[3, 4000] = math.inf
    x[4, 5:] = torch.finfo(torch.float32).min
    cum = torch.tensor([[0.0, -1.0, -2.0, -3.0, -4.0, -math.inf, math.nan, math.inf]], device="cuda")
    check_beam(kv, ws, x, cum, 24)
    check_beam(kv, ws, x[:1].contiguous(), cum[:, :1].contiguous(), 24)
    check_beam(kv, ws, x[2:4].contiguous(), cum[:, :2].contiguous(), 128)


def test_beam_strided_rows(kv, ws):
    big = torch.randn((6, 3, 1003), device="cuda")
    x = big[:, 1]
    check_beam(kv, ws, x, torch.zeros((3, 2), device="cuda"), 6)
    h = torch.randn((6, 1003), device="cuda").half()[:, 1:]  # rows that start off any 16-byte boundary
    s, t, p = kv.beam_select(h, torch.zeros((3, 2), device="cuda"), 6, workspace=ws)
    wt = beam_ref(h, torch.zeros((3, 2)), 6)[1]
    assert np.array_equal(t.cpu().numpy(), wt)


# ---------------------------------------------------------------- refusals of the binding

def test_binding_refusals(kv, ws):
    cache, table, lens = make(kv, [20], 2, 64, 16, "e4m3", "hnd")
    q = torch.randn((1, 4, 64), device="cuda")
    with pytest.raises(TypeError):
        kv.kv_attention(cache, 0, q.double(), table, lens, workspace=ws)
    with pytest.raises(TypeError):
        kv.kv_attention(cache, 0, q, table.long(), lens, workspace=ws)
    with pytest.raises(ValueError):
        kv.kv_attention(cache, 0, q[..., :32], table, lens, workspace=ws)
    with pytest.raises(ValueError):
        kv.kv_attention(cache, 0, q, table, torch.cat([lens, lens]), workspace=ws)
    with pytest.raises(qgemv.QGError) as e:
        kv.kv_attention(cache, 5, q, table, lens, workspace=ws)
    assert e.value.code == qgemv.QG_EINVAL
    with pytest.raises(qgemv.QGError) as e:
        kv.kv_attention(cache, 0, q[:, :3], table, lens, workspace=ws)
    assert e.value.code == qgemv.QG_EINVAL
    with pytest.raises(ValueError):
        kv.kv_append(cache, 0, q[:, :2], q[:, ::2], table, lens)
    with pytest.raises(ValueError):
        kv.KVCache(cache.k[..., ::2], cache.k_scale, cache.v[..., ::2], cache.v_scale)
    with pytest.raises(ValueError):
        kv.KVCache.allocate(1, 1, 1, 16, 64, fmt="e5m2")
    with pytest.raises(ValueError):
        kv.beam_select(torch.zeros((3, 8), device="cuda"), torch.zeros((1, 2), device="cuda"), 2, workspace=ws)
