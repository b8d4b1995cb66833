"""GPU tests of kv_append_rotary against a plain implementation in 64 bits that
rounds to fp32 where the definition does.

A product of two fp32 values is exact in 64 bits, and the sum of two fp32 values
rounded to 64 bits (2 * 24 + 2 <= 53) rounds to fp32 as the exact sum does: the
turned values are known bit for bit, and codes, scales and queries are compared so.
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_quantised_weight_gb300 import qgemv  # noqa: E402
from test_kv_gpu import DT, append_ref, i32, kv, make, starts_of, status_clean, values  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def turned(x, rope, pos, pairs):
    """x [rows, heads, dim] (fp32 values) at positions pos, each product and sum rounded to fp32."""
    half = rope.shape[1] // 2
    t = rope.double()[pos]
    c, s = t[:, None, :half], t[:, None, half:]
    x = x.double()
    a, b = (x[..., 0:2 * half:2], x[..., 1:2 * half:2]) if pairs == "interleaved" else (x[..., :half], x[..., half:2 * half])
    r = lambda y: y.float().double()  # noqa: E731
    lo, hi = r(r(a * c) - r(b * s)), r(r(a * s) + r(b * c))
    out = x.clone()
    if pairs == "interleaved":
        out[..., 0:2 * half:2], out[..., 1:2 * half:2] = lo, hi
    else:
        out[..., :half], out[..., half:2 * half] = lo, hi
    return out


def appended(cache, before, name, layer, x, table, lens, rows):
    """Codes and scales of the cache behind an append of x (float64, [rows, heads, dim])."""
    codes, scale = before[name]
    view = codes[layer] if cache.order == "hnd" else codes[layer].transpose(0, 2, 1, 3)
    page, st = cache.page_tokens, starts_of(rows)
    for b, n in enumerate(lens):
        at = n
        while at < n + rows[b]:
            pid, off = int(table[b, at // page]), at % page
            take = min(page - off, n + rows[b] - at)
            r = st[b] + at - n
            for h in range(cache.heads):
                view[pid, h], scale[layer, pid, h] = append_ref(view[pid, h], scale[layer, pid, h], off, x[r:r + take, h], cache.fmt)
            at += take
    return codes, scale


def snapshot(cache):
    return {n: (values(c.clone(), cache.fmt).cpu().numpy(), s.cpu().numpy().copy())
            for n, c, s in (("k", cache.k, cache.k_scale), ("v", cache.v, cache.v_scale))}


def parts(rows, q_heads, heads, dim, dtype, seed=1):
    """q, k, v as strided parts of one tensor."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, q_heads + 2 * heads, dim), device="cuda", generator=g)
    x *= torch.exp2(torch.randint(-4, 5, (rows, q_heads + 2 * heads, 1), device="cuda", generator=g).float())
    x = x.to(DT[dtype])
    return x[:, :q_heads], x[:, q_heads:q_heads + heads], x[:, q_heads + heads:]


def check(kv, lens, rows, q_heads, heads, dim, part, page, fmt, order, dtype, pairs, seed=0):  # noqa: F811
    after = [a + b for a, b in zip(lens, rows)]
    cache, table, _ = make(kv, after, heads, dim, page, fmt, order, seed=seed)
    st = starts_of(rows)
    q, k, v = parts(st[-1], q_heads, heads, dim, dtype, seed + 1)
    rope = kv.rotary_table(max(after) + 1, part, base=500.0)
    pos = torch.cat([torch.arange(n, n + r) for n, r in zip(lens, rows)]).cuda()
    before = snapshot(cache)
    out = kv.kv_append_rotary(cache, 1, q, k, v, rope, table, i32(lens), pairs=pairs,
                              starts=None if all(r == 1 for r in rows) else i32(st))
    assert out.dtype == q.dtype and out.is_contiguous()
    assert torch.equal(out, turned(q, rope, pos, pairs).to(q.dtype))
    for name, x, c, s in (("k", turned(k, rope, pos, pairs), cache.k, cache.k_scale), ("v", v.double(), cache.v, cache.v_scale)):
        codes, scale = appended(cache, before, name, 1, x.cpu().numpy(), table, lens, rows)
        assert np.array_equal(s.cpu().numpy(), scale), name
        assert np.array_equal(values(c, fmt).cpu().numpy(), codes), name


@pytest.mark.parametrize("pairs", ["interleaved", "halves"])
@pytest.mark.parametrize("dtype, fmt, order", [("f32", "e4m3", "hnd"), ("bf16", "int8", "nhd"), ("f16", "e4m3", "nhd"),
                                               ("f32", "int8", "nhd"), ("bf16", "e4m3", "hnd")])
@pytest.mark.parametrize("lens, rows", [([0], [1]), ([15, 16, 17, 40], [1, 1, 1, 1]), ([0, 5, 31, 64], [70, 0, 33, 1]),
                                        ([47], [16])], ids=str)
def test_append_rotary(kv, pairs, dtype, fmt, order, lens, rows):  # noqa: F811
    check(kv, lens, rows, 6, 3, 80, 80, 16, fmt, order, dtype, pairs, seed=sum(lens))


@pytest.mark.parametrize("pairs", ["interleaved", "halves"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim, part", [(16, 16), (64, 16), (64, 48), (96, 32), (128, 128), (256, 256), (256, 64)])
def test_append_rotary_dims(kv, pairs, dtype, dim, part):  # noqa: F811
    check(kv, [3, 30], [1, 1], 9, 1, dim, part, 16, "e4m3", "hnd", dtype, pairs, seed=dim)
    check(kv, [3, 30], [40, 2], 5, 1, dim, part, 32, "int8", "hnd", dtype, pairs, seed=part)


@pytest.mark.parametrize("page, dim", [(16, 64), (64, 128), (128, 128), (128, 256), (256, 96), (256, 256)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_append_rotary_blocks_of_all_sizes(kv, page, dim, dtype):  # noqa: F811
    """Blocks whose values a thread holds, and those that are read twice."""
    check(kv, [page // 2, page], [page + 3, 2 * page], 2, 2, dim, dim, page, "e4m3", "nhd", dtype, "halves", seed=page)


@pytest.mark.parametrize("q_heads", [1, 7, 8, 17, 64])
def test_append_rotary_query_heads(kv, q_heads):  # noqa: F811
    check(kv, [5], [1], q_heads, 1, 128, 128, 16, "e4m3", "hnd", "bf16", "halves")
    check(kv, [5, 0], [3, 20], q_heads, 1, 64, 64, 16, "e4m3", "hnd", "f32", "interleaved")


@pytest.mark.parametrize("q_heads", [7, 17, 40])
@pytest.mark.parametrize("dtype, dim, part", [("bf16", 128, 128), ("f32", 64, 48), ("f16", 96, 32)])
def test_append_rotary_query_heads_of_many_tokens(kv, q_heads, dtype, dim, part):  # noqa: F811
    """Blocks on both sides of a CTA for each SM at 2, 4, 8 and 16 heads a CTA, the last of them with fewer heads; more
    heads than a thread has on their way at once."""
    for n in (20, 40, 170):
        check(kv, [3 + i % 40 for i in range(n)], [1] * n, q_heads, 1, dim, part, 16, "e4m3", "hnd", dtype, "halves", seed=n)
    for n in (7, 18, 90):
        check(kv, [3 + i % 40 for i in range(n)], [2 + i % 19 for i in range(n)], q_heads, 1, dim, part, 16, "int8", "nhd", dtype,
              "interleaved", seed=n)


@pytest.mark.parametrize("rows", [1, 3])
@pytest.mark.parametrize("q_heads", [17, 40])
def test_append_rotary_of_many_tokens_in_place(kv, q_heads, rows):  # noqa: F811
    n = 170
    lens, st = [i % 50 for i in range(n)], [rows * i for i in range(n + 1)]
    cache, table, _ = make(kv, [x + rows for x in lens], 1, 128, 16, "e4m3", "hnd")
    q, k, v = parts(st[-1], q_heads, 1, 128, "bf16")
    q, rope = q.contiguous(), kv.rotary_table(64, 128)
    pos = torch.cat([torch.arange(x, x + rows) for x in lens]).cuda()
    want = turned(q, rope, pos, "halves").to(q.dtype)
    starts = None if rows == 1 else i32(st)
    assert kv.kv_append_rotary(cache, 0, q, k, v, rope, table, i32(lens), starts=starts, pairs="halves", out=q) is q
    assert torch.equal(q, want)


def test_append_rotary_of_many_sequences(kv):  # noqa: F811
    g = np.random.default_rng(3)
    rows = [int(x) for x in g.integers(0, 40, 75) * (g.random(75) < 0.6)]
    check(kv, [int(x) for x in g.integers(0, 60, 75)], rows, 2, 1, 64, 64, 16, "int8", "hnd", "bf16", "halves")


def test_append_rotary_without_queries_and_in_place(kv):  # noqa: F811
    cache, table, _ = make(kv, [20, 9], 2, 64, 16, "e4m3", "hnd")
    q, k, v = parts(2, 4, 2, 64, "f32")
    rope = kv.rotary_table(32, 64)
    args = (rope, table, i32([19, 8]))
    want = kv.kv_append_rotary(cache, 0, q, k, v, *args)
    held = [x.clone() for x in (cache.k, cache.k_scale, cache.v, cache.v_scale)]
    assert kv.kv_append_rotary(cache, 0, None, k, v, *args) is None
    same = q.contiguous()
    assert kv.kv_append_rotary(cache, 0, same, k, v, *args, out=same) is same
    assert torch.equal(same, want)
    for a, b in zip(held, (cache.k, cache.k_scale, cache.v, cache.v_scale)):
        assert torch.equal(a, b)


def test_append_rotary_rows_of_no_sequence_are_left(kv):  # noqa: F811
    cache, table, _ = make(kv, [9, 9], 2, 64, 16, "e4m3", "hnd")
    q, k, v = parts(7, 4, 2, 64, "bf16")
    out = torch.full((7, 4, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    kv.kv_append_rotary(cache, 0, q, k, v, kv.rotary_table(32, 64), table, i32([4, 4]), starts=i32([0, 2, 4]), out=out)
    assert (out[4:] == 5.0).all() and not (out[:4] == 5.0).all()


def test_append_rotary_special_values(kv):  # noqa: F811
    """Infinities and NaN turn by IEEE (an infinity times a sine of 0 is NaN); they do not reach the scale."""
    rows = [[math.inf, 1.0] * 8, [math.nan, 2.0] * 8, [0.0] * 16, [3.4e38, 3.4e38] * 8, [1e-45, 0.0] * 8, [-math.inf] * 16]
    for first in (0, 3):
        x = torch.tensor(rows, dtype=torch.float32, device="cuda").view(len(rows), 1, 16)
        cache, table, ln = make(kv, [first + 1] * len(rows), 1, 16, 16, "e4m3", "hnd", seed=1)
        cache.k_scale.zero_()
        rope = kv.rotary_table(8, 16)
        pos = torch.full((len(rows),), first, device="cuda")
        before = snapshot(cache)
        out = kv.kv_append_rotary(cache, 0, x, x, x, rope, table, ln - 1)
        want = turned(x, rope, pos, "interleaved")
        assert torch.equal(torch.nan_to_num(out, nan=7.0), torch.nan_to_num(want.float(), nan=7.0))
        codes, scale = appended(cache, before, "k", 0, want.cpu().numpy(), table, [first] * len(rows), [1] * len(rows))
        ids = table[:, 0].tolist()
        assert np.array_equal(cache.k_scale[0, ids].cpu().numpy(), scale[0, ids])
        assert np.array_equal(values(cache.k, "e4m3").cpu().numpy()[0, ids, 0, first], codes[0, ids, 0, first], equal_nan=True)


def test_append_rotary_positions_beyond_the_table(kv):  # noqa: F811
    cache, table, _ = make(kv, [40, 40, 40], 2, 64, 16, "e4m3", "hnd")
    q, k, v = parts(9, 4, 2, 64, "f32")
    held = cache.k.clone(), cache.v.clone()
    rope = kv.rotary_table(12, 32)
    # positions 10 .. 12 (the last has none), 30 .. 32 (none), length -1 (none)
    out = kv.kv_append_rotary(cache, 0, q, k, v, rope, table, i32([10, 30, -1]), starts=i32([0, 3, 6, 9]))
    assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS
    nan = torch.isnan(out)
    assert not nan[:2].any() and nan[2:, :, :32].all() and not nan[:, :, 32:].any()
    assert torch.equal(out[:, :, 32:], q[:, :, 32:])
    for c, was in zip((cache.k, cache.v), held):
        differ = (c != was).nonzero()
        assert {int(p) for p in differ[:, 1]} == {int(table[0, 0])} and {int(t) for t in differ[:, 3]} <= {10, 11} | set(range(10))


def test_append_rotary_bad_pages_write_nothing(kv):  # noqa: F811
    cache, table, _ = make(kv, [10, 10], 2, 64, 16, "e4m3", "hnd")
    q, k, v = parts(2, 2, 2, 64, "f32")
    was, rope = cache.k.clone(), kv.rotary_table(64, 64)
    for t, n in ((i32([[-1], [cache.pages]]), i32([3, 4])), (table, i32([16, -1]))):
        kv.kv_append_rotary(cache, 0, q, k, v, rope, t, n)
        assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS
        assert torch.equal(cache.k, was)


def test_append_rotary_in_a_graph_and_on_a_stream(kv):  # noqa: F811
    """One captured call replayed with other lengths and values."""
    lens = i32([3, 20])
    cache, table, _ = make(kv, [60, 60], 2, 64, 16, "e4m3", "hnd")
    other, _, _ = make(kv, [60, 60], 2, 64, 16, "e4m3", "hnd")
    q, k, v = (x.contiguous() for x in parts(5, 4, 2, 64, "bf16"))
    starts, rope, side = i32([0, 2, 5]), kv.rotary_table(80, 64), torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    kv.kv_append_rotary(cache, 0, q, k, v, rope, table, lens, starts=starts)
    for a, b in zip((other.k, other.v, other.k_scale, other.v_scale), (cache.k, cache.v, cache.k_scale, cache.v_scale)):
        a.copy_(b)
    with torch.cuda.graph(graph):
        out = kv.kv_append_rotary(cache, 0, q, k, v, rope, table, lens, starts=starts)
    for i in range(3):
        lens += i32([7, 4])
        q.normal_(), k.normal_(), v.normal_()
        graph.replay()
        side.wait_stream(torch.cuda.current_stream())
        want = kv.kv_append_rotary(other, 0, q, k, v, rope, table, lens, starts=starts, stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(out, want)
        for a, b in zip((other.k, other.v, other.k_scale, other.v_scale), (cache.k, cache.v, cache.k_scale, cache.v_scale)):
            assert torch.equal(a, b)


def test_rotary_table(kv):  # noqa: F811
    t = kv.rotary_table(1000, 64, base=10000.0)
    angle = np.arange(1000)[:, None] * 10000.0 ** (-np.arange(32) / 32)
    want = np.concatenate([np.cos(angle), np.sin(angle)], 1)
    assert t.shape == (1000, 64) and t.dtype == torch.float32
    # half a step of fp32, and the 64-bit angle's own last bits
    assert np.abs(t.double().cpu().numpy() - want).max() <= 2.0 ** -25 + 1000 * 2.0 ** -52
