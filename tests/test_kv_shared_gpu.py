"""GPU tests of kv_share and kv_attention_shared against a plain implementation in 64
bits that knows nothing of the sharing.

Tolerance: test_kv_gpu's, which counts (16 + L / 64) 2^-22 of A for sums of L / 64
steps and their joins.  The prefix's parts and the tokens behind it are joined once
more, each weight by an exponential (2^-22), two products, a sum and a quotient
(2^-24 each): 2 * 2^-22, which 512 tokens more in L cover.  What the prefix stores of a
row's largest weight W is 2^4 at least (2^6 less the next whole orders of score and
scale), half of f16's smallest step 2^-25: weights of bf16 queries are cut at 2^-29 W,
2^9 times what test_kv_gpu counts (two parts: 2^-40 W).
"""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_quantised_weight_gb300 import qgemv  # noqa: E402
from test_kv_gpu import DT, attention_ref, close, i32, kv, make, starts_of, status_clean, ws  # noqa: E402, F401

pytestmark = pytest.mark.gpu


LEAST = 16 << 20  # bytes of pages that a table has to have room for, beyond one sequence's, to be shared


def least_width(batch, heads, dim, page):
    return -(-LEAST // (2 * (batch - 1) * heads * dim * page))


MEMBERS = 4        # sequences that a batch has to have for each group


def shared_table(kv, shape, heads, dim, page, fmt, order, seed=0, layers=2, wide=True):  # noqa: F811
    """shape: for each group (tokens of the prefix, tokens of each sequence behind it).  Whole pages of a prefix are the
    first sequence's.  wide: the table has columns enough for its pages to be shared, however few are held, and sequences
    of five tokens and no group behind the others, as many as the groups are too small by.  Returns
    cache, table, lens (list), borders of the groups."""
    lens = [p + t for p, tails in shape for t in tails]
    lens += [5] * max(0, MEMBERS * len(shape) - len(lens)) if wide else []
    width = max(*(-(-n // page) for n in lens), least_width(len(lens), heads, dim, page)) if wide else None
    cache, table, _ = make(kv, lens, heads, dim, page, fmt, order, seed=seed, layers=layers, width=width)
    ids, at, borders = table.cpu().numpy(), 0, [0]
    for p, tails in shape:
        for i in range(len(tails)):
            ids[at + i, :p // page] = ids[at, :p // page]
        at += len(tails)
        borders.append(at)
    return cache, i32(ids.tolist()), lens, borders


def small(ref, dtype):
    """test_kv_gpu's reference with the prefix's cut of small weights."""
    return (*ref[:4], ref[4] * 2.0 ** 9) if dtype == "bf16" else ref


def plan_ref(ids, lens, starts, borders, page, pages):
    """The plan by its definition, one column after the other."""
    head, skip = [], [0] * len(lens)
    for g0, g1 in zip(borders, borders[1:]):
        busy = [b for b in range(g0, g1) if starts[b + 1] > starts[b]]
        tokens = 0
        if len(busy) > 1:
            most = min(max(0, lens[b] - (starts[b + 1] - starts[b]) + 1) for b in busy) // page
            while tokens < most and len({ids[b][tokens] for b in busy}) == 1 and 0 <= ids[busy[0]][tokens] < pages:
                tokens += 1
        head += [starts[g0], starts[g1] - starts[g0], tokens * page, busy[0] if busy else g0]
        for b in busy:
            skip[b] = tokens * page
    return head + skip


def check(kv, ws, shape, group, heads, dim, page, fmt, order, dtype, rows=None, seed=0, scale=None, out=False):  # noqa: F811
    cache, table, lens, borders = shared_table(kv, shape, heads, dim, page, fmt, order, seed)
    rows = [1] * len(lens) if rows is None else rows + [1] * (len(lens) - len(rows))
    st = starts_of(rows)
    starts = None if all(r == 1 for r in rows) else i32(st)
    g = torch.Generator(device="cuda").manual_seed(seed + 1)
    q = torch.randn((st[-1], group * heads, dim), device="cuda", generator=g).to(DT[dtype])
    plan = kv.kv_share(cache, table, i32(lens), i32(borders), starts=starts)
    assert plan.tolist() == plan_ref(table.tolist(), lens, st, borders, page, cache.pages)
    got, lse = kv.kv_attention_shared(cache, 1, q, table, i32(lens), plan, starts=starts, scale=scale, return_lse=True, workspace=ws)
    ref = attention_ref(cache, 1, q, table, lens, st, 1 / math.sqrt(dim) if scale is None else scale)
    close(got, lse, small(ref, dtype), max(lens) + 512, DT[dtype], one_part=dtype == "bf16")
    return cache, table, lens, borders, q, plan, got, lse


@pytest.mark.parametrize("fmt, order", [("e4m3", "hnd"), ("int8", "nhd")])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shape", [[(16, [1, 1])], [(15, [3, 4])], [(100, [1, 30, 17])], [(1000, [5] * 7)],
                                   [(129, [1, 2]), (0, [9, 9]), (64, [40])], [(2000, [300, 1, 77, 16])]], ids=str)
def test_shared(kv, ws, shape, fmt, order, dtype):  # noqa: F811
    check(kv, ws, shape, 4, 2, 64, 16, fmt, order, dtype, seed=len(shape))


@pytest.mark.parametrize("dtype, fmt", [("f32", "int8"), ("f16", "e4m3"), ("bf16", "e4m3"), ("bf16", "int8")])
@pytest.mark.parametrize("dim", [16, 48, 64, 80, 128, 144, 256])
@pytest.mark.parametrize("group", [1, 3, 8, 17])
def test_shared_heads_and_dims(kv, ws, dim, group, dtype, fmt):  # noqa: F811
    check(kv, ws, [(300, [20, 1, 45, 9, 33]), (150, [3, 70])], group, 2, dim, 16, fmt, "hnd", dtype, seed=dim + group)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("order", ["hnd", "nhd"])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_pages(kv, ws, page, order, dtype):  # noqa: F811
    check(kv, ws, [(700, [1, 20, 300]), (513, [2, 2])], 4, 3, 128, page, "e4m3", order, dtype, seed=page)


@pytest.mark.parametrize("members", [2, 8, 15, 33, 70])
@pytest.mark.parametrize("dtype, dim", [("bf16", 128), ("f32", 64), ("f16", 128), ("bf16", 256), ("f32", 128), ("f16", 64)])
def test_shared_by_many(kv, ws, members, dtype, dim):  # noqa: F811
    """Row counts on both sides of each block of query rows."""
    check(kv, ws, [(900, [1 + 7 * i % 50 for i in range(members)])], 4, 2, dim, 32, "e4m3", "hnd", dtype, seed=members)


@pytest.mark.parametrize("members, groups", [(2, 40), (5, 9), (64, 3)])
def test_shared_by_many_groups(kv, ws, members, groups):  # noqa: F811
    g = np.random.default_rng(groups)
    shape = [(int(g.integers(0, 500)), [int(x) for x in g.integers(1, 90, members)]) for _ in range(groups)]
    check(kv, ws, shape, 4, 1, 64, 16, "int8", "hnd", "bf16", seed=members)
    check(kv, ws, shape, 2, 2, 128, 16, "e4m3", "nhd", "f32", seed=members)


@pytest.mark.parametrize("prefix, members, heads", [(40000, 3, 1), (9001, 9, 2), (20000, 20, 1)])
@pytest.mark.parametrize("dtype, dim", [("bf16", 128), ("f32", 64), ("f16", 256)])
def test_shared_long(kv, ws, prefix, members, heads, dtype, dim):  # noqa: F811
    """Prefixes whose keys are cut among many CTAs."""
    check(kv, ws, [(prefix, [33 * (i + 1) for i in range(members)])], 4, heads, dim, 64, "e4m3", "hnd", dtype, seed=prefix)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("rows", [[2, 5, 1, 1, 3], [1, 0, 9, 0, 8], [0, 0, 4, 1, 1], [40, 1, 2, 60, 1]], ids=str)
def test_shared_several_rows(kv, ws, rows, dtype):  # noqa: F811
    """Rows of a chunk, sequences without rows, rows that see less than the sequences have in common."""
    check(kv, ws, [(200, [2, 30, 9]), (100, [70, 4])], 4, 2, 64, 16, "e4m3", "hnd", dtype, rows=rows, seed=sum(rows))


def test_shared_tails_of_nothing(kv, ws):  # noqa: F811
    """Sequences that end with the prefix: the last row sees all of it and the first one token less."""
    check(kv, ws, [(64, [0, 0, 0]), (128, [0, 5])], 2, 2, 64, 16, "e4m3", "hnd", "f32")
    check(kv, ws, [(64, [0, 0, 0]), (128, [0, 5])], 2, 2, 64, 16, "int8", "hnd", "bf16", rows=[1, 2, 1, 17, 1])


def test_sequences_of_no_group(kv, ws):  # noqa: F811
    """Borders that leave sequences at both ends out."""
    cache, table, lens, _ = shared_table(kv, [(0, [40]), (80, [3, 9, 1]), (96, [5, 5])], 2, 64, 16, "e4m3", "hnd")
    n = len(lens)
    q = torch.randn((n, 8, 64), device="cuda")
    for borders in ([1, 4], [1, 3], [0, 0, 1, 4], [0, 0, 1, 1, 4, 4], [6, 6]):
        plan = kv.kv_share(cache, table, i32(lens), i32(borders))
        assert plan.tolist() == plan_ref(table.tolist(), lens, list(range(n + 1)), borders, 16, cache.pages)
        out, lse = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, return_lse=True, workspace=ws)
        close(out, lse, attention_ref(cache, 0, q, table, lens, list(range(n + 1)), 1 / 8), max(lens) + 512, torch.float32)


def test_share_of_bad_inputs(kv, ws):  # noqa: F811
    cache, table, lens, borders = shared_table(kv, [(80, [3, 9, 1]), (96, [5, 5])], 2, 64, 16, "e4m3", "hnd", wide=False)
    for bad in ([0, 4, 2], [-1, 3, 5], [0, 3, 6], [5, 3, 5]):
        plan = kv.kv_share(cache, table, i32(lens), i32(bad))
        assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS and (plan == 0).all()
    # page numbers outside the cache are no common pages, from the first of them on
    ids = table.clone()
    ids[:3, 2] = cache.pages
    ids[3:, 0] = -1
    plan = kv.kv_share(cache, ids, i32(lens), i32(borders)).tolist()
    assert [plan[2], plan[6]] == [32, 0] and plan[8:] == [32, 32, 32, 0, 0]
    # lengths beyond the table, rows that are none
    plan = kv.kv_share(cache, table, i32([83, 5000, 81, 101, 101]), i32(borders)).tolist()
    assert plan[2] == 0 and plan[6] == 96
    plan = kv.kv_share(cache, table, i32(lens), i32(borders), starts=i32([0, 1, 0, 2, 3, 4])).tolist()
    assert plan[2] == 0 and plan[6] == 96
    plan = kv.kv_share(cache, table, i32(lens), i32(borders), starts=i32([0, 1, 2, 3, 4, 9]), rows=5).tolist()
    assert plan[2] == 80 and plan[6] == 0


def test_shared_bad_plans_are_reported(kv, ws):  # noqa: F811
    """Entries that do not fit the call reach nothing outside it; the groups that fit are right."""
    cache, table, lens, borders = shared_table(kv, [(320, [3, 9, 1]), (400, [5, 5])], 2, 64, 16, "e4m3", "hnd")
    q = torch.randn((8, 8, 64), device="cuda")
    good = kv.kv_share(cache, table, i32(lens), i32(borders))
    ref = attention_ref(cache, 0, q, table, lens, list(range(9)), 1 / 8)
    for at, value in ((0, -1), (0, 6), (1, 9), (1, -2), (2, -16), (2, 1 << 30), (2, 7), (3, 8), (3, -1), (8, -16), (9, 1 << 20), (10, 7)):
        plan = good.clone()
        plan[at] = value
        out = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, workspace=ws)
        assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS, (at, value)
        close(out[3:], None, tuple(x[3:] for x in ref), max(lens) + 512, torch.float32)


@pytest.mark.parametrize("change, wrong", [({1: 2}, [2]), ({1: 0}, [0, 1, 2]), ({0: 1, 1: 2}, [0]), ({2: 304}, [0, 1, 2]), ({2: 0}, [0, 1, 2]),
                                           ({8: 304}, [0]), ({9: 16, 10: 160}, [1, 2]), ({0: 3, 1: 2}, [0, 1, 2, 3, 4]), ({1: 5}, [3, 4]),
                                           ({4: 0, 5: 5}, [3, 4]), ({5: 1}, [4]), ({13: 16}, [5])], ids=str)
def test_shared_plans_that_disagree_are_reported(kv, ws, change, wrong):  # noqa: F811
    """Entries in range of which groups and sequences say different things, behind a call that left results for every
    row of them: rows whose entries agree are right."""
    cache, table, lens, borders = shared_table(kv, [(320, [3, 9, 1]), (400, [5, 5])], 2, 64, 16, "e4m3", "hnd")
    lens[5:], n = [40] * 3, len(lens)  # sequences of no group, which could share two pages
    table[5:, :3] = table[0, :3]
    q = torch.randn((n, 8, 64), device="cuda")
    good = kv.kv_share(cache, table, i32(lens), i32(borders))
    assert good.tolist() == [0, 3, 320, 0, 3, 2, 400, 3, 320, 320, 320, 400, 400, 0, 0, 0]
    others = kv.kv_share(cache, table, i32(lens), i32([5, 8]))
    assert others.tolist() == [5, 3, 32, 5] + [0] * 5 + [32] * 3
    for plan in (others, good):
        kv.kv_attention_shared(cache, 1, q, table, i32(lens), plan, workspace=ws)
    assert qgemv.qg_device_status() == qgemv.QG_OK
    plan, right = good.clone(), [b for b in range(n) if b not in wrong]
    for at, value in change.items():
        plan[at] = value
    out, lse = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, return_lse=True, workspace=ws)
    assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS
    ref = attention_ref(cache, 0, q, table, lens, list(range(n + 1)), 1 / 8)
    close(out[right], lse[right], tuple(x[right] for x in ref), max(lens) + 512, torch.float32)


def beyond_the_table(kv):  # noqa: F811
    """A batch whose second sequence has a page in every column; its lengths as they are, and with that one the table's."""
    cache, table, lens, borders = shared_table(kv, [(320, [3, 9, 1]), (400, [5, 5])], 2, 64, 16, "e4m3", "hnd")
    width = table.shape[1]
    table[1, 20:] = torch.arange(width - 20, device="cuda").int() % cache.pages
    return cache, table, lens, borders, 16 * width, [*lens[:1], 16 * width, *lens[2:]]


def test_shared_length_beyond_the_table(kv, ws):  # noqa: F811
    """It counts as the table, and the tokens shared are read once: by the prefix, not again and not instead of others."""
    cache, table, lens, borders, most, held = beyond_the_table(kv)
    q = torch.randn((8, 8, 64), device="cuda")
    plan = kv.kv_share(cache, table, i32(lens), i32(borders))
    ref = attention_ref(cache, 0, q, table, held, list(range(9)), 1 / 8)
    for more in (1, 16, 320, 5 * most):
        beyond = list(lens)
        beyond[1] = most + more
        out, lse = kv.kv_attention_shared(cache, 0, q, table, i32(beyond), plan, return_lse=True, workspace=ws)
        assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS
        close(out, lse, ref, most + 512, torch.float32)


def test_shared_length_and_plan_beyond_the_table(kv, ws):  # noqa: F811
    """An entry beyond the table too, by as much as the length among them: it counts as nothing shared."""
    cache, table, lens, borders, most, held = beyond_the_table(kv)
    q = torch.randn((8, 8, 64), device="cuda")
    good = kv.kv_share(cache, table, i32(lens), i32(borders))
    ref = attention_ref(cache, 0, q, table, held, list(range(9)), 1 / 8)
    for skip in (most + 16, 2 * most, 1 << 20):
        for more in (skip, skip + 16, skip - 16):
            beyond, plan = list(lens), good.clone()
            beyond[1] = most + more
            plan[9] = skip
            out, lse = kv.kv_attention_shared(cache, 0, q, table, i32(beyond), plan, return_lse=True, workspace=ws)
            assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS
            close(out, lse, ref, most + 512, torch.float32)


def test_shared_bad_pages_are_reported_and_masked(kv, ws):  # noqa: F811
    """A plan made before its pages were lost: they count as masked in all rows."""
    cache, table, lens, borders = shared_table(kv, [(320, [3, 9, 1])], 2, 64, 16, "e4m3", "hnd")
    q = torch.randn((4, 8, 64), device="cuda")
    plan = kv.kv_share(cache, table, i32(lens), i32(borders))
    for bad in (-1, cache.pages):
        ids = table.clone()
        ids[:, 5] = bad
        ids[1, 20] = bad  # the page behind the prefix
        out, lse = kv.kv_attention_shared(cache, 0, q, ids, i32(lens), plan, return_lse=True, workspace=ws)
        assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS
        keep = [c for c in range(21) if c != 5]
        for b in range(3):  # the same tokens in a table without the lost pages
            cols = [c for c in keep if not (b == 1 and c == 20)]
            n = len(cols) * 16 - (16 - lens[b] % 16) % 16 if cols[-1] == 20 else len(cols) * 16
            ref = attention_ref(cache, 0, q[b:b + 1], table[b:b + 1, cols], [n], [0, 1], 1 / 8)
            close(out[b:b + 1], lse[b:b + 1], ref, max(lens) + 512, torch.float32)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_shared_masked_tokens_do_not_reach(kv, ws, dtype, dim):  # noqa: F811
    """NaN codes in pages that no row sees, behind every sequence's end and in the part of a page behind it."""
    cache, table, lens, borders = shared_table(kv, [(330, [3, 9, 1, 20])], 2, dim, 16, "e4m3", "hnd")
    q = torch.randn((4, 8, dim), device="cuda").to(DT[dtype])
    plan = kv.kv_share(cache, table, i32(lens), i32(borders))
    want = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, return_lse=True, workspace=ws)
    held = torch.zeros((cache.pages, 16), dtype=torch.bool, device="cuda")
    for b, n in enumerate(lens):
        for t in range(n):
            held[table[b, t // 16], t % 16] = True
    for c in (cache.k, cache.v):
        c[0].masked_fill_(~held[:, None, :, None], 0x7F)
    free = ~held.any(1)
    cache.k_scale[0, free] = math.nan
    cache.v_scale[0, free] = math.inf
    got = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, return_lse=True, workspace=ws)
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("where", [5, 321, 330])
def test_shared_nan_codes_that_rows_see(kv, ws, dtype, where):  # noqa: F811
    """A NaN code of V in the prefix reaches its dim of every row of its head; behind it, of the row that holds it."""
    cache, table, lens, borders = shared_table(kv, [(320, [30, 40])], 2, 64, 16, "e4m3", "hnd")
    q = torch.randn((4, 8, 64), device="cuda").to(DT[dtype])
    plan = kv.kv_share(cache, table, i32(lens), i32(borders))
    want = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, workspace=ws)
    cache.v[0, table[1, where // 16], 1, where % 16, 37] = 0x7F
    got = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, workspace=ws)
    nan = torch.isnan(got)
    expect = torch.zeros_like(nan)
    expect[:2 if where < 320 else 0, 4:, 37] = True
    expect[1, 4:, 37] = True
    assert torch.equal(nan, expect)
    assert torch.equal(got[~nan], want[~nan])


@pytest.mark.parametrize("unit", [18, 24, 60, 120])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("dim, fmt, dtype", [(64, "e4m3", "f32"), (128, "int8", "bf16"), (128, "e4m3", "f16"), (256, "e4m3", "bf16")])
@pytest.mark.parametrize("members, n", [(2, 700), (40, 3000)])
def test_shared_scores_of_any_size(kv, ws, unit, sign, dim, fmt, dtype, members, n):  # noqa: F811
    """Scores that are whole multiples, up to 8, of 2^unit, in the prefix and behind it: all weight is on the tokens of
    the largest, in equal shares, over blocks whose V scales differ."""
    from test_kv_edges_gpu import code
    cache, table, lens, borders = shared_table(kv, [(n, [1 + i % 20 for i in range(members)])], 1, dim, 16, fmt, "hnd")
    cpu = torch.Generator().manual_seed(unit + n)
    g = torch.Generator(device="cuda").manual_seed(unit)
    what = torch.randint(-8, 9, (cache.pages, 16), generator=cpu)
    if sign < 0:
        what = what.abs() + 1
    by_value = {x: code(x, fmt) for x in range(-9, 10)}
    cache.k.zero_()
    cache.k_scale.fill_(1.0)
    cache.k[0, :, 0, :, 1] = torch.tensor([[by_value[int(x)] for x in row] for row in what], dtype=torch.uint8, device="cuda")
    cache.v.copy_(torch.randint(0, 100, cache.v.shape, device="cuda", generator=g, dtype=torch.uint8))
    cache.v_scale.copy_(torch.exp2(torch.randint(-6, 7, cache.v_scale.shape, device="cuda", generator=g).float()))
    q = torch.zeros((len(lens), 2, dim), device="cuda")
    q[:, :, 1] = sign
    q = q.to(DT[dtype])
    plan = kv.kv_share(cache, table, i32(lens), i32(borders))
    out, lse = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, scale=2.0 ** unit, return_lse=True, workspace=ws)
    from test_kv_gpu import gather
    for b in range(members):
        x = sign * torch.cat([what[p] for p in table[b, :(lens[b] + 15) // 16].tolist()])[:lens[b]].double().cuda()
        p = (x == x.max()).double()
        want = (p / p.sum()) @ gather(cache, 0, table, b, lens[b], "v")[:, 0]  # no value is negative
        eps = torch.finfo(DT[dtype]).eps / 2 + (2.0 ** -11 if dtype == "bf16" else 0.0) + (40 + lens[b] / 64) * 2.0 ** -22
        assert ((out[b].double() - want).abs() <= want * eps * 1.01 + 1e-30).all()
        top = x.max().item() * 2.0 ** unit
        assert ((lse[b].double() - top).abs() <= math.log(lens[b]) + 1e-4 + abs(top) * 2.0 ** -22).all()


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim, members", [(64, 3), (128, 40), (256, 5)])
def test_shared_scales_of_all_sizes(kv, ws, dtype, dim, members):  # noqa: F811
    """V scales 2^-40 to 2^-4 by page, some zero; K scales zero in some pages; rows whose weight is on small ones."""
    cache, table, lens, borders = shared_table(kv, [(500, [1 + 3 * i % 40 for i in range(members)])], 2, dim, 16, "e4m3", "hnd")
    g = torch.Generator(device="cuda").manual_seed(dim)
    cache.v_scale.copy_(torch.exp2(torch.randint(-40, -3, cache.v_scale.shape, device="cuda", generator=g).float()))
    cache.v_scale[0, ::7] = 0.0
    cache.k_scale[0, ::11] = 0.0
    cache.v_scale[0, table[0, 3]] = 0.0
    q = torch.randn((len(lens), 8, dim), device="cuda", generator=g).to(DT[dtype])
    plan = kv.kv_share(cache, table, i32(lens), i32(borders))
    out, lse = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, return_lse=True, workspace=ws)
    ref = attention_ref(cache, 0, q, table, lens, list(range(len(lens) + 1)), 1 / math.sqrt(dim))
    close(out, lse, small((*ref[:4], ref[4] * 2.0 ** 4), dtype), max(lens) + 512, DT[dtype], one_part=dtype == "bf16")


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim, members", [(64, 3), (128, 40), (256, 5)])
def test_shared_scales_of_all_sizes_to_the_stated_cut(kv, ws, dtype, dim, members, fmt):  # noqa: F811
    """As above, to the cut of small weights that the module's tolerance counts and no more."""
    for seed in range(4):
        cache, table, lens, borders = shared_table(kv, [(500, [1 + 3 * i % 40 for i in range(members)])], 2, dim, 16, fmt, "hnd", seed=seed)
        g = torch.Generator(device="cuda").manual_seed(dim + seed)
        cache.v_scale.copy_(torch.exp2(torch.randint(-40, -3, cache.v_scale.shape, device="cuda", generator=g).float()))
        cache.v_scale[0, ::7] = 0.0
        cache.k_scale[0, ::11] = 0.0
        cache.v_scale[0, table[0, 3]] = 0.0
        q = torch.randn((len(lens), 8, dim), device="cuda", generator=g).to(DT[dtype])
        plan = kv.kv_share(cache, table, i32(lens), i32(borders))
        out, lse = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, return_lse=True, workspace=ws)
        ref = attention_ref(cache, 0, q, table, lens, list(range(len(lens) + 1)), 1 / math.sqrt(dim))
        close(out, lse, small(ref, dtype), max(lens) + 512, DT[dtype], one_part=dtype == "bf16")


def test_shared_prefix_below_and_above_the_rest(kv, ws):  # noqa: F811
    """The prefix's scores lie 300 binary orders below those behind it, or above: one part's weight is 0."""
    from test_kv_edges_gpu import code
    for up in (True, False):
        cache, table, lens, borders = shared_table(kv, [(640, [3, 30, 17])], 1, 64, 16, "e4m3", "hnd")
        cache.k.fill_(code(1 if up else -2, "e4m3"))
        cache.k[:, table[0, :40].long()] = code(-2 if up else 1, "e4m3")
        cache.k_scale.fill_(1.0)
        q = torch.full((4, 2, 64), 100.0, device="cuda")
        plan = kv.kv_share(cache, table, i32(lens), i32(borders))
        out, lse = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, scale=math.log(2) / 64, return_lse=True, workspace=ws)
        close(out, lse, attention_ref(cache, 0, q, table, lens, [0, 1, 2, 3, 4], math.log(2) / 64), 1200, torch.float32)


def test_shared_non_finite_queries(kv, ws):  # noqa: F811
    """A query row with NaN gives NaN; the other rows of its block are as without it."""
    cache, table, lens, borders = shared_table(kv, [(500, [3, 30, 17, 8, 9])], 2, 128, 16, "e4m3", "hnd")
    q = torch.randn((5, 8, 128), device="cuda").bfloat16()
    plan = kv.kv_share(cache, table, i32(lens), i32(borders))
    want = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, workspace=ws)
    q[2, 3, 70] = math.nan
    got = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, workspace=ws)
    assert torch.isnan(got[2, 3]).all()
    got[2, 3] = want[2, 3]
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_shared_strided_queries_and_outputs(kv, ws, dtype):  # noqa: F811
    cache, table, lens, borders = shared_table(kv, [(500, [3, 30, 17, 8, 9])], 2, 64, 16, "e4m3", "hnd")
    wide = torch.randn((5, 20, 64), device="cuda").to(DT[dtype])
    q = wide[:, 5:13]
    plan = kv.kv_share(cache, table, i32(lens), i32(borders))
    out, lse = torch.empty((5, 8, 64), device="cuda", dtype=DT[dtype]), torch.empty((5, 8), device="cuda")
    want = kv.kv_attention_shared(cache, 0, q.contiguous(), table, i32(lens), plan, return_lse=True, workspace=ws)
    got = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, out=out, lse=lse, workspace=ws)
    assert got is out and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    assert torch.equal(kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan), want[0])  # a workspace of its own


def test_shared_rows_behind_the_last_are_left(kv, ws):  # noqa: F811
    cache, table, lens, borders = shared_table(kv, [(500, [30, 30])], 2, 64, 16, "e4m3", "hnd")
    q = torch.randn((11, 8, 64), device="cuda")
    starts = i32([0, 2, 5, 6, 7])
    plan = kv.kv_share(cache, table, i32(lens), i32(borders), starts=starts)
    out = torch.full((11, 8, 64), 3.0, device="cuda")
    kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, starts=starts, out=out, workspace=ws)
    assert (out[7:] == 3.0).all() and not (out[:7] == 3.0).any()


def test_shared_repeats_bit_for_bit_and_alternates(kv, ws):  # noqa: F811
    """The same bits again, with other calls of the same workspace between."""
    cache, table, lens, borders = shared_table(kv, [(3000, [3, 30, 17, 8] * 12)], 2, 128, 16, "e4m3", "hnd")
    q = torch.randn((48, 8, 128), device="cuda").bfloat16()
    plan = kv.kv_share(cache, table, i32(lens), i32(borders))
    first = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, return_lse=True, workspace=ws)
    for _ in range(5):
        other = kv.kv_attention(cache, 0, q, table, i32(lens), return_lse=True, workspace=ws)
        again = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, return_lse=True, workspace=ws)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    # two roundings of bf16, and what each of the two may be off by before them
    assert ((other[0].double() - first[0].double()).abs() <= 2.0 ** -7 * first[0].double().abs() + 2.0 ** -9 * first[0].abs().max()).all()


def test_shared_in_a_graph_and_on_a_stream(kv):  # noqa: F811
    """A captured plan and attention, replayed with other lengths, tables and queries, against direct calls."""
    side, own = torch.cuda.Stream(), kv.KVWorkspace("cuda")
    cache, table, lens, borders = shared_table(kv, [(600, [70, 60, 80]), (320, [50, 50])], 2, 64, 16, "e4m3", "hnd")
    q, ln, gr = torch.randn((len(lens), 8, 64), device="cuda"), i32(lens), i32(borders)

    def step():
        plan = kv.kv_share(cache, table, ln, gr)
        return plan, kv.kv_attention_shared(cache, 0, q, table, ln, plan, workspace=own)

    step()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        plan, out = step()
    torch.cuda.current_stream().wait_stream(side)
    first = table.clone()
    for i, cut in enumerate((0, 37, 4)):
        table.copy_(first)
        table[1, cut:] = table[1, cut:].roll(1)  # less in common
        ln.copy_(i32([n - 9 * i if n > 5 else n for n in lens]))
        q.normal_()
        graph.replay()
        want_plan = kv.kv_share(cache, table, ln, gr)
        want = kv.kv_attention_shared(cache, 0, q, table, ln, want_plan)
        assert torch.equal(plan, want_plan) and torch.equal(out, want)
        other = kv.kv_attention_shared(cache, 0, q, table, ln, plan, stream=side, workspace=own)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(other, want)
    # the roll brought a place without a page among those of sequence 1
    assert (table[1, :-(-int(ln[1]) // 16)] < 0).any() and qgemv.qg_device_status() == qgemv.QG_EBOUNDS


def test_shared_results_beyond_the_workspace(kv, ws):  # noqa: F811
    """More rows than the workspace holds results for."""
    batch = 1500
    cache, table, lens, borders = shared_table(kv, [(320, [1 + i % 30 for i in range(batch)])], 1, 128, 16, "e4m3", "hnd", layers=1)
    q = torch.randn((batch, 32, 128), device="cuda").bfloat16()
    plan = kv.kv_share(cache, table, i32(lens), i32(borders))
    out, lse = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, return_lse=True, workspace=ws)
    some = list(range(0, batch, 97)) + [batch - 1]
    ref = attention_ref(cache, 0, q[some], table[some], [lens[b] for b in some], list(range(len(some) + 1)), 128 ** -0.5)
    close(out[some], lse[some], small(ref, "bf16"), 900, torch.bfloat16, one_part=True)


def test_shared_from_a_width_on(kv, ws):  # noqa: F811
    """On both sides of the least width: below it kv_attention's bits, whatever the plan; from it on the plan is read."""
    cache, table, lens, borders = shared_table(kv, [(320, [3, 9, 1]), (400, [5, 5])], 2, 64, 16, "e4m3", "hnd")
    q, least = torch.randn((8, 8, 64), device="cuda"), least_width(8, 2, 64, 16)
    assert table.shape[1] == least
    ref = attention_ref(cache, 0, q, table, lens, list(range(9)), 1 / 8)
    for width in (least - 1, least):
        ids = table[:, :width].contiguous()
        plan = kv.kv_share(cache, ids, i32(lens), i32(borders))
        got = kv.kv_attention_shared(cache, 0, q, ids, i32(lens), plan, return_lse=True, workspace=ws)
        plain = kv.kv_attention(cache, 0, q, ids, i32(lens), return_lse=True, workspace=ws)
        close(*got, ref, max(lens) + 512, torch.float32)
        if width < least:
            assert torch.equal(got[0], plain[0]) and torch.equal(got[1], plain[1])
        plan[2] = 7
        kv.kv_attention_shared(cache, 0, q, ids, i32(lens), plan, workspace=ws)
        assert qgemv.qg_device_status() == (qgemv.QG_OK if width < least else qgemv.QG_EBOUNDS)


@pytest.mark.parametrize("members, shared", [(3, False), (4, True)])
def test_shared_from_four_sequences_a_group_on(kv, ws, members, shared):  # noqa: F811
    lens = [200 + i for i in range(3 * members)]
    cache, table, _ = make(kv, lens, 2, 64, 16, "e4m3", "hnd", width=least_width(len(lens), 2, 64, 16))
    for i in range(0, len(lens), members):
        table[i:i + members, :10] = table[i, :10].clone()
    q = torch.randn((len(lens), 8, 64), device="cuda")
    plan = kv.kv_share(cache, table, i32(lens), i32([0, members, 2 * members, 3 * members]))
    assert plan[2:12:4].tolist() == [160] * 3
    got = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, return_lse=True, workspace=ws)
    plain = kv.kv_attention(cache, 0, q, table, i32(lens), return_lse=True, workspace=ws)
    assert torch.equal(got[1], plain[1]) != shared
    close(*got, attention_ref(cache, 0, q, table, lens, list(range(len(lens) + 1)), 1 / 8), max(lens) + 512, torch.float32)


@pytest.mark.parametrize("alone", ["in groups", "behind the groups"])
def test_shared_beside_sequences_that_share_nothing(kv, ws, alone):  # noqa: F811
    """Twelve sequences behind a prompt and five of their own: with a group for each of the five the call has too few
    sequences a group to share; where the borders leave them out it shares."""
    lens = [643 + i for i in range(12)] + [50 + i for i in range(5)]
    n = len(lens)
    cache, table, _ = make(kv, lens, 2, 64, 16, "e4m3", "hnd", width=least_width(n, 2, 64, 16))
    table[:12, :40] = table[0, :40].clone()
    q = torch.randn((n, 8, 64), device="cuda")
    plan = kv.kv_share(cache, table, i32(lens), i32([0, 12, 13, 14, 15, 16, 17] if alone == "in groups" else [0, 12]))
    assert plan[2] == 640
    got = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, return_lse=True, workspace=ws)
    plain = kv.kv_attention(cache, 0, q, table, i32(lens), return_lse=True, workspace=ws)
    assert torch.equal(got[1], plain[1]) == (alone == "in groups")
    close(*got, attention_ref(cache, 0, q, table, lens, list(range(n + 1)), 1 / 8), max(lens) + 512, torch.float32)


@pytest.mark.parametrize("rows, shared", [(31, True), (32, False)])
def test_shared_up_to_many_rows(kv, ws, rows, shared):  # noqa: F811
    """128 query rows a sequence of 80 go to the kernel of prompts, which shares nothing."""
    lens = [200 + i for i in range(80)]
    cache, table, _, borders = shared_table(kv, [(160, [n - 160 for n in lens])], 1, 64, 16, "e4m3", "hnd")
    st = [rows * i for i in range(81)]
    q = torch.randn((st[-1], 4, 64), device="cuda").bfloat16()
    plan = kv.kv_share(cache, table, i32(lens), i32(borders), starts=i32(st))
    got = kv.kv_attention_shared(cache, 0, q, table, i32(lens), plan, starts=i32(st), return_lse=True, workspace=ws)
    plain = kv.kv_attention(cache, 0, q, table, i32(lens), starts=i32(st), return_lse=True, workspace=ws)
    assert torch.equal(got[1], plain[1]) != shared
    close(*got, small(attention_ref(cache, 0, q, table, lens, st, 1 / 8), "bf16"), max(lens) + 512, torch.bfloat16, one_part=True)


def test_shared_largest_batch(kv, ws):  # noqa: F811
    """4096 sequences in 1024 groups."""
    shape = [(40, [1 + i % 7, 2, 3, 6]) for i in range(1023)] + [(0, [5, 4, 5, 1])]
    check(kv, ws, shape, 2, 1, 64, 16, "e4m3", "hnd", "f32")
