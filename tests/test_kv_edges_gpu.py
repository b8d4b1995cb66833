"""More GPU tests of the decode-state operators: values, scales and sizes at the
ends of their ranges.  Helpers and tolerances are test_kv_gpu's."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_quantised_weight_gb300 import qgemv  # noqa: E402
from test_kv_gpu import (DT, append_ref, attention_ref, beam_ref, check_beam, close, counts, filled, fork_ref, gather,  # noqa: E402, F401
                         i32, kv, make, starts_of, status_clean, values, ws)

pytestmark = pytest.mark.gpu


def code(x, fmt):
    """The 8-bit code of a value that the format holds."""
    if fmt == "e4m3":
        return torch.tensor(float(x)).to(torch.float8_e4m3fn).view(torch.uint8).item()
    return x & 0xFF


def ordered_cache(kv, n, heads, dim, fmt, page=16):  # noqa: F811
    """A cache of zeros with scales 1 whose one sequence lies on pages 0, 1, 2, ..."""
    pages = (n + page - 1) // page
    cache = kv.KVCache.allocate(1, pages, heads, page, dim, fmt, "hnd")
    cache.k_scale.fill_(1.0)
    cache.v_scale.fill_(1.0)
    return cache, i32([list(range(pages))])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("group, dim, fmt", [(1, 64, "e4m3"), (4, 128, "int8")])
def test_attention_prompt_scores_that_rise_in_every_half_step(kv, ws, dtype, group, dim, fmt):  # noqa: F811
    """In every 64 tokens one score lies 12 binary orders above all before it, on a token whose value is
    zero: what is stored of the first half of each 128 is rescaled in place by the second."""
    n, rows = 512, 256
    cache, table = ordered_cache(kv, n, 1, dim, fmt)
    k = torch.zeros((n, dim), dtype=torch.uint8, device="cuda")
    v = torch.full_like(k, code(1, fmt))
    for half in range(n // 64):
        k[half * 64:, 0] = code(12 * half & ~7, fmt)  # in two parts that e4m3 holds
        k[half * 64:, 1] = code(12 * half & 7, fmt)
        k[half * 64 + 7, 2] = code(12, fmt)
        v[half * 64 + 7] = 0
    cache.k[0, :, 0] = k.view(-1, 16, dim)
    cache.v[0, :, 0] = v.view(-1, 16, dim)
    q = torch.zeros((rows, group, dim), device="cuda")
    q[:, :, :3] = math.log(2)
    q = q.to(DT[dtype])
    out, lse = kv.kv_attention(cache, 0, q, table, i32([n]), starts=i32([0, rows]), scale=1.0, return_lse=True, workspace=ws)
    close(out, lse, attention_ref(cache, 0, q, table, [n], [0, rows], 1.0), n, DT[dtype], one_part=dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("dim, fmt", [(64, "e4m3"), (64, "int8"), (128, "e4m3"), (256, "int8")])
@pytest.mark.parametrize("rows", [2, 5, 14, 200])
@pytest.mark.parametrize("scale", [4.0, 2.0 ** 20])
def test_attention_large_scale_behind_a_block_of_zeros(kv, ws, dtype, dim, fmt, rows, scale):  # noqa: F811
    """The first rows see blocks whose V scale is 0 alone, and give 0; a block of a large scale behind them,
    which only later rows see, does not reach them."""
    n = 16 + rows - 1
    cache, table = ordered_cache(kv, n, 2, dim, fmt)
    g = torch.Generator(device="cuda").manual_seed(rows)
    for c in (cache.k, cache.v):
        c.copy_(torch.randint(0, 100, c.shape, device="cuda", generator=g, dtype=torch.uint8))
    cache.k_scale.fill_(0.01)
    cache.v_scale[0, 0] = 0.0
    cache.v_scale[0, 1:] = scale * (2.0 ** -10 if fmt == "int8" and dtype == "f16" else 1.0)
    q = torch.randn((rows, 4, dim), device="cuda", generator=g).to(DT[dtype])
    out, lse = kv.kv_attention(cache, 0, q, table, i32([n]), starts=i32([0, rows]), scale=0.1, return_lse=True, workspace=ws)
    ref = attention_ref(cache, 0, q, table, [n], [0, rows], 0.1)
    assert (out[0] == 0).all()
    if dtype == "f16":  # what passes its range is infinite
        fits = ref[0].abs() <= 65504
        out = torch.where(fits, out, 0.0)
        ref = (torch.where(fits, ref[0], 0.0), *ref[1:])
    close(out, lse, ref, n, DT[dtype], one_part=dtype == "bf16")


@pytest.mark.parametrize("rows", [1, 3, 300])
@pytest.mark.parametrize("dim, fmt", [(64, "e4m3"), (128, "int8"), (256, "e4m3")])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_attention_large_scale_of_low_scores(kv, ws, dtype, dim, fmt, rows):  # noqa: F811
    """Blocks whose V scales differ by 2^120, the large one's scores 150 to 300 binary orders below: its weights are 0."""
    n = 20 + 2 * rows
    cache, table = ordered_cache(kv, n, 1, dim, fmt)
    g = torch.Generator(device="cuda").manual_seed(rows)
    cache.v.copy_(torch.randint(0, 100, cache.v.shape, device="cuda", generator=g, dtype=torch.uint8))
    cache.k.fill_(code(-2, fmt))
    cache.k[0, 0] = code(1, fmt)
    cache.v_scale.fill_(2.0 ** 60)
    cache.v_scale[0, 0] = 2.0 ** -60
    q = (50.0 + 50.0 * torch.rand((rows, 2, dim), device="cuda", generator=g)).to(DT[dtype])
    scale = math.log(2) / dim  # scores 50 to 100 on the first block, -200 to -100 behind it
    out, lse = kv.kv_attention(cache, 0, q, table, i32([n]), starts=i32([0, rows]), scale=scale, return_lse=True, workspace=ws)
    close(out, lse, attention_ref(cache, 0, q, table, [n], [0, rows], scale), n, DT[dtype], one_part=dtype == "bf16")


@pytest.mark.parametrize("unit", [18, 24, 30, 60, 120])
@pytest.mark.parametrize("sign", [1, -1])
@pytest.mark.parametrize("n, rows", [(1, 1), (3000, 1), (700, 3), (40, 40), (700, 300), (3000, 260)])
@pytest.mark.parametrize("dim, fmt, dtype", [(64, "e4m3", "f32"), (128, "int8", "bf16"), (128, "e4m3", "f16"), (256, "e4m3", "bf16")])
def test_attention_scores_of_any_size(kv, ws, unit, sign, n, rows, dim, fmt, dtype):  # noqa: F811
    """Scores that are whole multiples, up to 8, of 2^unit: all weight is on the tokens of the largest, in equal
    shares, over blocks whose V scales differ, warps, CTAs and parts.  The scores are exact, so their term of the
    tolerance falls away.  With sign -1 all are at -2^unit or below."""
    cache, table = ordered_cache(kv, n, 1, dim, fmt)
    g = torch.Generator(device="cuda").manual_seed(unit)
    what = torch.randint(-8, 9, (n,), generator=torch.Generator().manual_seed(n)).tolist()
    if sign < 0:
        what = [abs(x) + 1 for x in what]  # times a q of -1
    k = torch.zeros((cache.pages * 16, dim), dtype=torch.uint8)
    k[:n, 1] = torch.tensor([code(x, fmt) for x in what], dtype=torch.uint8)
    cache.k[0, :, 0] = k.view(-1, 16, dim).cuda()
    cache.v.copy_(torch.randint(0, 100, cache.v.shape, device="cuda", generator=g, dtype=torch.uint8))
    cache.v_scale.copy_(torch.exp2(torch.randint(-6, 7, cache.v_scale.shape, device="cuda", generator=g).float()))
    q = torch.zeros((rows, 2, dim), device="cuda")
    q[:, :, 1] = sign
    q = q.to(DT[dtype])
    scale = 2.0 ** unit
    out, lse = kv.kv_attention(cache, 0, q, table, i32([n]), starts=i32([0, rows]), scale=scale, return_lse=True, workspace=ws)
    # equal shares of the largest (64-bit scores of this size do not hold the logarithm of their number)
    x = sign * torch.tensor(what, dtype=torch.float64, device="cuda").expand(rows, n)
    seen = torch.arange(n, device="cuda")[None, :] <= n - rows + torch.arange(rows, device="cuda")[:, None]
    x = torch.where(seen, x, -math.inf)
    top = x.amax(1, keepdim=True)
    p = (x == top).double() / (x == top).sum(1, keepdim=True)
    want = (p @ gather(cache, 0, table, 0, n, "v")[:, 0])[:, None].expand(rows, 2, dim)  # no value is negative
    wl = (top * scale + torch.log((x == top).sum(1, keepdim=True))).expand(rows, 2)
    zero = torch.zeros_like(wl)
    close(out, lse, (want, wl, want, zero, zero), n, DT[dtype], one_part=dtype == "bf16")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("vocab", [9, 700, 32001])
def test_beam_zeros_of_both_signs_are_equal(kv, ws, dtype, vocab):  # noqa: F811
    """-0.0 and +0.0 score the same: the lowest (beam, token) comes first, whatever the signs."""
    g = torch.Generator(device="cuda").manual_seed(vocab)
    sign = torch.randint(0, 2, (4, vocab), device="cuda", generator=g).float() * 2 - 1
    for x in (sign * 0.0, torch.where(torch.arange(vocab, device="cuda") % 3 == 0, -1.0, sign * 0.0)):
        x[:, 0] = -0.0
        for keep in (1, 2, min(8, 2 * vocab)):
            check_beam(kv, ws, x.to(DT[dtype]), torch.zeros((2, 2), device="cuda"), keep)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_beam_scores_below_the_range_are_ranked(kv, ws, dtype):  # noqa: F811
    """Masked by the type's lowest value on a beam that is masked the same way: the scores are -inf in fp32,
    and still come in the order of their 64-bit values, all `keep` of them."""
    low = torch.finfo(DT[dtype]).min
    for vocab, keep in ((8, 24), (40, 120), (300, 128), (300, 3)):
        x = torch.randn((3, vocab), device="cuda", generator=torch.Generator(device="cuda").manual_seed(vocab))
        x[0, 2:] = low
        x[1, 3:] = low
        x[2] = low
        x = x.to(DT[dtype])
        cum = torch.tensor([[torch.finfo(torch.float32).min, -3.0, torch.finfo(torch.float32).min]], device="cuda")
        s, t, p = kv.beam_select(x, cum, keep, workspace=ws)
        want, wt, wp = beam_ref(x, cum, keep)
        assert np.array_equal(t.cpu().numpy(), wt) and np.array_equal(p.cpu().numpy(), wp)
        with np.errstate(over="ignore"):
            want = want.astype(np.float32)
        assert np.array_equal(np.isinf(want), np.isinf(s.cpu().numpy())) and (s[0, :-1] >= s[0, 1:]).all()


@pytest.mark.parametrize("batch", [2049, 4096])
def test_reserve_of_more_pages_than_32_bits_count(kv, ws, batch):  # noqa: F811
    """Sequences that together ask for 2^31 pages and more: too few, and those that fit get theirs."""
    page, width, pages = 16, 1 << 20, 5000
    if torch.cuda.mem_get_info()[0] < batch * width * 4 + (1 << 30):
        pytest.skip("not enough device memory")
    table = torch.empty((batch, width), dtype=torch.int32, device="cuda")
    table[:, :4] = -1
    add = torch.full((batch,), width * page, dtype=torch.int32, device="cuda")
    small = [3, 1024, batch - 1]
    add[small] = i32([3 * page, 1, page + 1])
    cache = kv.KVCache.allocate(1, pages, 1, page, 16)
    refs = torch.ones(pages, dtype=torch.int32, device="cuda")
    free = [2, 4095, 4096, 4500, 4999]
    refs[free] = 0
    kv.kv_reserve(cache, table, torch.zeros_like(add), refs, add=add, workspace=ws)
    assert qgemv.qg_device_status() == qgemv.QG_EPAGES
    assert table[3, :4].tolist() == [2, 4095, 4096, -1] and table[1024, :2].tolist() == [4500, -1]
    assert (table[batch - 1, :2] == -1).all() and refs.tolist().count(0) == 1
    others = torch.ones(batch, dtype=torch.bool, device="cuda")
    others[[3, 1024]] = False
    assert (table[others, :4] == -1).all()


def test_empty_tensors(kv, ws):  # noqa: F811
    cache, table = ordered_cache(kv, 40, 2, 64, "e4m3")
    none = torch.empty((0, 2, 64), device="cuda")
    was = [x.clone() for x in (cache.k, cache.v, cache.k_scale, cache.v_scale)]
    kv.kv_append(cache, 0, none, none, table, i32([40]), starts=i32([0, 0]))
    out, lse = kv.kv_attention(cache, 0, torch.empty((0, 4, 64), device="cuda"), table, i32([40]), starts=i32([0, 0]),
                               return_lse=True, workspace=ws)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)
    kv.kv_copy_pages(cache, i32([]), i32([]))
    assert all(torch.equal(a, b) for a, b in zip(was, (cache.k, cache.v, cache.k_scale, cache.v_scale)))


def check_append(cache, layer, k, v, table, lens, rows):
    """Appends and compares codes and scales of every page with test_kv_gpu's block by block reference."""
    from block_quantised_weight_gb300 import qgkv
    fmt, page, heads = cache.fmt, cache.page_tokens, cache.heads
    st = starts_of(rows)
    before = [(values(c.clone(), fmt).cpu().numpy(), s.cpu().numpy().copy()) for c, s in
              ((cache.k, cache.k_scale), (cache.v, cache.v_scale))]
    qgkv.kv_append(cache, layer, k, v, table, i32(lens), starts=None if all(r == 1 for r in rows) else i32(st))
    ids = table.cpu().numpy()
    for (codes, scale), c, s, x in zip(before, (cache.k, cache.v), (cache.k_scale, cache.v_scale), (k, v)):
        x = x.float().cpu().numpy().astype(np.float64)
        view = codes[layer] if cache.order == "hnd" else codes[layer].transpose(0, 2, 1, 3)
        for b in range(len(lens)):
            at, end = lens[b], lens[b] + rows[b]
            while at < end:
                pid, off = int(ids[b, at // page]), at % page
                n = min(page - off, end - at)
                r = st[b] + at - lens[b]
                for h in range(heads):
                    view[pid, h], scale[layer, pid, h] = append_ref(view[pid, h], scale[layer, pid, h], off, x[r:r + n, h], fmt)
                at += n
        assert np.array_equal(s.cpu().numpy(), scale)
        assert np.array_equal(values(c, fmt).cpu().numpy(), codes)


def new_rows(rows, heads, dim, dtype, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((rows, 2, heads, dim), device="cuda", generator=g)
    x = (x * torch.exp2(torch.randint(-6, 6, (rows, 2, heads, 1), device="cuda", generator=g).float())).to(DT[dtype])
    return x[:, 0], x[:, 1]


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("page, dim", [(32, 64), (64, 64), (64, 128), (128, 128), (256, 80), (256, 256)])
def test_append_blocks_of_every_size(kv, fmt, dtype, page, dim):  # noqa: F811
    """Blocks of 2 to 64 vectors a thread: held in registers, or read twice; a partly filled first page."""
    lens, rows = [page // 3, 0, 2 * page - 1], [page + 5, 2 * page, 3]
    cache, table, _ = make(kv, [a + b for a, b in zip(lens, rows)], 2, dim, page, fmt, "nhd" if dim == 80 else "hnd", seed=page)
    k, v = new_rows(sum(rows), 2, dim, dtype, dim)
    check_append(cache, 1, k, v, table, lens, rows)


@pytest.mark.parametrize("batch", [33, 70, 300])
def test_append_ragged_batch(kv, batch):  # noqa: F811
    """More sequences than a warp looks through at once, empty ones among them."""
    g = np.random.default_rng(batch)
    rows = [int(x) for x in g.integers(0, 40, batch) * (g.random(batch) < 0.6)]
    lens = [int(x) for x in g.integers(0, 60, batch)]
    cache, table, _ = make(kv, [a + b for a, b in zip(lens, rows)], 1, 64, 16, "int8", "hnd", seed=batch)
    k, v = new_rows(sum(rows), 1, 64, "bf16", batch)
    check_append(cache, 0, k, v, table, lens, rows)


@pytest.mark.parametrize("rows", [1, 2])
def test_largest_batch(kv, ws, rows):  # noqa: F811
    """4096 sequences: attention, append, fork, reserve and free of as many as a call takes."""
    batch, page, heads, dim = 4096, 16, 1, 64
    g = np.random.default_rng(rows)
    lens = [int(x) for x in g.integers(rows, 40, batch)]
    cache, table, ln = make(kv, [n + rows for n in lens], heads, dim, page, "e4m3", "hnd", seed=rows, layers=1, width=4)
    starts = None if rows == 1 else i32(starts_of([rows] * batch))
    k, v = new_rows(rows * batch, heads, dim, "f32", rows)
    kv.kv_append(cache, 0, k, v, table, i32(lens), starts=starts)
    held = [n + rows for n in lens]
    q = torch.randn((rows * batch, 2, dim), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    out, lse = kv.kv_attention(cache, 0, q, table, i32(held), starts=starts, return_lse=True, workspace=ws)
    some = list(range(0, batch, 97)) + [batch - 1]
    at = torch.tensor([[b * rows + i for i in range(rows)] for b in some], device="cuda").flatten()
    ref = attention_ref(cache, 0, q[at], table[some], [held[b] for b in some], starts_of([rows] * len(some)), 1 / 8)
    close(out[at], lse[at], ref, 64, torch.float32)

    ids, pages = table.cpu().numpy(), cache.pages + 4096
    pool = filled(kv, 1, pages, 1, page, 16)
    refs = counts(ids, held, page, pages)
    parent = [int(x) for x in g.integers(0, batch, batch)]
    want = fork_ref(ids, held, parent, refs, page)
    t2, l2, r2 = kv.kv_fork(pool, table, i32(held), i32(parent), i32(refs.tolist()), workspace=ws)
    assert want[4] == 0 and np.array_equal(t2.cpu().numpy(), want[0]) and np.array_equal(r2.cpu().numpy(), want[2])
    want_table, want_refs = want[0].copy(), want[2].copy()
    free = [p for p in range(pages) if want_refs[p] == 0]
    for b in range(batch):
        if want[1][b] % page == 0 and want[1][b] // page < 4:
            want_table[b, want[1][b] // page] = free.pop(0)
            want_refs[want_table[b, want[1][b] // page]] = 1
    full = [b for b in range(batch) if want[1][b] == 4 * page]
    kv.kv_reserve(pool, t2, l2, r2, workspace=ws)
    assert qgemv.qg_device_status() == (qgemv.QG_EBOUNDS if full else qgemv.QG_OK)
    assert np.array_equal(t2.cpu().numpy(), want_table) and np.array_equal(r2.cpu().numpy(), want_refs)
    kv.kv_free(pool, table, i32(held), i32(refs.tolist()))
    assert (table == -1).all()


def test_graph_replay_of_every_operator(kv):  # noqa: F811
    """One graph of a decode step's operators, replayed on other values, against the same calls made directly; on a
    stream of its own throughout."""
    page, pages, layers, heads, dim, beams, vocab = 16, 200, 2, 2, 64, 4, 3001
    side, ws = torch.cuda.Stream(), kv.KVWorkspace("cuda")  # noqa: F811
    table = torch.full((beams, 12), -1, dtype=torch.int32, device="cuda")
    lens, refs = torch.zeros(beams, dtype=torch.int32, device="cuda"), torch.zeros(pages, dtype=torch.int32, device="cuda")
    cache = filled(kv, layers, pages, heads, page, dim)
    starts = i32([0, 40, 80, 200, 360])
    k, v = new_rows(360, heads, dim, "bf16", 3)
    q = torch.randn((360, 4, dim), device="cuda").bfloat16()
    logits, cum = torch.randn((beams, vocab), device="cuda"), torch.zeros((1, beams), device="cuda")
    fixed = (cache.k, cache.v, cache.k_scale, cache.v_scale, table, lens, refs)
    first = [x.clone() for x in fixed]

    def step():
        new = starts[1:] - starts[:-1]
        kv.kv_reserve(cache, table, lens, refs, add=new, workspace=ws)
        for layer in range(layers):
            kv.kv_append(cache, layer, k, v, table, lens, starts=starts)
        lens.add_(new)
        a = kv.kv_attention(cache, 1, q, table, lens, starts=starts, workspace=ws)
        s, t, p = kv.beam_select(logits, cum, beams, workspace=ws)
        t2, l2, r2 = kv.kv_fork(cache, table, lens, p.view(-1), refs, workspace=ws)
        drop = p.view(-1) % 2 == 0
        t3, l3, r3, n = kv.kv_compact(cache, t2, l2, r2, drop=drop, workspace=ws)
        kv.kv_copy_pages(cache, n + 1, n + 2, count=torch.ones_like(n))
        kv.kv_free(cache, t3, l3, r3)
        return a, s, t, p, t2, l2, r2, t3, l3, r3, n

    def restore(i):
        g = torch.Generator(device="cuda").manual_seed(i)
        for x, y in zip(fixed, first):
            x.copy_(y)
        logits.copy_(torch.randn(logits.shape, device="cuda", generator=g))
        q.copy_(torch.randn(q.shape, device="cuda", generator=g))
        k.copy_(torch.randn(k.shape, device="cuda", generator=g))

    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        want = []
        for i in range(3):
            restore(i)
            want.append([x.clone() for x in (*step(), *fixed)])
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = step()
        for i in (2, 0, 1):
            restore(i)
            graph.replay()
            for a, b in zip((*outs, *fixed), want[i]):
                assert torch.equal(a, b)
    side.synchronize()
    assert (want[0][3] != want[1][3]).any() or (want[0][2] != want[1][2]).any()


def test_tensors_dropped_after_a_call_on_another_stream(kv):  # noqa: F811
    """The caller's tables are dropped while the stream of the call is still busy with what came before; their
    memory, free for its own stream, is not overwritten before the call has read it."""
    page, pages, batch = 16, 400, 30
    g = np.random.default_rng(4)
    lens = [int(x) for x in g.integers(1, 100, batch)]
    cache = filled(kv, 1, pages, 1, page, 16)
    ids = np.full((batch, 8), -1, np.int32)
    at, perm = 0, g.permutation(pages)
    for b, n in enumerate(lens):
        need = (n + page - 1) // page
        ids[b, :need] = perm[at:at + need]
        at += need
    refs = counts(ids, lens, page, pages)
    parent = [int(x) for x in g.integers(0, batch, 40)]
    want = fork_ref(ids, lens, parent, refs, page)
    side, own = torch.cuda.Stream(), kv.KVWorkspace("cuda")
    given = [i32(x) for x in (ids.tolist(), lens, parent, refs.tolist())]
    sizes = [t.shape for t in given]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # about 50 ms
    outs = kv.kv_fork(cache, *given, workspace=own, stream=side)
    del given
    taken = [torch.zeros(s, dtype=torch.int32, device="cuda") for s in sizes for _ in range(3)]
    side.synchronize()
    for a, b in zip(outs, want):
        assert np.array_equal(a.cpu().numpy(), b)
    assert len(taken) == 12


@pytest.mark.parametrize("rows", [1, 7, 40, 300])
@pytest.mark.parametrize("fmt, dim, group", [("e4m3", 64, 2), ("int8", 128, 7), ("int8", 96, 4), ("e4m3", 256, 3)])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
def test_attention_small_weights_beside_large_ones(kv, ws, rows, fmt, dim, group, dtype):  # noqa: F811
    """Sharp rows whose largest weights meet codes of zero in half of the dims: what is left there are weights far
    below the largest, W.

    A part's largest stored weight is 2^10 at least (k = 12, less the next whole order of the score and of the scale;
    prompts of bf16 queries 2^5), storing it takes half a step of f16, 2^-25, and a rescaling of what is stored two
    more for each of two parts: below 2^-34 W each (2^-28 W)."""
    n = 200 + rows
    cache, table, ln = make(kv, [n], 2, dim, 16, fmt, "hnd", seed=rows + dim)
    g = torch.Generator(device="cuda").manual_seed(dim)
    cache.v[torch.rand(cache.v.shape, device="cuda", generator=g) < 0.5] = 0
    q = torch.randn((rows, 2 * group, dim), device="cuda", generator=g).to(DT[dtype])
    out, lse = kv.kv_attention(cache, 1, q, table, ln, starts=i32([0, rows]), scale=0.7, return_lse=True, workspace=ws)
    want, wl, absum, smax, floor = attention_ref(cache, 1, q, table, [n], [0, rows], 0.7)
    prompt = dtype == "bf16" and dim <= 128 and rows > 100
    close(out, lse, (want, wl, absum, smax, floor * 2.0 ** (10 if prompt else 4)), n, DT[dtype], one_part=dtype == "bf16")
