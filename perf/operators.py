"""Cases of the decode-state operators: the 8-bit paged cache, the attention
that reads it, the page operations that beam search and serving need, and the
beam selection itself.

``run`` computes one pass of a case either in plain torch operations
(``own = False``) or through the entry points of
``block_quantised_weight_gb300.qgkv`` (``own = True``).

A cache holds ``layers x pages x heads x page_tokens x head_dim`` 8-bit codes
for K and as many for V, with one fp32 scale for each (layer, page, head): the
block that shares a scale is the tokens of one page.  A sequence is a row of a
page table (int32 page numbers, -1 where it has none) and a length.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one user's decode step on the TinyLlama-1.1B head shape: latency is all that counts
        dict(name="attn_one_user", op="attn", batch=1, q_heads=32, heads=4, dim=64, page=64, context=777, rows=1,
             fmt="e4m3", dtype="float32", order="hnd"),
        # a decode batch of ragged lengths on the head shape of an 8B model
        dict(name="attn_batch", op="attn", batch=48, q_heads=32, heads=8, dim=128, page=64, context=4100, rows=1,
             fmt="e4m3", dtype="bfloat16", order="hnd"),
        # a few long documents: the cache is streamed once, the work is split over the length
        dict(name="attn_long", op="attn", batch=3, q_heads=32, heads=8, dim=128, page=128, context=131072, rows=1,
             fmt="int8", dtype="bfloat16", order="nhd"),
        # prompts read in chunks behind what the cache already holds
        dict(name="attn_prompt", op="attn", batch=3, q_heads=32, heads=8, dim=128, page=64, context=6000, rows=2048,
             fmt="e4m3", dtype="bfloat16", order="hnd"),
        # one token for each sequence of a decode batch
        dict(name="append_step", op="append", batch=48, heads=4, dim=64, page=64, context=2000, rows=1, fmt="e4m3",
             dtype="float32", order="hnd"),
        # prompts stored after their chunk's projections
        dict(name="append_prompt", op="append", batch=5, heads=8, dim=128, page=64, context=900, rows=4001,
             fmt="int8", dtype="bfloat16", order="nhd"),
        # beam search of one request: four beams, all layers of the cache
        dict(name="fork_one", op="fork", requests=1, beams=4, layers=22, heads=4, dim=64, page=16, context=333,
             fmt="e4m3", order="hnd"),
        # beam search of a batch
        dict(name="fork_batch", op="fork", requests=48, beams=5, layers=22, heads=4, dim=64, page=16, context=600,
             fmt="e4m3", order="hnd"),
        # a small pool whose finished sequences are freed and whose rest is moved together
        dict(name="compact_small", op="compact", batch=16, layers=4, heads=4, dim=64, page=16, context=300, pages=700,
             fmt="int8", order="hnd"),
        # the same of a server's pool
        dict(name="compact_pool", op="compact", batch=200, layers=16, heads=8, dim=128, page=16, context=260,
             pages=6000, fmt="e4m3", order="hnd"),
        # the selection of one request over TinyLlama's vocabulary
        dict(name="beam_one", op="beam", requests=1, beams=4, keep=8, vocab=32000, dtype="float32"),
        # a batch with a larger vocabulary of odd size
        dict(name="beam_batch", op="beam", requests=48, beams=8, keep=16, vocab=128257, dtype="float32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges of listed(): any operator, sizes spread over their logarithm."""
    op = rng.choice(["attn", "attn", "attn", "append", "append", "fork", "compact", "beam"])
    fmt, order = rng.choice(["e4m3", "int8"]), rng.choice(["hnd", "nhd"])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["float32", "bfloat16", "float16"])
    heads, dim = rng.choice([1, 2, 4, 8]), rng.choice([64, 64, 80, 96, 128, 128, 256])
    if op == "attn":
        group = rng.choice([1, 3, 4, 6, 8, 8, 12])
        while True:
            batch, context = _log(rng, 1, 96), _log(rng, 1, 131072)
            rows = rng.choice([1, 1, 1, _log(rng, 1, 2048)])
            rows = min(rows, context)
            held = batch * context * heads * dim
            if held <= 3 * 131072 * 8 * 128 and held * rows * group <= 3 * 6000 * 8 * 128 * 2048 * 4:
                return dict(op=op, batch=batch, q_heads=heads * group, heads=heads, dim=dim, page=page,
                            context=context, rows=rows, fmt=fmt, dtype=dtype, order=order)
    if op == "append":
        while True:
            batch, context, rows = _log(rng, 1, 96), _log(rng, 1, 4000), rng.choice([1, _log(rng, 1, 4001)])
            if batch * rows * heads * dim <= 5 * 4001 * 8 * 128 and batch * (context + rows) <= 150000:
                return dict(op=op, batch=batch, heads=heads, dim=dim, page=page, context=context, rows=rows, fmt=fmt,
                            dtype=dtype, order=order)
    if op == "fork":
        while True:
            requests, beams, layers = _log(rng, 1, 64), rng.randint(2, 8), _log(rng, 1, 32)
            context = _log(rng, 8, 2000)
            if requests * beams * layers * heads * dim * page <= 48 * 5 * 22 * 4 * 64 * 16 and \
                    requests * beams * (context + page) * layers * heads * dim <= 48 * 5 * 620 * 22 * 4 * 64:
                return dict(op=op, requests=requests, beams=beams, layers=layers, heads=heads, dim=dim, page=page,
                            context=context, fmt=fmt, order=order)
    if op == "compact":
        while True:
            batch, layers, context = _log(rng, 2, 256), _log(rng, 1, 32), _log(rng, 8, 2000)
            pages = batch * (context // page + 1) + _log(rng, 8, 2000)
            if pages * layers * heads * dim * page <= 6000 * 16 * 8 * 128 * 16:
                return dict(op=op, batch=batch, layers=layers, heads=heads, dim=dim, page=page, context=context,
                            pages=pages, fmt=fmt, order=order)
    while True:
        requests, beams, vocab = _log(rng, 1, 128), rng.randint(1, 12), _log(rng, 500, 160000)
        keep = rng.choice([beams, 2 * beams])
        if requests * beams * vocab <= 48 * 8 * 128257:
            return dict(op="beam", requests=requests, beams=beams, keep=keep, vocab=vocab, dtype=dtype)


# ---------------------------------------------------------------- what a program has in hand

def _codes_as_values(codes, fmt):
    return codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8)


def _quantise(x, s, fmt):
    """Codes (uint8) of x for the scales s (broadcast; a scale of 0 stands for a block of zeros)."""
    y = torch.where(s > 0, x / torch.where(s > 0, s, 1.0), 0.0)
    if fmt == "e4m3":
        return y.clamp(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn).view(torch.uint8)
    return torch.nan_to_num(y, nan=0.0).clamp(-127, 127).round().to(torch.int8).view(torch.uint8)


def _scale_for(amax, fmt):
    """The scale that a largest magnitude asks for: a power of two for e4m3, amax/127 for int8."""
    if fmt == "int8":
        return amax / torch.full_like(amax, 127.0)  # a tensor: a division by a number may become a product
    m, e = torch.frexp(amax)
    e = torch.where(m > 0.875, e - 8, e - 9).clamp(min=-126)  # amax <= 448 * 2^e = 0.875 * 2^(e + 9)
    return torch.where(amax > 0, (e.int() + 127 << 23).view(torch.float32), 0.0)  # the exponent's bits: 2^e exactly


def _fill(shape, gen, dev):
    """Values as a cache meets them: normal, some channels several times as large."""
    x = torch.randn(shape, device=dev, generator=gen)
    return x * (1.0 + 5.0 * (torch.rand(shape[-1], device=dev, generator=gen) < 0.05))


def _make_cache(case, layers, pages, gen, dev):
    """Code and scale tensors [layers, pages, heads, page, dim] (or nhd order) and [layers, pages, heads]."""
    out = []
    for _ in range(2):
        codes = torch.empty((layers, pages, case["heads"], case["page"], case["dim"]), dtype=torch.uint8, device=dev)
        scale = torch.empty((layers, pages, case["heads"]), device=dev)
        step = max(1, (1 << 26) // max(1, codes[0, 0].numel()))
        for layer in range(layers):
            for at in range(0, pages, step):
                n = min(step, pages - at)
                x = _fill((n, case["heads"], case["page"], case["dim"]), gen, dev)
                s = _scale_for(x.abs().amax(dim=(2, 3)), case["fmt"])
                codes[layer, at:at + n] = _quantise(x, s[..., None, None], case["fmt"])
                scale[layer, at:at + n] = s
        if case["order"] == "nhd":
            codes = codes.transpose(2, 3).contiguous()
        out += [codes, scale]
    return out


def _ragged(batch, most, dev):
    """Lengths from about a third of `most` to `most`: the same ones for every seed, which only orders them."""
    i = torch.arange(batch, device=dev, dtype=torch.float64)
    return (most * (1.0 - 0.65 * i / batch)).long().clamp(min=1)


def _tables(lens, page, width, pages, gen, dev):
    """Page table of sequences of these lengths on pages in shuffled order, -1 behind the last."""
    need = (lens + page - 1) // page
    cols = torch.arange(width, device=dev)
    held = cols[None, :] < need[:, None]
    order = torch.randperm(pages, device=dev, generator=gen)
    table = torch.full((lens.numel(), width), -1, dtype=torch.int32, device=dev)
    table[held] = order[:int(held.sum())].int()
    return table


def _own_cache(s):
    from block_quantised_weight_gb300 import qgkv
    c = s["case"]
    return qgkv.KVCache(s["k"], s["k_scale"], s["v"], s["v_scale"], fmt=c["fmt"], order=c["order"])


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 17)
    s = {"case": case}
    op = case["op"]
    if op == "beam":
        rows = case["requests"] * case["beams"]
        x = torch.randn((rows, case["vocab"]), device=dev, generator=gen) * 2.5
        top = torch.randint(0, case["vocab"], (rows, 40), device=dev, generator=gen)
        x.scatter_add_(1, top, 6.0 * torch.rand((rows, 40), device=dev, generator=gen))
        x[:, :3] = -math.inf  # tokens that are not to be produced
        s["logits"] = x.to(getattr(torch, case["dtype"]))
        s["cum"] = -torch.rand((case["requests"], case["beams"]), device=dev, generator=gen) * 4.0 - 3.0
    elif op == "fork":
        page, beams = case["page"], case["beams"]
        turn = torch.randperm(case["requests"], device=dev, generator=gen)
        prompt = _ragged(case["requests"], case["context"], dev)[turn]
        lens = prompt + 1 + turn * 7919 % (case["context"] // 2 + 2)  # tokens produced so far
        lens = lens.repeat_interleave(beams)
        shared = (prompt // page).repeat_interleave(beams)  # whole prompt pages, held by all beams of a request
        width = (int(lens.max()) + page - 1) // page + 1
        cols = torch.arange(width, device=dev)
        held = cols[None, :] < ((lens + page - 1) // page)[:, None]
        first = (torch.arange(lens.numel(), device=dev) // beams * beams)[:, None]
        mine = held & ((cols[None, :] >= shared[:, None]) | (torch.arange(lens.numel(), device=dev)[:, None] == first))
        used = int(mine.sum())
        pages = used + lens.numel() + 5
        order = torch.randperm(pages, device=dev, generator=gen)[:used].int()
        table = torch.full((lens.numel(), width), -1, dtype=torch.int32, device=dev)
        table[mine] = order
        table = torch.where(held & ~mine, table[first[:, 0]], table)
        refs = torch.bincount(table[held].long(), minlength=pages).int()
        pick = torch.randint(0, beams, (lens.numel(),), device=dev, generator=gen)
        s.update(table=table, lens=lens.int(), refs=refs, parent=(first[:, 0] + pick).int())
        s["k"], s["k_scale"], s["v"], s["v_scale"] = _make_cache(case, case["layers"], pages, gen, dev)
    elif op == "compact":
        lens = _ragged(case["batch"], case["context"], dev)[torch.randperm(case["batch"], device=dev, generator=gen)]
        width = (case["context"] + case["page"] - 1) // case["page"]
        table = _tables(lens, case["page"], width, case["pages"], gen, dev)
        drop = torch.rand(case["batch"], device=dev, generator=gen) < 0.4
        refs = torch.bincount(table[table >= 0].long(), minlength=case["pages"]).int()
        s.update(table=table, lens=lens.int(), refs=refs, drop=drop)
        s["k"], s["k_scale"], s["v"], s["v_scale"] = _make_cache(case, case["layers"], case["pages"], gen, dev)
    else:
        dtype = getattr(torch, case["dtype"])
        turn = torch.randperm(case["batch"], device=dev, generator=gen)
        lens = _ragged(case["batch"], case["context"], dev)[turn]
        rows = torch.ones_like(lens)
        if case["rows"] > 1:
            rows = _ragged(case["batch"], case["rows"], dev).flip(0)[turn]
            rows = torch.minimum(rows, lens) if op == "attn" else rows
        starts = torch.zeros(case["batch"] + 1, dtype=torch.int32, device=dev)
        starts[1:] = rows.cumsum(0)
        total, after = int(rows.sum()), lens if op == "attn" else lens + rows
        width = (int(after.max()) + case["page"] - 1) // case["page"]
        pages = int(((after + case["page"] - 1) // case["page"]).sum()) + 3
        s.update(table=_tables(after, case["page"], width, pages, gen, dev), lens=lens.int(),
                 starts=None if case["rows"] == 1 else starts, most_rows=int(rows.max()))
        s["k"], s["k_scale"], s["v"], s["v_scale"] = _make_cache(case, 1, pages, gen, dev)
        if op == "attn":
            s["q"] = (torch.randn((total, case["q_heads"], case["dim"]), device=dev, generator=gen) * 1.5).to(dtype)
        else:
            # K and V come as two parts of one projection's output; a few tokens are larger than what is held
            kv = _fill((total, 2, case["heads"], case["dim"]), gen, dev)
            kv = kv * (1.0 + 3.0 * (torch.rand((total, 1, 1, 1), device=dev, generator=gen) < 0.1))
            s["kv"] = kv.to(dtype)
    if own:
        from block_quantised_weight_gb300 import qgkv
        if op != "beam":
            s["cache"] = _own_cache(s)
        s["workspace"] = qgkv.KVWorkspace(dev)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _run_own(s):
    from block_quantised_weight_gb300 import qgkv
    op, w = s["case"]["op"], s["workspace"]
    if op == "attn":
        return qgkv.kv_attention(s["cache"], 0, s["q"], s["table"], s["lens"], starts=s["starts"], return_lse=True,
                                 workspace=w)
    if op == "append":
        qgkv.kv_append(s["cache"], 0, s["kv"][:, 0], s["kv"][:, 1], s["table"], s["lens"], starts=s["starts"])
        return _state(s)
    if op == "fork":
        return qgkv.kv_fork(s["cache"], s["table"], s["lens"], s["parent"], s["refs"], workspace=w), _state(s)
    if op == "compact":
        return qgkv.kv_compact(s["cache"], s["table"], s["lens"], s["refs"], drop=s["drop"], workspace=w), _state(s)
    return qgkv.beam_select(s["logits"], s["cum"], s["case"]["keep"], workspace=w)


def _state(s):
    f = s["case"]["fmt"]
    return _codes_as_values(s["k"], f), s["k_scale"], _codes_as_values(s["v"], f), s["v_scale"]


def _held(s, name):
    """Dequantised [batch, heads, width * page, dim] of every sequence's pages, zero behind its length."""
    c = s["case"]
    page = s["table"].clamp(min=0).long()
    x = _codes_as_values(s[name][0], c["fmt"])[page].float()
    if c["order"] == "nhd":
        x = x.transpose(2, 3)
    x = (x * s[name + "_scale"][0][page][..., None, None]).transpose(1, 2)
    x = x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])
    pos = torch.arange(x.shape[2], device=x.device)
    return torch.where(pos[None, None, :, None] < s["lens"][:, None, None, None], x, 0.0)


def _attn_plain(s):
    c = s["case"]
    q, lens = s["q"], s["lens"].long()
    batch, heads, dim = c["batch"], c["heads"], c["dim"]
    group, most = c["q_heads"] // heads, s["most_rows"]
    if s["starts"] is None:
        at = torch.arange(batch, device=q.device)
        rows = torch.ones_like(at)
    else:
        at = s["starts"][:-1].long()
        rows = s["starts"][1:].long() - at
    i = torch.arange(most, device=q.device)
    real = i[None, :] < rows[:, None]
    idx = torch.where(real, at[:, None] + i[None, :], 0)
    x = q[idx].float().view(batch, most, heads, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, heads, group * most, dim)
    k, v = _held(s, "k"), _held(s, "v")
    score = (x @ k.transpose(2, 3) / math.sqrt(dim)).view(batch, heads, group, most, -1)
    last = lens[:, None] - rows[:, None] + i[None, :]  # the last position that row i sees
    seen = torch.arange(score.shape[-1], device=q.device)[None, None, :] <= last[:, :, None]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    m = score.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(score - m)
    total = e.sum(-1, keepdim=True)
    o = (e.view(batch, heads, group * most, -1) @ v).view(batch, heads, group, most, dim)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + torch.log(total))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, most, c["q_heads"], dim)
    lse = lse.permute(0, 3, 1, 2).reshape(batch, most, c["q_heads"])
    return o[real].to(q.dtype), lse[real]


def _append_plain(s):
    """Blocks that the new tokens touch, as [touched, page] tokens: old codes are rescaled where the scale grows."""
    c = s["case"]
    fmt, page, batch = c["fmt"], c["page"], c["batch"]
    lens = s["lens"].long()
    if s["starts"] is None:
        at = torch.arange(batch, device=lens.device)
        rows = torch.ones_like(at)
    else:
        at = s["starts"][:-1].long()
        rows = s["starts"][1:].long() - at
    slots = (s["most_rows"] + 2 * page - 2) // page
    slot = lens[:, None] // page + torch.arange(slots, device=lens.device)[None, :]
    touched = (slot * page < (lens + rows)[:, None]) & (rows > 0)[:, None]
    seq, which = touched.nonzero(as_tuple=True)
    slot = slot[seq, which]
    pid = s["table"][seq, slot].long()
    pos = slot[:, None] * page + torch.arange(page, device=lens.device)[None, :]
    old = pos < lens[seq][:, None]
    new = ~old & (pos < (lens + rows)[seq][:, None])
    row = torch.where(new, at[seq][:, None] + pos - lens[seq][:, None], 0)
    for part, name in enumerate(("k", "v")):
        x = s["kv"][:, part][row].float().transpose(1, 2)  # [touched, heads, page, dim]
        x = torch.where(new[:, None, :, None], x, 0.0)
        codes = s[name][0][pid]
        codes = codes.transpose(1, 2) if c["order"] == "nhd" else codes
        need = _scale_for(torch.where(x.isfinite(), x.abs(), 0.0).amax(dim=(2, 3)), fmt)
        was = torch.where(old.any(1)[:, None], s[name + "_scale"][0][pid], 0.0)
        now = torch.maximum(was, need)
        grown = torch.where(now > was, was / torch.where(now > 0, now, 1.0), 1.0)[..., None, None]
        again = _codes_as_values(codes.contiguous(), fmt).float() * grown
        if fmt == "e4m3":
            again = again.to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            again = again.round().to(torch.int8).view(torch.uint8)
        fresh = _quantise(x, now[..., None, None], fmt)
        put = torch.where(new[:, None, :, None], fresh, torch.where((old[:, None, :, None]) & (grown != 1.0), again, codes))
        s[name][0][pid] = put.transpose(1, 2) if c["order"] == "nhd" else put
        s[name + "_scale"][0][pid] = now
    return _state(s)


def _move_plain(s, src, dst):
    for name in ("k", "k_scale", "v", "v_scale"):
        s[name][:, dst] = s[name][:, src]


def _fork_plain(s):
    page, lens, table, refs = s["case"]["page"], s["lens"].long(), s["table"], s["refs"]
    parent = s["parent"].long()
    cols = torch.arange(table.shape[1], device=table.device)[None, :]
    held = cols < ((lens + page - 1) // page)[:, None]
    lens2, held2 = lens[parent], held[parent]
    table2 = torch.where(held2, table[parent], -1)
    refs2 = refs - torch.bincount(table[held].long(), minlength=refs.numel()) \
        + torch.bincount(table2[held2].long(), minlength=refs.numel())
    part = lens2 % page != 0
    last = (lens2 // page).clamp(max=table.shape[1] - 1)
    tail = table2.gather(1, last[:, None])[:, 0].long()
    same = (tail[:, None] == tail[None, :]) & part[:, None] & part[None, :]
    n = torch.arange(lens2.numel(), device=table.device)
    keeper = torch.where(same, n[None, :], lens2.numel()).amin(1) == n
    outside = refs2[tail.clamp(min=0)] > same.sum(1)
    copied = part & (outside | ~keeper)
    rank = copied.cumsum(0) - 1
    fresh = torch.sort((refs2 != 0).int(), stable=True)[1][rank.clamp(min=0)]  # free pages, lowest first
    src, dst, row = tail[copied], fresh[copied], n[copied]
    table2[row, last[copied]] = dst.int()
    refs2 = refs2 - torch.bincount(src, minlength=refs.numel()) + torch.bincount(dst, minlength=refs.numel())
    _move_plain(s, src, dst)
    return (table2, lens2.int(), refs2.int()), _state(s)


def _compact_plain(s):
    page, table, drop = s["case"]["page"], s["table"], s["drop"]
    lens = torch.where(drop, 0, s["lens"].long())
    cols = torch.arange(table.shape[1], device=table.device)[None, :]
    was = cols < ((s["lens"].long() + page - 1) // page)[:, None]
    gone = was & drop[:, None]
    pages = s["refs"].numel()
    refs = s["refs"] - torch.bincount(table[gone].long(), minlength=pages)
    live = refs > 0
    count = live.sum()
    at = torch.arange(pages, device=table.device)
    src = (live & (at >= count)).nonzero()[:, 0]
    dst = (~live & (at < count)).nonzero()[:, 0]
    to = at.clone()
    to[src] = dst
    held = was & ~gone
    table2 = torch.where(held, to[table.clamp(min=0).long()], -1).int()
    refs2 = torch.zeros_like(refs)
    refs2[to[live]] = refs[live]
    _move_plain(s, src, dst)
    return (table2, lens.int(), refs2.int(), count.int().reshape(1)), _state(s)


def _beam_plain(s):
    c = s["case"]
    x = s["logits"].double()
    m = x.amax(-1, keepdim=True)
    lse = m + torch.log(torch.exp(x - m).sum(-1, keepdim=True))  # 64 bits: neighbours in the order may be close
    score = (s["cum"].double().view(-1, 1) + (x - lse)).view(c["requests"], -1)
    top, at = torch.sort(score, dim=-1, descending=True, stable=True)
    top, at = top[:, :c["keep"]], at[:, :c["keep"]]
    first = torch.arange(c["requests"], device=x.device)[:, None] * c["beams"]
    return top.float(), (at % c["vocab"]).int(), (first + at // c["vocab"]).int()


_PLAIN = {"attn": _attn_plain, "append": _append_plain, "fork": _fork_plain, "compact": _compact_plain,
          "beam": _beam_plain}


# ---------------------------------------------------------------- what a pass cannot do without

def _mean_tokens(case, most):
    return max(1.0, 0.675 * (case["batch"] - 1) * most + most)


def work(case):
    op = case["op"]
    if op == "beam":
        rows = case["requests"] * case["beams"]
        size = 4 if case["dtype"] == "float32" else 2
        return {"bytes": rows * case["vocab"] * size + rows * 4 + case["requests"] * case["keep"] * 12,
                "flops": 4.0 * rows * case["vocab"]}
    size = 4 if case.get("dtype") == "float32" else 2
    token = case["heads"] * case["dim"] * 2  # codes of one token, K and V
    if op == "attn":
        tokens = _mean_tokens(case, case["context"])
        rows = _mean_tokens(case, case["rows"]) if case["rows"] > 1 else case["batch"]
        seen = tokens / case["batch"] - (rows / case["batch"] - 1) / 2  # of the mean row
        b = tokens * token + tokens / case["page"] * (case["heads"] * 8 + 4) \
            + rows * case["q_heads"] * (case["dim"] * 2 * size + 4)
        return {"bytes": b, "flops": 4.0 * rows * case["q_heads"] * case["dim"] * max(seen, 1.0)}
    if op == "append":
        rows = _mean_tokens(case, case["rows"]) if case["rows"] > 1 else case["batch"]
        blocks = rows / case["page"] + case["batch"]
        return {"bytes": rows * token * (size + 1) + blocks * case["heads"] * 16, "flops": 3.0 * rows * token}
    moved = case["layers"] * case["heads"] * (case["page"] * case["dim"] * 2 + 8) * 2  # one page, read and written
    if op == "fork":
        rows = case["requests"] * case["beams"]
        width = case["context"] / case["page"]
        again = (1.0 - 1.0 / case["beams"]) ** case["beams"]  # share of rows that are not a parent's first child
        return {"bytes": rows * again * (1 - 1.0 / case["page"]) * moved + rows * width * 8 + rows * width * 8,
                "flops": 0.0}
    used = case["batch"] * (0.675 * case["context"] / case["page"] + 0.5)
    live = 0.6 * used
    holes = live * max(0.0, 1.0 - live / case["pages"])
    return {"bytes": holes * moved + used * 8 + case["pages"] * 8, "flops": 0.0}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"attn": _attn_exact, "append": _append_exact, "beam": _beam_exact}.get(case["op"], lambda s: None)(s)


def _tokens(s, name, b, n):
    """K or V of the first n tokens of sequence b, [n, heads, dim], in 64 bits."""
    c = s["case"]
    ids = s["table"][b, :(n + c["page"] - 1) // c["page"]].tolist()
    codes = _codes_as_values(s[name][0, ids], c["fmt"]).double()
    scale = s[name + "_scale"][0, ids].double()
    if c["order"] == "hnd":
        codes = codes.permute(0, 2, 1, 3)
    return (codes * scale[:, None, :, None]).flatten(0, 1)[:n]


def _attn_exact(s):
    c = s["case"]
    if 4.0 * c["batch"] * c["rows"] * c["q_heads"] * c["dim"] * c["context"] > 3e12:
        return None
    group = c["q_heads"] // c["heads"]
    lens = s["lens"].tolist()
    starts = list(range(c["batch"] + 1)) if s["starts"] is None else s["starts"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=s["q"].device)
    lse = torch.full(s["q"].shape[:2], -math.inf, dtype=torch.float64, device=s["q"].device)
    for b in range(c["batch"]):
        n, rows = lens[b], starts[b + 1] - starts[b]
        k, v = _tokens(s, "k", b, n), _tokens(s, "v", b, n)
        sees = torch.arange(n - rows, n, device=k.device)
        hidden = torch.arange(n, device=k.device)[None, :] > sees[:, None]
        for h in range(c["q_heads"]):
            score = s["q"][starts[b]:starts[b + 1], h].double() @ k[:, h // group].T * c["dim"] ** -0.5
            score[hidden] = -math.inf
            lse[starts[b]:starts[b + 1], h] = torch.logsumexp(score, 1)
            out[starts[b]:starts[b + 1], h] = torch.softmax(score, 1) @ v[:, h // group]
    return out, lse


def _round_e4m3(x):
    """Nearest e4m3 value, ties to even, of 64-bit values within +-448."""
    e = torch.frexp(x.abs())[1].long() - 1
    step = (e.clamp(min=-6) - 3 + 1023 << 52).view(torch.float64)
    return torch.round(x / step) * step


def _append_exact(s):
    """Sequence by sequence and block by block; the block scale is held in fp32, the codes follow from it."""
    c = s["case"]
    fmt, page = c["fmt"], c["page"]
    lens = s["lens"].tolist()
    starts = list(range(c["batch"] + 1)) if s["starts"] is None else s["starts"].tolist()
    table = s["table"].tolist()
    outs = []
    for part, name in enumerate(("k", "v")):
        codes = _codes_as_values(s[name], fmt).double()
        scale = s[name + "_scale"].clone()
        heads_first = codes if c["order"] == "hnd" else codes.transpose(2, 3)
        for b in range(c["batch"]):
            at, end = lens[b], lens[b] + starts[b + 1] - starts[b]
            while at < end:
                pid, off = table[b][at // page], at % page
                n = min(page - off, end - at)
                r = starts[b] + at - lens[b]
                x = s["kv"][r:r + n, part].double().transpose(0, 1)
                a = x.abs().amax(dim=(1, 2))
                if fmt == "e4m3":
                    frac, up = torch.frexp((a / torch.full_like(a, 448.0)).clamp(min=2.0 ** -126))
                    up = up.long() - (frac == 0.5).long()  # the lowest power of two that is not below a / 448
                    need = torch.where(a > 0, (up + 1023 << 52).view(torch.float64), 0.0)
                else:
                    need = (a / torch.full_like(a, 127.0)).float().double()
                was = scale[0, pid].double() if off else torch.zeros_like(need)
                now = torch.maximum(was, need)
                live = torch.where(now > 0, now, 1.0)[:, None, None]
                block = heads_first[0, pid]
                if off:
                    ratio = (was / torch.where(now > 0, now, 1.0)).float().double()[:, None, None]
                    moved = (block[:, :off] * ratio).float().double()
                    moved = _round_e4m3(moved) if fmt == "e4m3" else torch.round(moved)
                    block[:, :off] = torch.where((now > was)[:, None, None], moved, block[:, :off])
                y = (x / live).float().double()
                block[:, off:off + n] = _round_e4m3(y) if fmt == "e4m3" else torch.round(y)
                scale[0, pid] = now.float()
                at += n
        outs += [codes if fmt == "e4m3" else None, scale.double()]
    return tuple(outs)


def _beam_exact(s):
    c = s["case"]
    x = s["logits"].double()
    score = (torch.log_softmax(x, -1) + s["cum"].double().reshape(-1, 1)).view(c["requests"], -1)
    return torch.topk(score, c["keep"], dim=-1)[0], None, None
