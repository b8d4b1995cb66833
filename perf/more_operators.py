"""Cases of the operators around a decode step: the append that rotates keys and
queries to their positions, the attention of sequences that share a prefix, and
the adjustment of logits before the selection.

``run`` computes one pass of a case either in plain torch operations
(``own = False``) or through the entry points of
``block_quantised_weight_gb300.qgkv`` (``own = True``).

The cache is the one of ``qgkv``: 8-bit codes in pages, one fp32 scale for each
(layer, page, head) of K and of V; a sequence is a row of a page table and a
length.  Sequences of a group hold the same pages in their first columns.
"""
import math

import torch

own = False

E4M3_MAX = 448.0


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one token for each sequence of a decode batch on the TinyLlama-1.1B head shape
        dict(name="rotary_step", op="rotary", batch=48, q_heads=32, heads=4, dim=64, turned=64, page=64, context=2000,
             rows=1, fmt="e4m3", dtype="float32", order="hnd", pairs="interleaved"),
        # verification chunks of a draft, heads turned in part, odd sizes
        dict(name="rotary_chunk", op="rotary", batch=7, q_heads=12, heads=4, dim=96, turned=32, page=32, context=501,
             rows=131, fmt="int8", dtype="float16", order="hnd", pairs="halves"),
        # prompts stored after their chunk's projections, head shape of an 8B model
        dict(name="rotary_prompt", op="rotary", batch=5, q_heads=32, heads=8, dim=128, turned=128, page=64, context=900,
             rows=4001, fmt="e4m3", dtype="bfloat16", order="nhd", pairs="halves"),
        # four beams of one request through all layers of one step: short, latency is all that counts
        dict(name="shared_beams", op="shared", groups=1, members=4, q_heads=32, heads=4, dim=64, page=64, prefix=777,
             tail=40, rows=1, layers=22, fmt="e4m3", dtype="float32", order="hnd"),
        # a decode batch behind one long system prompt
        dict(name="shared_batch", op="shared", groups=1, members=48, q_heads=32, heads=8, dim=128, page=64, prefix=8200,
             tail=600, rows=1, layers=2, fmt="e4m3", dtype="bfloat16", order="hnd"),
        # beams of many requests, prompts of different lengths
        dict(name="shared_requests", op="shared", groups=24, members=8, q_heads=32, heads=4, dim=64, page=16,
             prefix=3501, tail=300, rows=1, layers=2, fmt="e4m3", dtype="float16", order="hnd"),
        # answers sampled in parallel about two long documents
        dict(name="shared_document", op="shared", groups=2, members=16, q_heads=32, heads=8, dim=128, page=128,
             prefix=65536, tail=900, rows=1, layers=1, fmt="int8", dtype="bfloat16", order="nhd"),
        # one request's beams under a grammar
        dict(name="logits_one", op="logits", requests=1, beams=4, vocab=32000, history=333, repetition=True,
             counts=False, listed=0, temperature=False, mask=True, dtype="float32"),
        # a sampling batch without a grammar, logits in 16 bits
        dict(name="logits_sampled", op="logits", requests=96, beams=1, vocab=50257, history=1500, repetition=False,
             counts=True, listed=64, temperature=True, mask=False, dtype="bfloat16"),
        # beams of a batch with everything, a larger vocabulary of odd size
        dict(name="logits_batch", op="logits", requests=48, beams=8, vocab=128257, history=2500, repetition=True,
             counts=True, listed=100, temperature=True, mask=True, dtype="float32"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the ranges of listed(): any operator, sizes spread over their logarithm."""
    op = rng.choice(["rotary", "shared", "shared", "logits"])
    fmt, order = rng.choice(["e4m3", "int8"]), rng.choice(["hnd", "nhd"])
    page = rng.choice([16, 32, 64, 128])
    dtype = rng.choice(["float32", "bfloat16", "float16"])
    heads, dim, group = rng.choice([1, 2, 4, 8]), rng.choice([64, 64, 80, 96, 128, 128, 256]), rng.choice([1, 3, 4, 4, 8])
    if op == "rotary":
        turned, pairs = rng.choice([dim, dim, dim // 32 * 16, 32]), rng.choice(["interleaved", "halves"])
        while True:
            batch, context, rows = _log(rng, 1, 96), _log(rng, 1, 4000), rng.choice([1, _log(rng, 1, 4001)])
            if batch * rows * heads * dim * (2 + group) <= 5 * 4001 * 8 * 128 * 6 and batch * (context + rows) <= 150000:
                return dict(op=op, batch=batch, q_heads=heads * group, heads=heads, dim=dim, turned=turned, page=page,
                            context=context, rows=rows, fmt=fmt, dtype=dtype, order=order, pairs=pairs)
    if op == "shared":
        while True:
            groups, members, layers = _log(rng, 1, 32), _log(rng, 2, 64), _log(rng, 1, 22)
            prefix, tail, rows = _log(rng, 16, 65536), _log(rng, 1, 1500), rng.choice([1, 1, 1, rng.randint(2, 8)])
            seen = groups * members * (prefix + tail) * heads * dim
            if seen * layers <= 32 * 66436 * 8 * 128 and seen * layers * rows * group <= 32 * 66436 * 8 * 128 * 4:
                return dict(op=op, groups=groups, members=members, q_heads=heads * group, heads=heads, dim=dim,
                            page=page, prefix=prefix, tail=tail, rows=rows, layers=layers, fmt=fmt, dtype=dtype,
                            order=order)
    while True:
        requests, beams, vocab = _log(rng, 1, 200), rng.choice([1, 1, 2, 4, 5, 8]), _log(rng, 500, 160000)
        history = _log(rng, 1, 8000)
        if requests * beams * vocab <= 48 * 8 * 128257:
            flags = [rng.random() < 0.6 for _ in range(4)]
            if not any(flags):
                flags[0] = True
            return dict(op=op, requests=requests, beams=beams, vocab=vocab, history=history, repetition=flags[0],
                        counts=flags[1], listed=rng.choice([0, _log(rng, 1, 300)]), temperature=flags[2],
                        mask=flags[3], dtype=dtype)


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


def _starts(rows):
    starts = torch.zeros(rows.numel() + 1, dtype=torch.int32, device=rows.device)
    starts[1:] = rows.cumsum(0)
    return starts


def _prepare_rotary(case, gen, dev):
    dtype = getattr(torch, case["dtype"])
    turn = torch.randperm(case["batch"], device=dev, generator=gen)
    lens = _ragged(case["batch"], case["context"], dev)[turn]
    rows = torch.ones_like(lens)
    if case["rows"] > 1:
        rows = _ragged(case["batch"], case["rows"], dev).flip(0)[turn]
    need = (lens + rows + case["page"] - 1) // case["page"]
    width, pages, total = int(need.max()), int(need.sum()) + 3, int(rows.sum())
    held = torch.arange(width, device=dev)[None, :] < need[:, None]
    table = torch.full((case["batch"], width), -1, dtype=torch.int32, device=dev)
    table[held] = torch.randperm(pages, device=dev, generator=gen)[:int(held.sum())].int()
    s = {"table": table, "lens": lens.int(), "starts": None if case["rows"] == 1 else _starts(rows),
         "most_rows": int(rows.max())}
    s["k"], s["k_scale"], s["v"], s["v_scale"] = _make_cache(case, 1, pages, gen, dev)
    # q, K and V are parts of one projection's output; a few tokens are larger than what is held
    x = _fill((total, case["q_heads"] + 2 * case["heads"], case["dim"]), gen, dev)
    s["qkv"] = (x * (1.0 + 3.0 * (torch.rand((total, 1, 1), device=dev, generator=gen) < 0.1))).to(dtype)
    # cosines and sines of every position, angles in 64 bits
    half = case["turned"] // 2
    freq = 10000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
    angle = torch.arange(case["context"] + case["rows"], device=dev, dtype=torch.float64)[:, None] * freq
    s["rope"] = torch.cat((torch.cos(angle), torch.sin(angle)), dim=1).float()
    return s


def _prepare_shared(case, gen, dev):
    groups, members, page = case["groups"], case["members"], case["page"]
    batch = groups * members
    prefix = _ragged(groups, case["prefix"], dev)[torch.randperm(groups, device=dev, generator=gen)]
    prefix = prefix.repeat_interleave(members)
    tail = _ragged(batch, case["tail"], dev)[torch.randperm(batch, device=dev, generator=gen)]
    lens = prefix + tail
    rows = tail.clamp(max=case["rows"])
    need = (lens + page - 1) // page
    width = int(need.max())
    cols, seq = torch.arange(width, device=dev)[None, :], torch.arange(batch, device=dev)[:, None]
    held = cols < need[:, None]
    first = seq // members * members
    mine = held & ((cols >= (prefix // page)[:, None]) | (seq == first))  # whole pages of the prefix are the first's
    pages = int(mine.sum()) + 3
    table = torch.full((batch, width), -1, dtype=torch.int32, device=dev)
    table[mine] = torch.randperm(pages, device=dev, generator=gen)[:pages - 3].int()
    table = torch.where(held & ~mine, table[first[:, 0]], table)
    s = {"table": table, "lens": lens.int(), "starts": None if case["rows"] == 1 else _starts(rows),
         "groups": torch.arange(groups + 1, dtype=torch.int32, device=dev) * members, "most_rows": int(rows.max())}
    s["k"], s["k_scale"], s["v"], s["v_scale"] = _make_cache(case, case["layers"], pages, gen, dev)
    q = torch.randn((case["layers"], int(rows.sum()), case["q_heads"], case["dim"]), device=dev, generator=gen)
    s["q"] = (q * 1.5).to(getattr(torch, case["dtype"]))
    return s


def _prepare_logits(case, gen, dev):
    rows, vocab = case["requests"] * case["beams"], case["vocab"]
    x = torch.randn((rows, vocab), device=dev, generator=gen) * 2.5
    top = torch.randint(0, vocab, (rows, 40), device=dev, generator=gen)
    x.scatter_add_(1, top, 6.0 * torch.rand((rows, 40), device=dev, generator=gen))
    s = {"logits": x.to(getattr(torch, case["dtype"]))}

    def uniform(lo, hi):
        return lo + (hi - lo) * torch.rand(rows, device=dev, generator=gen)

    history = lens = prompt = None
    if case["repetition"] or case["counts"]:
        # frequent tokens come again: the square puts half of a history on a quarter of the vocabulary
        at = torch.rand((rows, case["history"]), device=dev, generator=gen) ** 2
        history = (at * vocab).int().clamp(max=vocab - 1)
        lens = _ragged(rows, case["history"], dev)[torch.randperm(rows, device=dev, generator=gen)].int()
        prompt = lens // 3
    s.update(history=history, lens=lens, prompt=prompt)
    s["repetition"] = uniform(1.0, 1.4) if case["repetition"] else None
    s["presence"] = uniform(0.0, 0.8) if case["counts"] else None
    s["frequency"] = uniform(0.0, 0.5) if case["counts"] else None
    s["bias_tokens"] = s["bias"] = None
    if case["listed"]:
        n = min(case["listed"], vocab)
        order = torch.rand((rows, vocab), device=dev, generator=gen).topk(n, dim=1)[1]  # no token twice
        room = torch.arange(n, device=dev)[None, :] < _ragged(rows, n, dev)[:, None]
        s["bias_tokens"] = torch.where(room, order, -1).int()
        s["bias"] = torch.randn((rows, n), device=dev, generator=gen) * 4.0
    s["temperature"] = uniform(0.5, 1.3) if case["temperature"] else None
    s["mask"] = s["mask_rows"] = None
    if case["mask"]:
        words = (vocab + 31) // 32
        # one mask a request; a grammar leaves few tokens or most of them
        dense = torch.randint(-2**31, 2**31, (2, case["requests"], words), device=dev, generator=gen).int()
        few = (torch.rand((case["requests"], 1), device=dev, generator=gen) < 0.5)
        s["mask"] = torch.where(few, dense[0] & dense[1] & dense[0].roll(7, 1) & dense[1].roll(5, 1), dense[0] | dense[1])
        s["mask_rows"] = (torch.arange(rows, device=dev) // case["beams"]).int()
    return s


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 29)
    make = {"rotary": _prepare_rotary, "shared": _prepare_shared, "logits": _prepare_logits}[case["op"]]
    s = {"case": case, **make(case, gen, dev)}
    if own and case["op"] != "logits":
        from block_quantised_weight_gb300 import qgkv
        s["cache"] = qgkv.KVCache(s["k"], s["k_scale"], s["v"], s["v_scale"], fmt=case["fmt"], order=case["order"])
        s["workspace"] = qgkv.KVWorkspace(dev)
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return _run_own(s) if own else _PLAIN[s["case"]["op"]](s)


def _parts(s):
    """q, k and v of the projection's output."""
    c = s["case"]
    a, b = c["q_heads"], c["q_heads"] + c["heads"]
    return s["qkv"][:, :a], s["qkv"][:, a:b], s["qkv"][:, b:]


def _run_own(s):
    from block_quantised_weight_gb300 import qgkv
    c = s["case"]
    if c["op"] == "rotary":
        q, k, v = _parts(s)
        turned = qgkv.kv_append_rotary(s["cache"], 0, q, k, v, s["rope"], s["table"], s["lens"], starts=s["starts"],
                                       pairs=c["pairs"])
        return (turned,) + _state(s)
    if c["op"] == "shared":
        plan = qgkv.kv_share(s["cache"], s["table"], s["lens"], s["groups"], starts=s["starts"])
        return plan, [qgkv.kv_attention_shared(s["cache"], i, s["q"][i], s["table"], s["lens"], plan, starts=s["starts"],
                                               return_lse=True, workspace=s["workspace"]) for i in range(c["layers"])]
    return qgkv.adjust_logits(s["logits"], history=s["history"], lens=s["lens"], prompt_lens=s["prompt"],
                              repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"],
                              bias_tokens=s["bias_tokens"], bias=s["bias"], temperature=s["temperature"],
                              mask=s["mask"], mask_rows=s["mask_rows"])


def _state(s):
    f = s["case"]["fmt"]
    return _codes_as_values(s["k"], f), s["k_scale"], _codes_as_values(s["v"], f), s["v_scale"]


def _spans(s):
    """First row and number of rows of each sequence."""
    if s["starts"] is None:
        at = torch.arange(s["lens"].numel(), device=s["lens"].device)
        return at, torch.ones_like(at)
    at = s["starts"][:-1].long()
    return at, s["starts"][1:].long() - at


def _turn(x, rope, pos, pairs):
    """x [rows, heads, dim] turned to the positions pos [rows]: products and their sum each rounded to 32 bits."""
    x = x.float()
    half = rope.shape[1] // 2
    cos, sin = rope[pos][:, None, :half], rope[pos][:, None, half:]
    if pairs == "interleaved":
        a, b = x[..., 0:2 * half:2], x[..., 1:2 * half:2]
    else:
        a, b = x[..., :half], x[..., half:2 * half]
    lo, hi = a * cos - b * sin, a * sin + b * cos
    y = torch.stack((lo, hi), -1).flatten(-2) if pairs == "interleaved" else torch.cat((lo, hi), -1)
    return torch.cat((y, x[..., 2 * half:]), -1)


def _append(s, name, values):
    """Values [rows, heads, dim] into the blocks that they touch; old codes are rescaled where the scale grows."""
    c = s["case"]
    fmt, page = c["fmt"], c["page"]
    lens = s["lens"].long()
    at, rows = _spans(s)
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
    x = torch.where(new[:, None, :, None], values[row].transpose(1, 2), 0.0)  # [touched, heads, page, dim]
    codes = s[name][0][pid]
    codes = codes.transpose(1, 2) if c["order"] == "nhd" else codes
    need = _scale_for(torch.where(x.isfinite(), x.abs(), 0.0).amax(dim=(2, 3)), fmt)
    was = torch.where(old.any(1)[:, None], s[name + "_scale"][0][pid], 0.0)
    now = torch.maximum(was, need)
    grown = torch.where(now > was, was / torch.where(now > 0, now, 1.0), 1.0)[..., None, None]
    again = _codes_as_values(codes.contiguous(), fmt).float() * grown
    again = again.to(torch.float8_e4m3fn) if fmt == "e4m3" else again.round().to(torch.int8)
    put = torch.where(old[:, None, :, None] & (grown != 1.0), again.view(torch.uint8), codes)
    put = torch.where(new[:, None, :, None], _quantise(x, now[..., None, None], fmt), put)
    s[name][0][pid] = put.transpose(1, 2) if c["order"] == "nhd" else put
    s[name + "_scale"][0][pid] = now


def _rotary_plain(s):
    c = s["case"]
    q, k, v = _parts(s)
    at, rows = _spans(s)
    pos = (s["lens"].long() - at).repeat_interleave(rows) + torch.arange(q.shape[0], device=q.device)
    _append(s, "k", _turn(k, s["rope"], pos, c["pairs"]))
    _append(s, "v", v.float())
    return (_turn(q, s["rope"], pos, c["pairs"]).to(q.dtype),) + _state(s)


def _plan_plain(s):
    """What the sequences of each group have in common: whole pages that all hold and every row sees.  int32:
    (first row, rows, tokens, first sequence) of each group, then the tokens for each sequence."""
    c = s["case"]
    at, rows = _spans(s)
    table = s["table"].view(c["groups"], c["members"], -1)
    same = (table == table[:, :1]).all(1).int().cumprod(1).sum(1)
    least = (s["lens"].long() - rows + 1).view(c["groups"], c["members"]).amin(1) // c["page"]
    tokens = torch.minimum(same, least) * c["page"]
    first = s["groups"][:-1].long()
    plan = torch.stack((at[first], rows.view(c["groups"], -1).sum(1), tokens, first), 1)
    return torch.cat((plan.flatten(), tokens.repeat_interleave(c["members"]))).int()


def _held(s, name, layer):
    """Dequantised [batch, heads, width * page, dim] of every sequence's pages, zero behind its length."""
    c = s["case"]
    page = s["table"].clamp(min=0).long()
    x = _codes_as_values(s[name][layer], c["fmt"])[page].float()
    if c["order"] == "nhd":
        x = x.transpose(2, 3)
    x = (x * s[name + "_scale"][layer][page][..., None, None]).transpose(1, 2)
    x = x.reshape(x.shape[0], x.shape[1], -1, x.shape[-1])
    pos = torch.arange(x.shape[2], device=x.device)
    return torch.where(pos[None, None, :, None] < s["lens"][:, None, None, None], x, 0.0)


def _attend(s, layer):
    c = s["case"]
    q, lens = s["q"][layer], s["lens"].long()
    batch, heads, dim = lens.numel(), c["heads"], c["dim"]
    group, most = c["q_heads"] // heads, s["most_rows"]
    at, rows = _spans(s)
    i = torch.arange(most, device=q.device)
    real = i[None, :] < rows[:, None]
    idx = torch.where(real, at[:, None] + i[None, :], 0)
    x = q[idx].float().view(batch, most, heads, group, dim).permute(0, 2, 3, 1, 4).reshape(batch, heads, group * most, dim)
    score = (x @ _held(s, "k", layer).transpose(2, 3) / math.sqrt(dim)).view(batch, heads, group, most, -1)
    last = lens[:, None] - rows[:, None] + i[None, :]  # the last position that row i sees
    seen = torch.arange(score.shape[-1], device=q.device)[None, None, :] <= last[:, :, None]
    score = score.masked_fill(~seen[:, None, None], -math.inf)
    m = score.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, 0.0, m)
    e = torch.exp(score - m)
    total = e.sum(-1, keepdim=True)
    o = (e.view(batch, heads, group * most, -1) @ _held(s, "v", layer)).view(batch, heads, group, most, dim)
    o = torch.where(total > 0, o / total, 0.0)
    lse = (m + torch.log(total))[..., 0]
    o = o.permute(0, 3, 1, 2, 4).reshape(batch, most, c["q_heads"], dim)
    lse = lse.permute(0, 3, 1, 2).reshape(batch, most, c["q_heads"])
    return o[real].to(q.dtype), lse[real]


def _shared_plain(s):
    return _plan_plain(s), [_attend(s, i) for i in range(s["case"]["layers"])]


def _logits_plain(s):
    x = s["logits"].float()
    if s["history"] is not None:
        col = torch.arange(s["history"].shape[1], device=x.device)[None, :]
        at = s["history"].long()
        there, fresh = col < s["lens"][:, None], col >= s["prompt"][:, None]
        zero = torch.zeros(x.shape, dtype=torch.int32, device=x.device)
        if s["repetition"] is not None:
            seen = zero.scatter_add(1, at, there.int()) > 0
            rho = s["repetition"][:, None]
            x = torch.where(seen, torch.where(x > 0, x / rho, x * rho), x)
        if s["presence"] is not None:
            n = zero.scatter_add(1, at, (there & fresh).int())
            x = torch.where(n > 0, x - s["frequency"][:, None] * n.float() - s["presence"][:, None], x)
    if s["bias"] is not None:
        at = s["bias_tokens"].long()
        add = torch.zeros_like(x).scatter_add(1, at.clamp(min=0), torch.where(at >= 0, s["bias"], 0.0))
        x = x + add
    if s["temperature"] is not None:
        x = x / s["temperature"][:, None]
    if s["mask"] is not None:
        bits = (s["mask"][:, :, None] >> torch.arange(32, device=x.device, dtype=torch.int32)) & 1
        allowed = bits.flatten(1)[:, :x.shape[1]].bool()[s["mask_rows"].long()]
        x = x.masked_fill(~allowed, -math.inf)
    return x.to(s["logits"].dtype)


_PLAIN = {"rotary": _rotary_plain, "shared": _shared_plain, "logits": _logits_plain}


# ---------------------------------------------------------------- what a pass cannot do without

def _mean(n, most):
    """Mean of _ragged(n, most)."""
    return max(1.0, most * (1.0 - 0.325 * (n - 1) / n))


def work(case):
    size = 4 if case["dtype"] == "float32" else 2
    if case["op"] == "logits":
        rows = case["requests"] * case["beams"]
        values = rows * case["vocab"]
        b = 2 * values * size + rows * case["listed"] * 8
        if case["repetition"] or case["counts"]:
            b += rows * _mean(rows, case["history"]) * 4
        if case["mask"]:
            b += case["requests"] * case["vocab"] / 8
        return {"bytes": b, "flops": 6.0 * values}
    token = case["heads"] * case["dim"] * 2  # codes of one token, K and V
    if case["op"] == "rotary":
        rows = case["batch"] * _mean(case["batch"], case["rows"]) if case["rows"] > 1 else case["batch"]
        blocks = rows / case["page"] + case["batch"]
        b = rows * (token * (size + 1) + case["q_heads"] * case["dim"] * 2 * size + case["turned"] * 4)
        return {"bytes": b + blocks * case["heads"] * 16, "flops": rows * (case["q_heads"] * case["dim"] * 3.0 + 5.0 * token)}
    batch = case["groups"] * case["members"]
    prefix, tail = _mean(case["groups"], case["prefix"]), _mean(batch, case["tail"])
    tokens = case["groups"] * prefix + batch * tail
    rows = batch * min(case["rows"], tail)
    b = tokens * token + tokens / case["page"] * (case["heads"] * 8 + 4) \
        + rows * case["q_heads"] * (case["dim"] * 2 * size + 4)
    return {"bytes": case["layers"] * b, "flops": 4.0 * case["layers"] * rows * case["q_heads"] * case["dim"] * (prefix + tail)}


# ---------------------------------------------------------------- the definition in 64 bits

def exact(case, seed):
    global own
    kept, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = kept
    return {"rotary": _rotary_exact, "shared": _shared_exact, "logits": _logits_exact}[case["op"]](s)


def _round_e4m3(x):
    """Nearest e4m3 value, ties to even, of 64-bit values within +-448."""
    e = torch.frexp(x.abs())[1].long() - 1
    step = (e.clamp(min=-6) - 3 + 1023 << 52).view(torch.float64)
    return torch.round(x / step) * step


def _turn_exact(x, rope, at, pairs):
    """x [n, heads, dim] of the positions at .. at + n - 1: a complex product for each pair."""
    x = x.double()
    half = rope.shape[1] // 2
    t = rope[at:at + x.shape[0]].double()
    z = torch.complex(t[:, :half], t[:, half:])[:, None]
    out = x.clone()
    if pairs == "interleaved":
        w = torch.view_as_complex(x[..., :2 * half].unflatten(-1, (half, 2)).contiguous()) * z
        out[..., :2 * half] = torch.view_as_real(w).flatten(-2)
    else:
        w = torch.complex(x[..., :half].contiguous(), x[..., half:2 * half].contiguous()) * z
        out[..., :half], out[..., half:2 * half] = w.real, w.imag
    return out


def _rotary_exact(s):
    """Sequence by sequence and block by block; the block scale is held in fp32, the codes follow from it."""
    c = s["case"]
    fmt, page = c["fmt"], c["page"]
    q, k, v = _parts(s)
    lens, table = s["lens"].tolist(), s["table"].tolist()
    starts = list(range(c["batch"] + 1)) if s["starts"] is None else s["starts"].tolist()
    turned = torch.empty(q.shape, dtype=torch.float64, device=q.device)
    outs = [turned]
    for name, part in (("k", k), ("v", v)):
        codes = _codes_as_values(s[name], fmt).double()
        scale = s[name + "_scale"].clone()
        heads_first = codes if c["order"] == "hnd" else codes.transpose(2, 3)
        for b in range(c["batch"]):
            r0, r1 = starts[b], starts[b + 1]
            if name == "k":
                turned[r0:r1] = _turn_exact(q[r0:r1], s["rope"], lens[b], c["pairs"])
                x_all = _turn_exact(part[r0:r1], s["rope"], lens[b], c["pairs"])
            else:
                x_all = part[r0:r1].double()
            at, end = lens[b], lens[b] + r1 - r0
            while at < end:
                pid, off = table[b][at // page], at % page
                n = min(page - off, end - at)
                x = x_all[at - lens[b]:at - lens[b] + n].transpose(0, 1)
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


def _shared_exact(s):
    """Each sequence by itself, as if nothing were shared."""
    c = s["case"]
    batch, group = c["groups"] * c["members"], c["q_heads"] // c["heads"]
    if 4.0 * c["layers"] * batch * c["rows"] * c["q_heads"] * c["dim"] * (c["prefix"] + c["tail"]) > 1.5e12:
        return None
    lens, table = s["lens"].tolist(), s["table"].tolist()
    starts = list(range(batch + 1)) if s["starts"] is None else s["starts"].tolist()
    done = []
    for layer in range(c["layers"]):
        q = s["q"][layer].double()
        out = torch.zeros_like(q)
        lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
        for b in range(batch):
            n, rows = lens[b], starts[b + 1] - starts[b]
            ids = table[b][:(n + c["page"] - 1) // c["page"]]
            kv = []
            for name in ("k", "v"):
                codes = _codes_as_values(s[name][layer, ids], c["fmt"]).double()
                codes = codes.transpose(1, 2) if c["order"] == "nhd" else codes
                codes = codes * s[name + "_scale"][layer, ids].double()[..., None, None]
                kv.append(codes.transpose(0, 1).flatten(1, 2)[:, :n])  # [heads, n, dim]
            x = q[starts[b]:starts[b + 1]].transpose(0, 1).unflatten(0, (c["heads"], group))
            score = torch.einsum("hgrd,hnd->hgrn", x, kv[0]) * c["dim"] ** -0.5
            hidden = torch.arange(n, device=q.device)[None, :] > torch.arange(n - rows, n, device=q.device)[:, None]
            score.masked_fill_(hidden, -math.inf)
            lse[starts[b]:starts[b + 1]] = torch.logsumexp(score, -1).flatten(0, 1).T
            o = torch.einsum("hgrn,hnd->hgrd", torch.softmax(score, -1), kv[1])
            out[starts[b]:starts[b + 1]] = o.flatten(0, 1).transpose(0, 1)
        done.append((out, lse))
    return None, done


def _logits_exact(s):
    """Row by row, and the listed tokens of each."""
    x = s["logits"].double()
    vocab = x.shape[1]
    for r in range(x.shape[0]):
        row = x[r]
        if s["history"] is not None:
            n, p = int(s["lens"][r]), int(s["prompt"][r])
            if s["repetition"] is not None:
                at = s["history"][r, :n].long().unique()
                rho = s["repetition"][r].double()
                row[at] = torch.where(row[at] > 0, row[at] / rho, row[at] * rho)
            if s["presence"] is not None:
                at, count = s["history"][r, p:n].long().unique(return_counts=True)
                row[at] -= s["frequency"][r].double() * count.double() + s["presence"][r].double()
        if s["bias"] is not None:
            at = s["bias_tokens"][r].long()
            row[at[at >= 0]] += s["bias"][r][at >= 0].double()
        if s["temperature"] is not None:
            row /= s["temperature"][r].double()
        if s["mask"] is not None:
            token = torch.arange(vocab, device=x.device)
            word = s["mask"][int(s["mask_rows"][r])][token // 32].long()
            row[(word >> token % 32) & 1 == 0] = -math.inf
    return x
