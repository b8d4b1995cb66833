"""GPU tests of a decode step's operators run together: pages reserved, keys turned and appended, attention over shared
pages, logits adjusted, beams selected and forked.  Each result of each step is held against what its own operator's tests
hold it to, with that step's inputs; a captured step is held against direct calls, bit for bit."""
import os
import sys
from types import SimpleNamespace

import pytest

torch = pytest.importorskip("torch")

from block_quantised_weight_gb300 import qgemv  # noqa: E402
from test_kv_gpu import DT, attention_ref, close, i32, kv, status_clean  # noqa: E402, F401
from test_kv_rotary_gpu import turned  # noqa: E402
from test_kv_shared_gpu import least_width, plan_ref, small  # noqa: E402
from test_logits_gpu import reference  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu

HEADS, GROUP, DIM, PAGE, VOCAB = 2, 4, 64, 16, 1000


def decoder(kv, requests, beams, prompts, dtype, fmt, pairs, pages=600, most=64):  # noqa: F811
    """One layer whose queries, keys and values are looked up, behind prompts that each request's beams share."""
    g = torch.Generator(device="cuda").manual_seed(requests + beams)
    rand = lambda *n: torch.randn(n, device="cuda", generator=g)  # noqa: E731
    s = SimpleNamespace(requests=requests, beams=beams, dtype=DT[dtype], pairs=pairs)
    s.ws = kv.KVWorkspace("cuda")
    s.cache = kv.KVCache.allocate(1, pages, HEADS, PAGE, DIM, fmt)
    s.refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    s.rope = kv.rotary_table(4096, 48)
    s.eq, s.ek, s.ev = (rand(VOCAB, h, DIM).to(s.dtype) for h in (HEADS * GROUP, HEADS, HEADS))
    s.head = 0.3 * rand(HEADS * GROUP * DIM, VOCAB)
    batch = requests * beams
    width = least_width(batch, HEADS, DIM, PAGE)
    table, lens = torch.full((requests, width), -1, dtype=torch.int32, device="cuda"), i32([0] * requests)
    said = [torch.randint(0, VOCAB, (n,), device="cuda", generator=g) for n in prompts]
    starts = [0]
    for n in prompts:
        starts.append(starts[-1] + n)
    kv.kv_reserve(s.cache, table, lens, s.refs, add=i32(prompts), workspace=s.ws)
    at = torch.cat(said)
    kv.kv_append_rotary(s.cache, 0, s.eq[at], s.ek[at], s.ev[at], s.rope, table, lens, starts=i32(starts), pairs=pairs)
    lens += i32(prompts)
    parent = i32([r for r in range(requests) for _ in range(beams)])
    s.table, s.lens, s.refs = kv.kv_fork(s.cache, table, lens, parent, s.refs, workspace=s.ws)
    s.groups = i32([beams * r for r in range(requests + 1)])
    s.history = torch.zeros((batch, max(prompts) + most), dtype=torch.int32, device="cuda")
    for r, x in enumerate(said):
        s.history[beams * r:beams * (r + 1), :len(x)] = x.int()
    s.said = i32([prompts[r] for r in range(requests) for _ in range(beams)])
    s.given = s.said.clone()
    s.rules = dict(repetition=0.8 + torch.rand(batch, device="cuda", generator=g), presence=0.2 * rand(batch),
                   frequency=0.1 * rand(batch), temperature=0.5 + torch.rand(batch, device="cuda", generator=g),
                   bias_tokens=torch.randint(0, VOCAB, (batch, 5), device="cuda", generator=g).int(), bias=rand(batch, 5),
                   mask=torch.randint(-2 ** 31, 2 ** 31, (2, 32), device="cuda", generator=g).int(),
                   mask_rows=i32([i % 3 - 1 for i in range(batch)]))
    s.tokens = torch.randint(0, VOCAB, (batch,), device="cuda", generator=g).int()
    s.cum = torch.zeros((requests, beams), device="cuda")
    return s


def step(kv, s):  # noqa: F811
    """One token for each beam; the state is updated in place.  Returns what the step worked out."""
    kv.kv_reserve(s.cache, s.table, s.lens, s.refs, workspace=s.ws)
    at = s.tokens.long()
    q = kv.kv_append_rotary(s.cache, 0, s.eq[at], s.ek[at], s.ev[at], s.rope, s.table, s.lens, pairs=s.pairs)
    s.lens += 1
    plan = kv.kv_share(s.cache, s.table, s.lens, s.groups)
    out, lse = kv.kv_attention_shared(s.cache, 0, q, s.table, s.lens, plan, return_lse=True, workspace=s.ws)
    s.history.scatter_(1, s.said[:, None].long(), s.tokens[:, None])
    s.said += 1
    logits = out.float().flatten(1) @ s.head
    adjusted = kv.adjust_logits(logits, history=s.history, lens=s.said, prompt_lens=s.given, **s.rules)
    scores, tokens, parents = kv.beam_select(adjusted, s.cum, s.beams, workspace=s.ws)
    seen = SimpleNamespace(**{n: x.clone() for n, x in dict(
        q=q, plan=plan, out=out, lse=lse, logits=logits, adjusted=adjusted, scores=scores, tokens=tokens, parents=parents).items()})
    # as they are before the fork, which copies onto pages that no child keeps
    c = s.cache
    seen.before = SimpleNamespace(at=at, **{n: getattr(s, n).clone() for n in ("table", "lens", "history", "said")})
    seen.cache = SimpleNamespace(heads=c.heads, page_tokens=c.page_tokens, fmt=c.fmt, order=c.order,
                                 **{n: getattr(c, n).clone() for n in ("k", "v", "k_scale", "v_scale")})
    table, lens, refs = kv.kv_fork(s.cache, s.table, s.lens, parents.view(-1), s.refs, workspace=s.ws)
    for name, x in dict(table=table, lens=lens, refs=refs, history=s.history[parents.view(-1).long()], cum=scores,
                        tokens=tokens.view(-1)).items():
        getattr(s, name).copy_(x)
    return seen


@pytest.mark.parametrize("dtype, fmt, pairs", [("f32", "int8", "halves"), ("f16", "e4m3", "interleaved"), ("bf16", "e4m3", "halves")])
@pytest.mark.parametrize("requests, beams, prompts", [(1, 4, [333]), (3, 2, [40, 1, 100]), (2, 9, [64, 150])])
def test_steps(kv, requests, beams, prompts, dtype, fmt, pairs):  # noqa: F811
    s = decoder(kv, requests, beams, prompts, dtype, fmt, pairs)
    batch, shared = requests * beams, 0
    for _ in range(20):
        seen = step(kv, s)
        b = seen.before
        lens, starts = b.lens.tolist(), list(range(batch + 1))
        want = turned(s.eq[b.at], s.rope, b.lens.long() - 1, pairs)
        assert torch.equal(seen.q, want.to(s.dtype))
        want = plan_ref(b.table.tolist(), lens, starts, s.groups.tolist(), PAGE, s.cache.pages)
        assert seen.plan.tolist() == want
        shared += sum(want[2:4 * requests:4])
        ref = attention_ref(seen.cache, 0, seen.q, b.table, lens, starts, DIM ** -0.5)
        close(seen.out, seen.lse, small(ref, dtype), max(lens) + 512, s.dtype, one_part=dtype == "bf16")
        want = reference(seen.logits, dict(s.rules, history=b.history, lens=b.said, prompt_lens=s.given), torch.float32)
        assert torch.equal(seen.adjusted.cpu(), want)
    assert shared > 0
    kv.kv_free(s.cache, s.table, s.lens, s.refs)
    assert (s.refs == 0).all()


@pytest.mark.parametrize("dtype, fmt", [("f32", "e4m3"), ("bf16", "int8")])
def test_a_captured_step(kv, dtype, fmt):  # noqa: F811
    """Two decoders of the same state, one stepped by calls, one by a graph's replays."""
    direct, held = (decoder(kv, 2, 4, [100, 47], dtype, fmt, "interleaved") for _ in range(2))
    for s in (direct, held):
        step(kv, s)  # first use
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = step(kv, held)
    torch.cuda.current_stream().wait_stream(side)
    for _ in range(25):
        want = step(kv, direct)
        graph.replay()
        for name in ("q", "plan", "out", "lse", "adjusted", "scores", "tokens", "parents"):
            assert torch.equal(getattr(got, name), getattr(want, name)), name
        for name in ("table", "lens", "refs", "history", "cum"):
            assert torch.equal(getattr(held, name), getattr(direct, name)), name
    for name in ("k", "v", "k_scale", "v_scale"):
        a, b = (getattr(s.cache, name)[0][s.refs > 0] for s in (held, direct))
        assert torch.equal(a, b), name


SMALL = dict(layers=2, hidden=256, q_heads=4, kv_heads=2, ffn=512, vocab=1000, pages=64, seed=3)


@pytest.mark.parametrize("fmt", ["e4m3", "int8"])
def test_beam_decode_with_a_penalty_and_banned_tokens(kv, fmt):  # noqa: F811
    """The search's scores against log-softmax sums (64 bits) of its tokens decoded apart, with the penalty and the mask
    as defined: 0.05 of a score, for codes that fall on the other side of a rounding."""
    import beam_decode
    from block_quantised_weight_gb300 import qgkv
    prompt, steps, penalty, banned = [(31 * i + 5) % 1000 for i in range(13)], 9, 1.4, list(range(0, 1000, 3)) + [31, 999]
    model = beam_decode.Model(**SMALL, fmt=fmt)
    scores, tokens = beam_decode.beam_search(model, prompt, beams=4, steps=steps, repetition=penalty, banned=banned)
    assert (scores[:-1] >= scores[1:]).all() and (model.refs == 0).all()
    assert not set(tokens.flatten().tolist()) & set(banned)

    other = beam_decode.Model(**SMALL, fmt=fmt)
    table, lens = torch.full((4, 8), -1, dtype=torch.int32, device="cuda"), i32([0] * 4)
    for b in range(4):
        logits = other.prefill(prompt, table[b:b + 1], lens[b:b + 1])
    logits = logits.expand(4, -1).contiguous()
    want = torch.zeros(4, dtype=torch.float64, device="cuda")
    for t in range(steps):
        x = logits.double()
        for b in range(4):
            came = sorted(set(prompt + tokens[b, :t].tolist()))
            x[b, came] = torch.where(x[b, came] > 0, x[b, came] / penalty, x[b, came] * penalty)
        x[:, banned] = -torch.inf
        want += torch.log_softmax(x, -1).gather(1, tokens[:, t:t + 1].long())[:, 0]
        if t + 1 < steps:
            qgkv.kv_reserve(other.cache, table, lens, other.refs, workspace=other.workspace)
            logits = other.step(tokens[:, t].contiguous(), table, lens)
            lens += 1
    assert qgemv.qg_device_status() == qgemv.QG_OK
    assert ((scores.double() - want).abs() <= 0.05).all(), (scores, want)


def test_beam_decode_step_over_shared_pages(kv):  # noqa: F811
    """Steps of four beams with and without their shared pages: logits of about 1 differ by roundings of the cache's codes
    and of sums in another order, 0.05 as above."""
    import beam_decode
    from block_quantised_weight_gb300 import qgkv
    model = beam_decode.Model(**SMALL, fmt="e4m3")
    table, lens = torch.full((1, least_width(4, 2, 64, 16)), -1, dtype=torch.int32, device="cuda"), i32([0])
    model.prefill([(7 * i + 1) % 1000 for i in range(150)], table, lens)
    table, lens, model.refs = qgkv.kv_fork(model.cache, table, lens, i32([0] * 4), model.refs, workspace=model.workspace)
    for t in range(20):
        qgkv.kv_reserve(model.cache, table, lens, model.refs, workspace=model.workspace)
        tokens = i32([(97 * t + 11 * b) % 1000 for b in range(4)])
        apart = model.step(tokens, table, lens)
        together = model.step(tokens, table, lens, groups=i32([0, 4]))
        assert ((apart - together).abs() <= 0.05).all()
        lens += 1


def test_pages_behind_32_bits(kv):  # noqa: F811
    """The same appends and attention on the first pages of a small cache and on the last of one of more than 2^32 bytes."""
    heads, page, dim, pages = 8, 256, 256, 8300
    assert pages * heads * page * dim > 1 << 32
    g = torch.Generator(device="cuda").manual_seed(5)
    rope, n = kv.rotary_table(1024, 256), [600, 3, 5]
    q, k, v = (torch.randn((sum(n), h, dim), device="cuda", generator=g).bfloat16() for h in (32, heads, heads))
    rows = torch.randn((4, 32, dim), device="cuda", generator=g).bfloat16()
    got = []
    for held, first in ((8, 0), (pages, pages - 8)):
        cache = kv.KVCache.allocate(1, held, heads, page, dim)
        table = torch.full((4, least_width(4, heads, dim, page)), -1, dtype=torch.int32, device="cuda")
        table[:2, :2] = i32([first + 7, first + 1])
        table[:2, 2] = i32([first + 4, first + 2])  # two sequences of no group see nothing
        turn = kv.kv_append_rotary(cache, 0, q[:600], k[:600], v[:600], rope, table[:1], i32([0]), starts=i32([0, 600]))
        kv.kv_copy_pages(cache, i32([first + 4]), i32([first + 2]))
        kv.kv_append_rotary(cache, 0, q[600:], k[600:], v[600:], rope, table[:2], i32([600, 600]), starts=i32([0, 3, 8]))
        lens = i32([603, 605, 0, 0])
        plan = kv.kv_share(cache, table, lens, i32([0, 2]))
        assert plan[2] == 512
        out = kv.kv_attention_shared(cache, 0, rows, table, lens, plan, return_lse=True)
        got.append((turn, *out, cache.k[0, first:first + 8].clone(), cache.v[0, first:first + 8].clone(),
                    cache.k_scale[0, first:first + 8].clone(), cache.v_scale[0, first:first + 8].clone()))
        close(*out, small(attention_ref(cache, 0, rows, table, [603, 605, 0, 0], [0, 1, 2, 3, 4], dim ** -0.5), "bf16"), 605 + 512,
              torch.bfloat16, one_part=True)
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_logits_behind_32_bits(kv):  # noqa: F811
    """The last rows of more than 2^31 logits (and 2^32 bytes) against the same rows by themselves."""
    rows, vocab, some = 16800, 128001, 5
    assert rows * vocab > 1 << 31
    x = torch.zeros((rows, vocab), dtype=torch.float16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(2)
    x[-some:] = torch.randn((some, vocab), device="cuda", generator=g).half()
    a = dict(history=torch.randint(0, vocab, (rows, 40), device="cuda", generator=g).int(), lens=i32([40] * rows),
             frequency=torch.rand(rows, device="cuda", generator=g), temperature=0.5 + torch.rand(rows, device="cuda", generator=g))
    got = kv.adjust_logits(x, **a)
    want = kv.adjust_logits(x[-some:].contiguous(), **{n: t[-some:].contiguous() for n, t in a.items()})
    assert torch.equal(got[-some:], want)
    assert torch.equal(kv.adjust_logits(x, **a, out=x)[-some:], want)


def test_shared_attention_on_two_streams_at_once(kv):  # noqa: F811
    """Calls that may overlap, each with a workspace of its own, have the bits of calls by themselves."""
    from test_kv_shared_gpu import shared_table
    cases, streams = [], [torch.cuda.Stream() for _ in range(2)]
    for i, dtype in enumerate(("f32", "bf16")):
        cache, table, lens, borders = shared_table(kv, [(2000, [40 + 9 * j for j in range(12)])], 2, 128, 16, "e4m3", "hnd", seed=i)
        q = torch.randn((12, 8, 128), device="cuda").to(DT[dtype])
        w, ln = kv.KVWorkspace("cuda"), i32(lens)
        plan = kv.kv_share(cache, table, ln, i32(borders))
        cases.append((cache, q, table, ln, plan, w, kv.kv_attention_shared(cache, 0, q, table, ln, plan, workspace=w)))
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for i, (cache, q, table, ln, plan, w, _) in enumerate(cases):
            with torch.cuda.stream(streams[i]):
                got[i].append(kv.kv_attention_shared(cache, 0, q, table, ln, plan, workspace=w))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(x, cases[i][-1]) for x in got[i])
