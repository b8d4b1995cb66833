"""GPU tests of adjust_logits against a plain implementation in 64 bits that rounds
to fp32 where the definition does: products, quotients, sums and differences of two
fp32 values, rounded to 64 bits and then to fp32, are those rounded once (53 >= 2 *
24 + 2), so results are compared bit for bit."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")

from block_quantised_weight_gb300 import qgemv  # noqa: E402
from test_kv_gpu import DT, i32, kv, status_clean, ws  # noqa: E402, F401

pytestmark = pytest.mark.gpu


def reference(x, a, out_dtype):
    """x [rows, vocab]; a: the call's arguments as host arrays."""
    f32 = lambda v: np.asarray(v, np.float64).astype(np.float32).astype(np.float64)  # noqa: E731
    x = x.float().cpu().numpy().astype(np.float64)
    get = lambda n: a[n].cpu().numpy() if a.get(n) is not None else None  # noqa: E731
    history, lens, prompt = get("history"), get("lens"), get("prompt_lens")
    with np.errstate(all="ignore"):
        for r in range(x.shape[0]):
            row = x[r]
            if history is not None:
                n = max(0, min(int(lens[r]), history.shape[1]))
                p = 0 if prompt is None else int(prompt[r])
                came, made = {}, {}
                for i in range(n):
                    t = int(history[r, i])
                    if 0 <= t < x.shape[1]:
                        came[t] = 1
                        if i >= p:
                            made[t] = made.get(t, 0) + 1
                for t in came:
                    if a.get("repetition") is not None:
                        rho = np.float64(get("repetition")[r])
                        row[t] = f32(row[t] / rho if row[t] > 0 else row[t] * rho)
                for t, c in made.items():
                    if a.get("frequency") is not None:
                        row[t] = f32(row[t] - f32(np.float64(get("frequency")[r]) * c))
                    if a.get("presence") is not None:
                        row[t] = f32(row[t] - np.float64(get("presence")[r]))
            if a.get("bias") is not None:
                last = {int(t): float(v) for t, v in zip(get("bias_tokens")[r], get("bias")[r])}
                for t, v in last.items():
                    if 0 <= t < x.shape[1]:
                        row[t] = f32(row[t] + v)
            if a.get("temperature") is not None:
                row[:] = f32(row / np.float64(get("temperature")[r]))
            if a.get("mask") is not None:
                m = r if a.get("mask_rows") is None else int(get("mask_rows")[r])
                if 0 <= m < a["mask"].shape[0]:
                    bits = np.unpackbits(get("mask")[m].view(np.uint8), bitorder="little")[:x.shape[1]]
                    row[bits == 0] = -math.inf
    return torch.from_numpy(x).float().to(out_dtype)


def arguments(rows, vocab, width, biases, masks, seed, which="hprfbtm"):
    g = torch.Generator(device="cuda").manual_seed(seed)
    u = lambda lo, hi: lo + (hi - lo) * torch.rand(rows, device="cuda", generator=g)  # noqa: E731
    a = {}
    if "h" in which:
        # few tokens, so that they repeat; some outside the vocabulary
        a["history"] = (torch.randint(-2, 12, (rows, width), device="cuda", generator=g) * (vocab // 9 + 1)).int()
        a["lens"] = torch.randint(0, width + 1, (rows,), device="cuda", generator=g).int()
        a["prompt_lens"] = a["lens"] // 2
        if "p" in which:
            a["presence"] = u(-0.5, 1.0)
        if "r" in which:
            a["repetition"] = u(0.8, 1.7)
        if "f" in which:
            a["frequency"] = u(-0.2, 0.6)
    if "b" in which:
        # the same token more than once, and places without one
        a["bias_tokens"] = torch.randint(-1, vocab + 2, (rows, biases), device="cuda", generator=g).int()
        a["bias_tokens"][:, biases // 2:] = a["bias_tokens"][:, :biases - biases // 2].flip(1)
        a["bias"] = 4 * torch.randn((rows, biases), device="cuda", generator=g)
    if "t" in which:
        a["temperature"] = u(0.3, 2.0)
    if "m" in which:
        a["mask"] = torch.randint(-2**31, 2**31, (masks, (vocab + 31) // 32 + 2), device="cuda", generator=g).int()
        a["mask_rows"] = torch.randint(-1, masks, (rows,), device="cuda", generator=g).int()
    return a


def check(kv, x, a, out=None, out_dtype=None):  # noqa: F811
    want = reference(x, a, out_dtype or x.dtype)
    got = kv.adjust_logits(x, **a, **({} if out is None else {"out": out}))
    assert got.dtype == want.dtype
    same = (got.cpu() == want) | (torch.isnan(got.cpu()) & torch.isnan(want))
    assert same.all(), (~same).nonzero()[:5]
    return got


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("rows, vocab, width, biases", [(1, 1, 1, 1), (3, 31, 5, 2), (2, 33, 40, 40), (4, 1024, 700, 33),
                                                        (5, 1025, 3, 300), (7, 32001, 2000, 100)])
def test_adjust_logits(kv, dtype, rows, vocab, width, biases):  # noqa: F811
    g = torch.Generator(device="cuda").manual_seed(vocab)
    x = (3 * torch.randn((rows, vocab), device="cuda", generator=g)).to(DT[dtype])
    a = arguments(rows, vocab, width, biases, 3, vocab)
    check(kv, x, a)
    if dtype != "f32":
        check(kv, x, a, out=torch.empty((rows, vocab), device="cuda"), out_dtype=torch.float32)
    check(kv, x.clone(), a, out=None)
    same = x.clone()
    want = reference(x, a, x.dtype)
    kv.adjust_logits(same, **a, out=same)
    assert torch.equal(same.cpu(), want)


@pytest.mark.parametrize("which", ["h", "hr", "hp", "hf", "hpf", "b", "t", "m", "hrm", "bm", "hpfbm", ""])
@pytest.mark.parametrize("in_place", [False, True])
def test_adjust_logits_each_part(kv, which, in_place):  # noqa: F811
    rows, vocab = 4, 2500
    x = torch.randn((rows, vocab), device="cuda", generator=torch.Generator(device="cuda").manual_seed(5))
    a = arguments(rows, vocab, 60, 20, 2, len(which), which)
    want = reference(x, a, x.dtype)
    got = kv.adjust_logits(x, **a, out=x if in_place else None)
    assert (got is x) == in_place and torch.equal(got.cpu(), want)


@pytest.mark.parametrize("rows, vocab", [(300, 5001), (2, 200003), (70, 50257)])
def test_adjust_logits_spans(kv, rows, vocab):  # noqa: F811
    """Spans of all sizes; rows apart by more than the vocabulary, from an odd address."""
    g = torch.Generator(device="cuda").manual_seed(rows)
    x = torch.randn((rows, vocab + 7), device="cuda", generator=g)[:, 3:3 + vocab]
    a = arguments(rows, vocab, 50, 9, rows, rows)
    check(kv, x, a)
    out = torch.full((rows, vocab + 5), 9.0, device="cuda")
    check(kv, x, a, out=out[:, 1:1 + vocab])
    assert (out[:, 0] == 9.0).all() and (out[:, 1 + vocab:] == 9.0).all()


def test_adjust_logits_special_values(kv):  # noqa: F811
    """Infinities, NaN, zeros and subnormals; penalties of 0, 1 and infinity; a history of one token throughout."""
    vals = [0.0, -0.0, math.inf, -math.inf, math.nan, 1e-45, -1e-45, 3e38, -3e38, 1.0, -1.0]
    x = torch.tensor(vals, device="cuda").repeat(6, 3)
    width = 5000
    t = torch.arange(x.shape[1], device="cuda").repeat(6, width // x.shape[1] + 1)[:, :width].int()
    t[5] = 2
    f = lambda *v: torch.tensor(v, device="cuda", dtype=torch.float32)  # noqa: E731
    a = dict(history=t.contiguous(), lens=i32([width, 20, 0, width, 7, width]), prompt_lens=i32([0, 3, 0, -4, 90, 1]),
             repetition=f(1.0, 0.0, 2.0, math.inf, 1.3, 1.1), presence=f(0.0, math.inf, 1.0, 0.5, 2.0, 0.1),
             frequency=f(0.1, 0.0, 1.0, 0.7, math.nan, 1e30), temperature=f(1.0, 0.5, 0.0, -1.0, math.inf, 1e-30))
    check(kv, x, a)
    check(kv, x, {k: v for k, v in a.items() if k != "temperature"})


def test_adjust_logits_masked_wins(kv):  # noqa: F811
    """A masked token is -inf whatever else applies to it, NaN and +inf among it."""
    x = torch.full((3, 70), math.nan, device="cuda")
    x[1] = math.inf
    mask = torch.zeros((1, 3), dtype=torch.int32, device="cuda")
    out = kv.adjust_logits(x, temperature=torch.tensor([0.0, -1.0, 1.0], device="cuda"), mask=mask,
                           mask_rows=i32([0, 0, -1]), bias_tokens=i32([[3], [3], [3]]),
                           bias=torch.full((3, 1), math.inf, device="cuda"))
    assert (out[:2] == -math.inf).all() and torch.isnan(out[2]).all()


def test_adjust_logits_bad_lengths_and_masks_are_reported(kv):  # noqa: F811
    x = torch.randn((3, 100), device="cuda")
    a = dict(history=i32([[1, 2], [3, 4], [5, 6]]), lens=i32([3, -1, 2]), presence=torch.ones(3, device="cuda"),
             mask=torch.zeros((1, 4), dtype=torch.int32, device="cuda"), mask_rows=i32([1, -2, -1]))
    want = reference(x, {**a, "mask": None}, x.dtype)
    got = kv.adjust_logits(x, **a)
    assert qgemv.qg_device_status() == qgemv.QG_EBOUNDS
    assert torch.equal(got.cpu(), want)


def test_adjust_logits_long_history(kv):  # noqa: F811
    """A token that came 300000 times."""
    x = torch.randn((2, 50), device="cuda")
    a = dict(history=torch.full((2, 300000), 7, dtype=torch.int32, device="cuda"), lens=i32([300000, 299999]),
             prompt_lens=i32([1, 299999]), frequency=torch.tensor([1e-4, 1.0], device="cuda"))
    check(kv, x, a)


def test_adjust_logits_empty(kv):  # noqa: F811
    x = torch.randn((2, 50), device="cuda")
    none = torch.empty((2, 0), dtype=torch.int32, device="cuda")
    got = kv.adjust_logits(x, history=none, lens=i32([0, 0]), presence=torch.ones(2, device="cuda"), bias_tokens=none,
                           bias=none.float())
    assert torch.equal(got, x) and got is not x
    assert kv.adjust_logits(x[:0], temperature=torch.ones(0, device="cuda")).shape == (0, 50)


def test_adjust_logits_then_selection_in_a_graph(kv):  # noqa: F811
    """Adjusted rows go to the selection, as one captured step on a stream of its own, replayed on other values."""
    own, side = kv.KVWorkspace("cuda"), torch.cuda.Stream()
    beams, vocab = 4, 3001
    a = arguments(beams, vocab, 30, 6, 1, 9)
    a["mask_rows"].zero_()
    x, cum = torch.randn((beams, vocab), device="cuda"), torch.zeros((1, beams), device="cuda")
    step = lambda: kv.beam_select(kv.adjust_logits(x, **a), cum, 5, workspace=own)  # noqa: E731
    step()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = step()
    for seed in range(3):
        x.normal_()
        a["lens"].copy_(torch.randint(0, 31, (beams,)).int())
        graph.replay()
        y = reference(x, a, torch.float32).double()
        scores = torch.log_softmax(y, -1).flatten()
        top, at = torch.sort(scores, descending=True, stable=True)
        assert torch.equal(outs[1][0].cpu(), (at[:5] % vocab).int()) and torch.equal(outs[2][0].cpu(), (at[:5] // vocab).int())
