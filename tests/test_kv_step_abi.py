"""Host checks (no GPU) of the entry points around a decode step: refusals of the
append with rotation, the shared prefix and the logits adjustment, devices and streams of their
bindings.  Pointers are never dereferenced, validation fails first."""
import ctypes

import pytest

torch = pytest.importorskip("torch")

from block_quantised_weight_gb300 import qgemv  # noqa: E402
from test_kv_abi import A, E, G, L, at, cache, kv  # noqa: E402, F401
from test_kv_host import OnDevice, cache_on, calls, on  # noqa: E402, F401

F32 = dict(dtype=torch.float32)


def rotary(kv, **change):  # noqa: F811
    a = dict(layer=0, q=at(0), k=at(1), v=at(2), type=0, rows=3, q_heads=32, q_row=32 * 64, q_head=64, kv_row=4 * 64,
             kv_head=64, rope=at(8), positions=100, turned=64, pairs=0, out=at(9), table=at(3), width=8, lens=at(4),
             starts=None, batch=3)
    a.update(change)
    return kv.load()["qgkv_append_rotary"](ctypes.byref(cache(kv)), *a.values(), None)


@pytest.mark.parametrize("change, code", [
    (dict(layer=2), E), (dict(k=None), E), (dict(v=None), E), (dict(type=3), E), (dict(rows=2), E), (dict(batch=0), E),
    (dict(q_heads=0), E), (dict(q_heads=65537), E), (dict(out=None), E), (dict(rope=None), E), (dict(positions=0), E),
    (dict(turned=0), E), (dict(turned=24), E), (dict(turned=80), E), (dict(pairs=2), E), (dict(kv_head=32), E),
    (dict(q_row=32), E), (dict(table=None), E), (dict(lens=None), E),
    (dict(q=at(0) + 4), G), (dict(k=at(1) + 8), G), (dict(rope=at(8) + 4), G), (dict(out=at(9) + 8), G), (dict(q_row=32 * 64 + 1), G),
    (dict(starts=at(5) + 2, rows=7), G),
    (dict(out=at(0) + 64), L), (dict(out=at(0), q_row=33 * 64), L), (dict(out=at(1)), L), (dict(out=at(8) + 1600), L),
    (dict(out=A + 64), L), (dict(k=A + 1024), L), (dict(q=A + (1 << 28)), L), (dict(rope=A), L), (dict(out=at(3)), L),
])
def test_append_rotary_refusals(kv, change, code):  # noqa: F811
    assert rotary(kv, **change) == code


def test_append_rotary_of_no_rows_is_no_error(kv):  # noqa: F811
    assert rotary(kv, rows=0, starts=at(5), q=None, k=None, v=None, out=None) == qgemv.QG_OK


def logits(kv, **change):  # noqa: F811
    a = dict(x=at(0), type=0, rows=3, vocab=1000, row=1000, out=at(1), out_type=0, out_row=1000, history=at(2), width=20,
             lens=at(3), prompt=at(4), repetition=at(5), presence=at(6), frequency=at(7), bias_tokens=at(8), bias=at(9),
             biases=5, temperature=at(10), mask=at(11), words=32, masks=3, mask_rows=at(12))
    a.update(change)
    return kv.load()["qglogits_adjust"](*a.values(), None)


@pytest.mark.parametrize("change, code", [
    (dict(x=None), E), (dict(out=None), E), (dict(type=3), E), (dict(out_type=1), E), (dict(type=1, out_type=2), E),
    (dict(rows=-1), E), (dict(rows=(1 << 18) + 1), E), (dict(vocab=0), E), (dict(vocab=1 << 31), E), (dict(row=999), E),
    (dict(out_row=999), E), (dict(lens=None), E), (dict(history=None), E), (dict(width=0), E), (dict(width=1 << 20), E),
    (dict(history=None, lens=None, prompt=None, repetition=None, presence=None), E),
    (dict(biases=-1), E), (dict(biases=2048), E), (dict(bias=None), E), (dict(bias_tokens=None), E), (dict(biases=0), E),
    (dict(mask=None), E), (dict(masks=0), E), (dict(words=31), E), (dict(mask_rows=None, masks=2), E),
    (dict(x=at(0) + 2), G), (dict(out=at(1) + 1), G), (dict(history=at(2) + 2), G), (dict(mask=at(11) + 1), G),
    (dict(temperature=at(10) + 3), G), (dict(bias=at(9) + 2), G),
    (dict(out=at(0) + 4000), L), (dict(out=at(0), out_row=1001), L), (dict(out=at(2)), L), (dict(out=at(11) + 64), L),
    (dict(out=at(12)), L), (dict(type=2, out=at(0)), L),
])
def test_logits_refusals(kv, change, code):  # noqa: F811
    assert logits(kv, **change) == code


def test_logits_of_no_rows_is_no_error(kv):  # noqa: F811
    assert logits(kv, rows=0, x=None, out=None) == qgemv.QG_OK


def share(kv, **change):  # noqa: F811
    a = dict(pages=64, page_tokens=16, table=at(0), width=8, lens=at(1), starts=None, rows=3, batch=3, groups=at(2), n=2,
             plan=at(3))
    a.update(change)
    return kv.load()["qgkv_share"](*a.values(), None)


@pytest.mark.parametrize("change, code", [
    (dict(pages=0), E), (dict(page_tokens=24), E), (dict(table=None), E), (dict(lens=None), E), (dict(width=0), E),
    (dict(rows=2), E), (dict(rows=-1, starts=at(4)), E), (dict(batch=4097), E), (dict(groups=None), E), (dict(n=0), E),
    (dict(n=4097), E), (dict(plan=None), E), (dict(page_tokens=256, width=1 << 23), E), (dict(groups=at(2) + 1), G), (dict(plan=at(3) + 4), G),
    (dict(starts=at(4) + 2), G), (dict(plan=at(0)), L), (dict(plan=at(1)), L), (dict(plan=at(2)), L),
    (dict(plan=at(4), starts=at(4)), L),
])
def test_share_refusals(kv, change, code):  # noqa: F811
    assert share(kv, **change) == code


def shared(kv, c=None, **change):  # noqa: F811
    a = dict(layer=0, q=at(0), out=at(1), lse=at(2), type=0, rows=3, q_heads=32, row=32 * 64, head=64, table=at(3),
             width=8, lens=at(4), starts=None, batch=3, plan=at(6), n=2, scale=0.125, ws=at(16), wb=1 << 30)
    a.update(change)
    c = cache(kv) if c is None else c
    return kv.load()["qgkv_attention_shared"](ctypes.addressof(c), *a.values(), None)


@pytest.mark.parametrize("change, code", [
    (dict(layer=2), E), (dict(q=None), E), (dict(out=None), E), (dict(type=3), E), (dict(q_heads=30), E), (dict(rows=4), E),
    (dict(batch=0), E), (dict(width=0), E), (dict(plan=None), E), (dict(n=0), E), (dict(n=4097), E), (dict(ws=None), E),
    (dict(scale=float("nan")), E), (dict(q=at(0) + 4), G), (dict(plan=at(6) + 4), G), (dict(ws=at(16) + 128), G),
    (dict(wb=1 << 20), qgemv.QG_ESCRATCH), (dict(out=at(0) + 64), L), (dict(out=A + 64), L), (dict(lse=at(1) + 64), L),
    (dict(out=at(6)), L), (dict(lse=at(6)), L),
])
def test_attention_shared_refusals(kv, change, code):  # noqa: F811
    assert shared(kv, **change) == code


def test_attention_shared_of_no_rows_is_no_error(kv):  # noqa: F811
    assert shared(kv, rows=0, starts=at(5), q=None, out=None, lse=None) == qgemv.QG_OK


def Space(qgkv, take, device):
    w = qgkv.KVWorkspace.__new__(qgkv.KVWorkspace)
    w.buffer, w.ptr, w.bytes = take(on(device, 8, dtype=torch.uint8)), 0, 8
    return w


# every tensor of every call: position in this list is the one that lies elsewhere
OPERATORS = {
    "qgkv_share": (6, lambda k, d, t: k.kv_share(t(cache_on(k, d[0])), t(on(d[1], 2, 2)), t(on(d[2], 2)), t(on(d[3], 2)),
                                                 starts=t(on(d[4], 3)), out=t(on(d[5], 6)))),
    "qgkv_attention_shared": (9, lambda k, d, t: k.kv_attention_shared(
        t(cache_on(k, d[0])), 0, t(on(d[1], 2, 4, 64, **F32)), t(on(d[2], 2, 2)), t(on(d[3], 2)), t(on(d[4], 6)),
        starts=t(on(d[5], 3)), out=t(on(d[6], 2, 4, 64, **F32)), lse=t(on(d[7], 2, 4, **F32)), workspace=Space(k, t, d[8]))),
    "qgkv_append_rotary": (7, lambda k, d, t: k.kv_append_rotary(
        t(cache_on(k, d[0])), 0, t(on(d[1], 1, 4, 64, **F32)), t(on(d[2], 1, 2, 64, **F32)), t(on(d[2], 1, 2, 64, **F32)),
        t(on(d[3], 9, 64, **F32)), t(on(d[4], 1, 2)), t(on(d[5], 1)), out=t(on(d[6], 1, 4, 64, **F32)))),
    "qglogits_adjust": (12, lambda k, d, t: k.adjust_logits(
        t(on(d[0], 2, 9, **F32)), t(on(d[1], 2, 4)), t(on(d[2], 2)), t(on(d[3], 2)), t(on(d[4], 2, **F32)), t(on(d[5], 2, **F32)),
        t(on(d[6], 2, **F32)), t(on(d[7], 2, 3)), t(on(d[7], 2, 3, **F32)), t(on(d[8], 2, **F32)), t(on(d[9], 1, 1)),
        t(on(d[10], 2)), out=t(on(d[11], 2, 9, **F32)))),
}


@pytest.mark.parametrize("name", OPERATORS)
def test_tensors_of_another_device_are_refused(calls, name):  # noqa: F811
    qgkv, made = calls
    count, call = OPERATORS[name]
    call(qgkv, [0] * count, lambda x: x)
    assert made == [name]
    for elsewhere in range(count):
        with pytest.raises(ValueError, match="device"):
            call(qgkv, [int(i == elsewhere) for i in range(count)], lambda x: x)
    assert made == [name]


@pytest.mark.parametrize("name", OPERATORS)
def test_tensors_are_lent_to_the_stream_of_a_call(calls, monkeypatch, name):  # noqa: F811
    import contextlib
    qgkv, made = calls
    lent, current, given = [], ["main"], []

    @contextlib.contextmanager
    def enter(stream):
        current.append(stream)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(OnDevice, "record_stream", lambda self, stream: lent.append((self.data_ptr(), stream)), raising=False)

    def take(x):
        given.extend((x.k, x.k_scale, x.v, x.v_scale) if isinstance(x, qgkv.KVCache) else (x,))
        return x

    count, call = OPERATORS[name]

    class Streamed:
        KVCache, KVWorkspace = qgkv.KVCache, qgkv.KVWorkspace

        def __getattr__(self, f):
            return lambda *a, **b: getattr(qgkv, f)(*a, **b, stream="side")

    call(Streamed(), [0] * count, take)
    assert made == [name] and current == ["main"]
    assert {(t.data_ptr(), "side") for t in given} <= set(lent)


def test_binding_refusals(calls):  # noqa: F811
    qgkv, made = calls
    c, q, k = cache_on(qgkv, 0), on(0, 1, 4, 64, **F32), on(0, 1, 2, 64, **F32)
    rope, table, lens = on(0, 9, 64, **F32), on(0, 1, 2), on(0, 1)
    call = lambda q=q, k=k, v=k, rope=rope, **more: qgkv.kv_append_rotary(c, 0, q, k, v, rope, table, lens, **more)  # noqa: E731
    for bad in (dict(pairs="neox"), dict(v=on(0, 1, 2, 64, dtype=torch.float16)), dict(q=on(0, 2, 4, 64, **F32)),
                dict(q=on(0, 1, 4, 64, dtype=torch.bfloat16)), dict(q=None, out=q), dict(out=on(0, 1, 4, 32, **F32))):
        with pytest.raises(ValueError):
            call(**bad)
    for bad in (dict(rope=on(0, 9, 64, dtype=torch.float64)), dict(k=on(0, 1, 2, 64)), dict(out=on(0, 1, 4, 64))):
        with pytest.raises((TypeError, ValueError)):
            call(**bad)
    x = on(0, 2, 9, **F32)
    for bad in (dict(lens=on(0, 3)), dict(bias=on(0, 2, 3, **F32)), dict(bias_tokens=on(0, 2, 3)), dict(out=on(0, 2, 8, **F32)),
                dict(bias_tokens=on(0, 2, 3), bias=on(0, 2, 4, **F32)), dict(temperature=on(0, 2, 1, **F32))):
        with pytest.raises(ValueError):
            qgkv.adjust_logits(x, **bad)
    for bad in (dict(history=on(0, 2, 3, dtype=torch.int64)), dict(mask=on(0, 1, 1, dtype=torch.uint8)),
                dict(presence=on(0, 2)), dict(out=on(0, 2, 9))):
        with pytest.raises(TypeError):
            qgkv.adjust_logits(x, **bad)
    plan = lambda n: qgkv.kv_attention_shared(c, 0, q, table, lens, on(0, n))  # noqa: E731
    for n in (0, 1, 4, 6):
        with pytest.raises(ValueError):
            plan(n)
    with pytest.raises(ValueError):
        qgkv.kv_share(c, table, lens, on(0, 1))
    with pytest.raises(ValueError):
        qgkv.kv_share(c, table, lens, on(0, 2), out=on(0, 6))
    with pytest.raises(TypeError):
        qgkv.kv_share(c, table, lens, on(0, 2, dtype=torch.int64))
    assert not made
