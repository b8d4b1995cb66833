"""Entry points of include/qgkv.h: exports and refusals on the host (no GPU:
the pointers below are never dereferenced, validation fails first)."""
import ctypes
import os
import re

import pytest

from block_quantised_weight_gb300 import build, qgemv

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
A = 0x100000  # fake, 256-byte aligned "device" addresses
E, G, S, L = qgemv.QG_EINVAL, qgemv.QG_EALIGN, qgemv.QG_ESCRATCH, qgemv.QG_EALIAS


@pytest.fixture(scope="module")
def kv():
    build.build()
    from block_quantised_weight_gb300 import qgkv
    qgkv.load()
    return qgkv


def cache(kv, **change):
    f = dict(k=A, v=A + (1 << 28), k_scale=A + (2 << 28), v_scale=A + (3 << 28), layers=2, pages=64,
             layer_stride=64 * 4 * 16 * 64, page_stride=4 * 16 * 64, heads=4, page_tokens=16, head_dim=64, format=1,
             order=0)
    f.update(change)
    return kv.QgkvCache(**f)


P = A + (4 << 28)  # table, lens, starts, q, k and outputs, 1 MB apart


def at(i):
    return P + (i << 20)


def test_header_and_binding_agree(kv):
    txt = re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", "qgkv.h")).read(), flags=re.S)
    names = set(re.findall(r"^\s*QG_API\s+\w+\s+(qg\w+)\s*\(", txt, flags=re.M))
    assert names == set(kv.EXPORTS)
    assert set(kv.load()) == names
    for n in ("MAX_BATCH", "MAX_BEAMS", "MAX_KEEP"):
        assert int(re.search(rf"QGKV_{n} (\d+)", txt).group(1)) == getattr(kv, f"QGKV_{n}")
    assert qgemv.strerror(qgemv.QG_EPAGES) not in ("", "unknown status")


def attention(kv, c=None, **change):
    a = dict(layer=0, q=at(0), out=at(1), lse=at(2), type=0, rows=3, q_heads=32, row=32 * 64, head=64, table=at(3),
             width=8, lens=at(4), starts=None, batch=3, scale=0.125, ws=at(16), wb=1 << 30)
    a.update(change)
    c = cache(kv) if c is None else c
    return kv.load()["qgkv_attention"](ctypes.addressof(c), *a.values(), None)


@pytest.mark.parametrize("change, code", [
    (dict(k=None), E), (dict(v_scale=None), E), (dict(format=3), E), (dict(order=2), E), (dict(layers=0), E),
    (dict(pages=0), E), (dict(pages=(1 << 20) + 1), E), (dict(heads=0), E), (dict(page_tokens=48), E),
    (dict(page_tokens=512), E), (dict(head_dim=72), E), (dict(head_dim=272), E), (dict(head_dim=0), E),
    (dict(page_stride=4 * 16 * 64 - 16), E), (dict(page_stride=4 * 16 * 64 + 8), G), (dict(k=A + 8), G),
    (dict(k_scale=A + 2), G),
])
def test_cache_refusals(kv, change, code):
    assert attention(kv, cache(kv, **change)) == code


@pytest.mark.parametrize("change, code", [
    (dict(layer=2), E), (dict(layer=-1), E), (dict(q=None), E), (dict(out=None), E), (dict(type=3), E),
    (dict(q_heads=30), E), (dict(q_heads=0), E), (dict(rows=4), E), (dict(batch=0), E), (dict(batch=5000), E),
    (dict(width=0), E), (dict(table=None), E), (dict(lens=None), E), (dict(row=32), E), (dict(head=60), E),
    (dict(scale=float("nan")), E), (dict(scale=float("inf")), E), (dict(ws=None), E),
    (dict(q=at(0) + 4), G), (dict(out=at(1) + 4), G), (dict(head=65), G), (dict(lse=at(2) + 2), G),
    (dict(starts=at(5) + 1), G), (dict(ws=at(16) + 128), G), (dict(wb=1 << 20), S),
    (dict(out=at(0) + 64), L), (dict(out=A + 64), L), (dict(lse=at(1) + 64), L),
])
def test_attention_refusals(kv, change, code):
    assert attention(kv, **change) == code


def append(kv, **change):
    a = dict(layer=0, k=at(0), v=at(1), type=0, rows=3, row=4 * 64, head=64, table=at(3), width=8, lens=at(4),
             starts=None, batch=3)
    a.update(change)
    return kv.load()["qgkv_append"](ctypes.byref(cache(kv)), *a.values(), None)


@pytest.mark.parametrize("change, code", [
    (dict(layer=7), E), (dict(k=None), E), (dict(v=None), E), (dict(type=-1), E), (dict(rows=2), E),
    (dict(rows=-1, starts=at(5)), E), (dict(head=32), E), (dict(table=None), E), (dict(k=at(0) + 8), G),
    (dict(row=4 * 64 + 2), G), (dict(lens=at(4) + 1), G), (dict(k=A + 1024), L), (dict(v=A + (1 << 28)), L),
])
def test_append_refusals(kv, change, code):
    assert append(kv, **change) == code


def fork(kv, **change):
    a = dict(table=at(0), width=8, lens=at(1), batch=3, parent=at(2), batch2=4, refs=at(3), table2=at(4), lens2=at(5),
             refs2=at(6), ws=at(16), wb=1 << 30)
    a.update(change)
    return kv.load()["qgkv_fork"](ctypes.byref(cache(kv)), *a.values(), None)


@pytest.mark.parametrize("change, code", [
    (dict(parent=None), E), (dict(batch2=0), E), (dict(batch2=5000), E), (dict(refs=None), E), (dict(lens2=None), E),
    (dict(refs=at(3) + 4), G), (dict(refs2=at(6) + 8), G), (dict(wb=100), S), (dict(table2=at(0)), L),
    (dict(refs2=at(3)), L), (dict(lens2=at(4) + 16), L), (dict(lens2=at(1)), L),
])
def test_fork_refusals(kv, change, code):
    assert fork(kv, **change) == code


def test_other_page_refusals(kv):
    held = cache(kv)
    f, c = kv.load(), ctypes.byref(held)
    compact = lambda *a: f["qgkv_compact"](c, at(0), 8, at(1), 3, *a, at(16), 1 << 30, None)  # noqa: E731
    assert compact(None, None, at(4), at(5), at(6), at(7)) == E
    assert compact(None, at(3), at(4), at(5), at(6), None) == E
    assert compact(None, at(3), at(0), at(5), at(6), at(7)) == L
    assert compact(at(5), at(3), at(4), at(5), at(6), at(7)) == L
    assert f["qgkv_copy_pages"](c, None, at(1), None, 4, None) == E
    assert f["qgkv_copy_pages"](c, at(0), at(1), None, -1, None) == E
    assert f["qgkv_copy_pages"](c, at(0) + 2, at(1), None, 4, None) == G
    assert f["qgkv_reserve"](0, 16, at(0), 8, at(1), None, 3, at(3), at(16), 1 << 30, None) == E
    assert f["qgkv_reserve"](64, 24, at(0), 8, at(1), None, 3, at(3), at(16), 1 << 30, None) == E
    assert f["qgkv_reserve"](64, 16, at(0), 8, at(1), None, 3, at(0), at(16), 1 << 30, None) == L
    assert f["qgkv_free"](64, 16, at(0), 8, at(1), None, 3, None, None) == E
    assert f["qgkv_free"](64, 16, at(0), 8, at(0), None, 3, at(3), None) == L


def beam(kv, **change):
    a = dict(logits=at(0), type=0, cum=at(4), requests=2, beams=4, vocab=1000, row=1000, keep=8, scores=at(5),
             tokens=at(6), parents=at(7), ws=at(16), wb=1 << 30)
    a.update(change)
    return kv.load()["qgbeam_select"](*a.values(), None)


@pytest.mark.parametrize("change, code", [
    (dict(logits=None), E), (dict(cum=None), E), (dict(type=5), E), (dict(requests=0), E), (dict(beams=65), E),
    (dict(vocab=0), E), (dict(row=999), E), (dict(keep=0), E), (dict(keep=129), E), (dict(vocab=1, row=1, keep=5), E),
    (dict(logits=at(0) + 2), G), (dict(wb=4096), S), (dict(tokens=at(5) + 8), L), (dict(scores=at(0) + 400), L),
    (dict(requests=4096, beams=64, keep=128, scores=1 << 40, tokens=2 << 40, parents=3 << 40, cum=4 << 40), None),
])
def test_beam_refusals(kv, change, code):
    if code is None:  # refused for its partial results before any launch, or for want of a device before that
        assert beam(kv, **change) in (S, qgemv.QG_ECUDA)
    else:
        assert beam(kv, **change) == code
