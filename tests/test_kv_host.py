"""Host checks of the decode-state sources and binding (no GPU)."""
import os
import re

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "block_quantised_weight_gb300", "csrc")


def test_prompt_kernel_waits_for_stored_probabilities():
    """Stores to tensor memory are asynchronous, and nothing orders a load of the same columns behind
    them but a wait for the stores: the first half's probabilities are read back only after one."""
    src = open(os.path.join(CSRC, "kv_prompt.cu")).read()
    at = src.index("if (half == 1) {")
    calls = re.findall(r"\b(tmem_stored|tmem_load32|tmem_store32)\(", src[at:])
    assert calls[:3] == ["tmem_stored", "tmem_load32", "tmem_store32"]


torch = pytest.importorskip("torch")


class OnDevice(torch.Tensor):
    """A host tensor that says it lies on a CUDA device; its memory is never used."""

    at = 0

    @property
    def is_cuda(self):
        return True

    def get_device(self):
        return self.at


def on(device, *shape, dtype=torch.int32):
    t = torch.Tensor._make_subclass(OnDevice, torch.zeros(shape, dtype=dtype))
    t.at = device
    return t


@pytest.fixture
def calls(monkeypatch):
    """The binding with device 0 current and its calls recorded instead of made."""
    from block_quantised_weight_gb300 import qgkv
    made = []
    monkeypatch.setattr(qgkv, "_call", lambda name, *args: made.append(name))
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0)
    return qgkv, made


def cache_on(qgkv, device):
    code = dict(dtype=torch.uint8)
    scale = dict(dtype=torch.float32)
    return qgkv.KVCache(on(device, 1, 3, 2, 16, 64, **code), on(device, 1, 3, 2, **scale),
                        on(device, 1, 3, 2, 16, 64, **code), on(device, 1, 3, 2, **scale))


class Workspace:
    def __init__(self, device):
        self.buffer, self.ptr, self.bytes = on(device, 8, dtype=torch.uint8), 0, 8


# every tensor of every call: position in this list is the one that lies elsewhere
OPERATORS = {
    "qgkv_append": (4, lambda k, d: k.kv_append(
        cache_on(k, d[0]), 0, on(d[1], 1, 2, 64, dtype=torch.float32), on(d[1], 1, 2, 64, dtype=torch.float32),
        on(d[2], 1, 2), on(d[3], 1))),
    "qgkv_attention": (8, lambda k, d: k.kv_attention(
        cache_on(k, d[0]), 0, on(d[1], 1, 4, 64, dtype=torch.float32), on(d[2], 1, 2), on(d[3], 1), on(d[4], 2),
        out=on(d[5], 1, 4, 64, dtype=torch.float32), lse=on(d[6], 1, 4, dtype=torch.float32), workspace=Workspace(d[7]))),
    "qgkv_copy_pages": (4, lambda k, d: k.kv_copy_pages(cache_on(k, d[0]), on(d[1], 1), on(d[2], 1), on(d[3], 1))),
    "qgkv_fork": (9, lambda k, d: k.kv_fork(
        cache_on(k, d[0]), on(d[1], 1, 2), on(d[2], 1), on(d[3], 2), on(d[4], 3),
        out=(on(d[5], 2, 2), on(d[6], 2), on(d[7], 3)), workspace=Workspace(d[8]))),
    "qgkv_reserve": (5, lambda k, d: k.kv_reserve(
        cache_on(k, 0), on(d[0], 1, 2), on(d[1], 1), on(d[2], 3), on(d[3], 1), workspace=Workspace(d[4]))),
    "qgkv_free": (4, lambda k, d: k.kv_free(
        cache_on(k, 0), on(d[0], 1, 2), on(d[1], 1), on(d[2], 3), on(d[3], 1, dtype=torch.uint8))),
}


@pytest.mark.parametrize("name", OPERATORS)
def test_tensors_of_another_device_are_refused(calls, name):
    """A launch goes to the current device: a pointer of another one must not reach it."""
    qgkv, made = calls
    count, call = OPERATORS[name]
    call(qgkv, [0] * count)
    assert made == [name]
    for elsewhere in range(count):
        with pytest.raises(ValueError, match="device"):
            call(qgkv, [int(i == elsewhere) for i in range(count)])
    with pytest.raises(ValueError, match="device"):
        call(qgkv, [1] * count)
    assert made == [name]


def test_compaction_and_selection_of_another_device_are_refused(calls, monkeypatch):
    """The calls that make their own outputs."""
    qgkv, made = calls
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: on(0, *shape, dtype=dtype))
    names = []
    for d in ([0] * 8, *([int(i == j) for j in range(8)] for i in range(8))):
        compact = lambda: qgkv.kv_compact(  # noqa: E731
            cache_on(qgkv, 0), on(d[0], 1, 2), on(d[1], 1), on(d[2], 3), drop=on(d[3], 1, dtype=torch.uint8),
            out=(on(0, 1, 2), on(0, 1), on(d[4], 3)), workspace=Workspace(0))
        select = lambda: qgkv.beam_select(on(d[5], 2, 9, dtype=torch.float32), on(d[6], 1, 2, dtype=torch.float32), 2,  # noqa: E731
                                          workspace=Workspace(d[7]))
        for at, call in ((slice(0, 5), compact), (slice(5, 8), select)):
            if any(d[at]):
                with pytest.raises(ValueError, match="device"):
                    call()
            elif not any(d):
                call()
                names = list(made)
    assert made == names == ["qgkv_compact", "qgbeam_select"]


def test_cache_of_two_devices_is_refused(calls):
    qgkv, _ = calls
    one = cache_on(qgkv, 0)
    with pytest.raises(ValueError, match="device"):
        qgkv.KVCache(one.k, one.k_scale, one.v, on(1, 1, 3, 2, dtype=torch.float32))


def test_no_rows_and_no_pages_are_no_error():
    """An empty tensor's address is null: nothing to do, on the host already."""
    import ctypes
    from block_quantised_weight_gb300 import build, qgemv, qgkv
    build.build()
    base = 0x100000
    c = qgkv.QgkvCache(base, base + (1 << 28), base + (2 << 28), base + (3 << 28), 2, 64, 64 * 4096, 4096, 4, 16, 64, 1, 0)
    table, lens, starts, ws = (base + (4 << 28) + (i << 20) for i in range(4))
    f, ref = qgkv.load(), ctypes.addressof(c)
    for k in (None, base + (5 << 28)):
        assert f["qgkv_append"](ref, 0, k, k, 0, 0, 256, 64, table, 8, lens, starts, 3, None) == qgemv.QG_OK
        assert f["qgkv_attention"](ref, 0, k, k, None, 2, 0, 32, 2048, 64, table, 8, lens, starts, 3, 0.1, ws, 1 << 30,
                                   None) == qgemv.QG_OK
        assert f["qgkv_copy_pages"](ref, k, k, None, 0, None) == qgemv.QG_OK
    # with rows, or with what is wrong anyway, they stay errors
    assert f["qgkv_append"](ref, 0, None, base, 0, 1, 256, 64, table, 8, lens, starts, 3, None) == qgemv.QG_EINVAL
    assert f["qgkv_attention"](ref, 0, base, None, None, 2, 1, 32, 2048, 64, table, 8, lens, starts, 3, 0.1, ws, 1 << 30,
                               None) == qgemv.QG_EINVAL
    assert f["qgkv_append"](ref, 0, None, None, 9, 0, 256, 64, table, 8, lens, starts, 3, None) == qgemv.QG_EINVAL
    assert f["qgkv_copy_pages"](ref, None, None, None, -1, None) == qgemv.QG_EINVAL


def test_attention_rows_beyond_32_bits_are_refused():
    """The query rows of a cache head are counted in 32 bits on the device."""
    import ctypes
    from block_quantised_weight_gb300 import build, qgemv, qgkv
    build.build()
    base = 0x100000
    c = qgkv.QgkvCache(base, base + (1 << 28), base + (2 << 28), base + (3 << 28), 1, 64, 64 * 4096, 4096, 1, 64, 16, 1, 0)
    table, lens, starts, ws = (base + (4 << 28) + (i << 20) for i in range(4))
    far = 1 << 45
    attention = lambda rows, heads: qgkv.load()["qgkv_attention"](  # noqa: E731
        ctypes.addressof(c), 0, far, 2 * far, None, 2, rows, heads, 16 * heads, 16, table, 8, lens, starts, 3, 0.1, ws,
        1 << 30, None)
    assert attention(1 << 20, 1 << 11) == qgemv.QG_EINVAL
    assert attention((1 << 31) - 511, 1) == qgemv.QG_EINVAL
    assert attention(1 << 30, 65536) == qgemv.QG_EINVAL


def test_no_verdict_of_a_bounded_wait_is_dropped():
    """A wait that gave up ends its warp's further waits and copies (a wait that drains copies in flight says
    that it has no use for the verdict)."""
    for name in ("kv_rows.cuh", "kv_prompt.cu"):
        src = open(os.path.join(CSRC, name)).read()
        assert "mbar_wait_bounded(" in src
        assert not re.search(r"^\s*mbar_wait_bounded\(", src, flags=re.M), name
        assert not re.search(r"[;{}]\s*mbar_wait_bounded\(", src), name


STREAMED = {
    "kv_append": lambda k, t: k.kv_append(t(cache_on(k, 0)), 0, t(on(0, 1, 2, 64, dtype=torch.float32)),
                                          t(on(0, 1, 2, 64, dtype=torch.float32)), t(on(0, 1, 2)), t(on(0, 1)),
                                          starts=t(on(0, 2)), stream="side"),
    "kv_attention": lambda k, t: k.kv_attention(
        t(cache_on(k, 0)), 0, t(on(0, 1, 4, 64, dtype=torch.float32)), t(on(0, 1, 2)), t(on(0, 1)), starts=t(on(0, 2)),
        out=t(on(0, 1, 4, 64, dtype=torch.float32)), lse=t(on(0, 1, 4, dtype=torch.float32)), workspace=t(Space(k)),
        stream="side"),
    "kv_copy_pages": lambda k, t: k.kv_copy_pages(t(cache_on(k, 0)), t(on(0, 1)), t(on(0, 1)), t(on(0, 1)), stream="side"),
    "kv_fork": lambda k, t: k.kv_fork(t(cache_on(k, 0)), t(on(0, 1, 2)), t(on(0, 1)), t(on(0, 2)), t(on(0, 3)),
                                      out=(t(on(0, 2, 2)), t(on(0, 2)), t(on(0, 3))), workspace=t(Space(k)), stream="side"),
    "kv_compact": lambda k, t: k.kv_compact(
        t(cache_on(k, 0)), t(on(0, 1, 2)), t(on(0, 1)), t(on(0, 3)), drop=t(on(0, 1, dtype=torch.uint8)),
        out=(t(on(0, 1, 2)), t(on(0, 1)), t(on(0, 3))), workspace=t(Space(k)), stream="side"),
    "kv_reserve": lambda k, t: k.kv_reserve(cache_on(k, 0), t(on(0, 1, 2)), t(on(0, 1)), t(on(0, 3)), add=t(on(0, 1)),
                                            workspace=t(Space(k)), stream="side"),
    "kv_free": lambda k, t: k.kv_free(cache_on(k, 0), t(on(0, 1, 2)), t(on(0, 1)), t(on(0, 3)),
                                      drop=t(on(0, 1, dtype=torch.uint8)), stream="side"),
    "beam_select": lambda k, t: k.beam_select(t(on(0, 2, 9, dtype=torch.float32)), t(on(0, 1, 2, dtype=torch.float32)), 2,
                                              workspace=t(Space(k)), stream="side"),
}


def Space(qgkv):
    w = qgkv.KVWorkspace.__new__(qgkv.KVWorkspace)
    w.buffer, w.ptr, w.bytes = on(0, 8, dtype=torch.uint8), 0, 8
    return w


@pytest.mark.parametrize("name", STREAMED)
def test_tensors_are_lent_to_the_stream_of_a_call(calls, monkeypatch, name):
    """A caller may drop a tensor right after a call on another stream (`table, lens, refs = kv_fork(...)`): its
    memory must not be used again before that stream is done."""
    import contextlib
    qgkv, made = calls
    lent, current = [], ["main"]

    @contextlib.contextmanager
    def enter(stream):
        current.append(stream)
        yield
        current.pop()

    monkeypatch.setattr(torch.cuda, "current_stream", lambda *a: current[-1])
    monkeypatch.setattr(torch.cuda, "stream", enter)
    monkeypatch.setattr(OnDevice, "record_stream", lambda self, stream: lent.append((self.data_ptr(), stream)), raising=False)
    monkeypatch.setattr(torch, "empty", lambda shape, dtype=None, device=None: on(0, *shape, dtype=dtype))
    given = []

    def take(x):
        if isinstance(x, qgkv.KVCache):
            given.extend((x.k, x.k_scale, x.v, x.v_scale))
        else:
            given.append(getattr(x, "buffer", x))
        return x

    STREAMED[name](qgkv, take)
    assert len(made) == 1 and current == ["main"]
    assert {(t.data_ptr(), "side") for t in given} <= set(lent)


def test_row_kernel_joins_its_warp_after_a_wait():
    """mma and movmatrix take whole warps; lanes leave a bounded wait one by one."""
    src = open(os.path.join(CSRC, "kv_rows.cuh")).read()
    at = src.index("if (!mbar_try_wait(bar + taken % S")
    body = re.sub(r"//[^\n]*", "", src[at:])
    depth, end = 0, 0
    for end, ch in enumerate(body):  # the end of the wait's block
        depth += {"{": 1, "}": -1}.get(ch, 0)
        if ch == "}" and depth == 0:
            break
    assert body[end + 1:].lstrip().startswith("__syncwarp();")
    assert "mma16816" not in body[:end]
