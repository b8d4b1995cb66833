"""More GPU tests of the decode-state operators: values, scales and sizes at the
ends of their ranges.  Helpers and tolerances are test_kv_gpu's."""
import math

import pytest

torch = pytest.importorskip("torch")

from test_kv_gpu import (DT, attention_ref, close, i32, kv, status_clean, ws)  # noqa: E402, F401

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
