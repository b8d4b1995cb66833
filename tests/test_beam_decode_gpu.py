"""The decode example end to end: beams that fork, share and copy pages have
the scores that their own tokens get without any of it."""
import os
import sys

import pytest

torch = pytest.importorskip("torch")

from block_quantised_weight_gb300 import build, qgemv  # noqa: E402

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt, prompt_tokens, steps", [("e4m3", 13, 9), ("int8", 16, 20), ("e4m3", 1, 18)])
def test_beam_search_scores_are_those_of_its_tokens(fmt, prompt_tokens, steps):
    """The search's cumulative scores against log-softmax sums (64 bits) of the same tokens
    decoded as four independent sequences with pages of their own.  The two decodes cut the
    attention's tokens differently, so values differ in their last bits, and a code of the cache
    can fall on the other side of a rounding (a step of 2^-4 of one value): 0.05 of a score."""
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    build.build()
    import beam_decode
    from block_quantised_weight_gb300 import qgkv
    small = dict(layers=2, hidden=256, q_heads=4, kv_heads=2, ffn=512, vocab=1000, pages=64, fmt=fmt, seed=3)
    model = beam_decode.Model(**small)
    prompt = [(31 * i + 5) % 1000 for i in range(prompt_tokens)]
    scores, tokens = beam_decode.beam_search(model, prompt, beams=4, steps=steps)
    assert (scores[:-1] >= scores[1:]).all()
    assert len({tuple(t) for t in tokens.tolist()}) == 4
    assert (model.refs == 0).all()

    other = beam_decode.Model(**small)
    width = 8
    table = torch.full((4, width), -1, dtype=torch.int32, device="cuda")
    lens = torch.zeros(4, dtype=torch.int32, device="cuda")
    for b in range(4):  # the prompt four times, each with pages of its own
        row, n = table[b:b + 1], lens[b:b + 1]
        logits = other.prefill(prompt, row, n)
    logits = logits.expand(4, -1).contiguous()
    want = torch.zeros(4, dtype=torch.float64, device="cuda")
    for t in range(steps):
        want += torch.log_softmax(logits.double(), -1).gather(1, tokens[:, t:t + 1].long())[:, 0]
        if t + 1 < steps:
            qgkv.kv_reserve(other.cache, table, lens, other.refs, workspace=other.workspace)
            logits = other.step(tokens[:, t].contiguous(), table, lens)
            lens += 1
    assert qgemv.qg_device_status() == qgemv.QG_OK
    assert ((scores.double() - want).abs() <= 0.05).all(), (scores, want)
