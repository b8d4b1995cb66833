"""Beam search with block-quantised weights and an 8-bit paged cache.

A TinyLlama-shaped decoder (RMSNorm, rotary positions, grouped-query attention,
SwiGLU) with synthetic Q4_K weights: the linear layers are the fused GEMVs of
``qgemv``, everything between them is ``qgkv`` - the rotary positions with the
cache's append, the attention with the pages that beams share read once, penalties and
masks of the logits, the selection over beams and vocabulary, and the fork of
the beams' pages.  torch holds the memory and does the embedding lookup.

    python examples/beam_decode.py [--layers 22] [--steps 32] [--beams 4] [--repetition 1.1] [--prompt 21]
"""
from __future__ import annotations

import argparse
import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

from block_quantised_weight_gb300 import qgemv, qgkv, synth  # noqa: E402


class Model:
    """Weights of a decoder with Q4_K matrices, and its cache."""

    def __init__(self, layers=22, hidden=2048, q_heads=32, kv_heads=4, ffn=5632, vocab=32000, pages=512,
                 page_tokens=16, fmt="e4m3", seed=0, device="cuda"):
        self.hidden, self.q_heads, self.kv_heads, self.dim = hidden, q_heads, kv_heads, hidden // q_heads
        self.vocab, self.device, self.eps = vocab, device, 1e-5
        g = torch.Generator(device=device).manual_seed(seed)
        kv = kv_heads * self.dim

        def q4k(rows, cols, at):
            return torch.from_numpy(synth.gen_q4k(rows, cols, seed * 1000 + at)).to(device)

        def norm():
            return 0.4 + 0.2 * torch.rand(hidden, device=device, generator=g)

        self.layers = [dict(q=q4k(hidden, hidden, 9 * i), k=q4k(kv, hidden, 9 * i + 1), v=q4k(kv, hidden, 9 * i + 2),
                            o=q4k(hidden, hidden, 9 * i + 3), gate=q4k(ffn, hidden, 9 * i + 4),
                            up=q4k(ffn, hidden, 9 * i + 5), down=q4k(hidden, ffn, 9 * i + 6), norm1=norm(), norm2=norm())
                       for i in range(layers)]
        self.head, self.norm = q4k(vocab, hidden, 8999), norm()
        self.embedding = torch.randn((vocab, hidden), device=device, generator=g)
        self.cache = qgkv.KVCache.allocate(layers, pages, kv_heads, page_tokens, self.dim, fmt, device=device)
        self.refs = torch.zeros(pages, dtype=torch.int32, device=device)
        self.workspace = qgkv.KVWorkspace(device)
        self.rope = qgkv.rotary_table(pages * page_tokens, self.dim, device=device)

    def step(self, tokens, table, lens, starts=None, groups=None):
        """Logits of `tokens` (at most four rows), which go behind each sequence's lens[b]
        tokens: one a sequence, or by `starts`.  The pages must be reserved.  groups: borders of
        sequences that share pages."""
        rows = tokens.shape[0]
        x = self.embedding[tokens.long()].contiguous()
        held = (lens + (1 if starts is None else starts[1:] - starts[:-1])).int()
        plan = None if groups is None else qgkv.kv_share(self.cache, table, held, groups, starts=starts)
        for i, w in enumerate(self.layers):
            q, k, v = qgemv.qgemv_q4k_fused_group([w["q"], w["k"], w["v"]], x, norm_weight=w["norm1"], eps=self.eps)
            q, k, v = (t.view(rows, -1, self.dim) for t in (q, k, v))
            q = qgkv.kv_append_rotary(self.cache, i, q, k, v, self.rope, table, lens, starts=starts)
            if plan is None:
                a = qgkv.kv_attention(self.cache, i, q, table, held, starts=starts, workspace=self.workspace)
            else:
                a = qgkv.kv_attention_shared(self.cache, i, q, table, held, plan, starts=starts, workspace=self.workspace)
            x = qgemv.qgemv_q4k_fused(w["o"], a.view(rows, self.hidden), residual=x)
            gate, up = qgemv.qgemv_q4k_fused_group([w["gate"], w["up"]], x, norm_weight=w["norm2"], eps=self.eps)
            x = qgemv.qgemv_q4k_fused(w["down"], gate, up=up, residual=x)
        return qgemv.qgemv_q4k_fused(self.head, x, norm_weight=self.norm, eps=self.eps)

    def prefill(self, prompt, table, lens):
        """Put `prompt` (one sequence) into the cache, four tokens a pass; logits of its last token."""
        for at in range(0, len(prompt), 4):
            part = torch.tensor(prompt[at:at + 4], dtype=torch.int32, device=self.device)
            n = torch.tensor([len(part)], dtype=torch.int32, device=self.device)
            starts = torch.tensor([0, len(part)], dtype=torch.int32, device=self.device)
            qgkv.kv_reserve(self.cache, table, lens, self.refs, add=n, workspace=self.workspace)
            logits = self.step(part, table, lens, starts=starts)
            lens += n
        return logits[-1:]


def beam_search(model, prompt, beams=4, steps=16, repetition=1.0, banned=()):
    """(scores, tokens) of the best `beams` continuations of `prompt` by `steps` tokens.  repetition: the penalty of
    tokens that came before, the prompt's among them; banned: tokens that are not produced."""
    dev, ws = model.device, model.workspace
    width = (len(prompt) + steps + model.cache.page_tokens) // model.cache.page_tokens + 1
    table = torch.full((1, width), -1, dtype=torch.int32, device=dev)
    lens = torch.zeros(1, dtype=torch.int32, device=dev)
    logits = model.prefill(prompt, table, lens)
    cum = torch.zeros((1, 1), device=dev)
    before = torch.tensor([prompt], dtype=torch.int32, device=dev)
    history = torch.empty((1, 0), dtype=torch.int32, device=dev)
    groups = torch.tensor([0, beams], dtype=torch.int32, device=dev)
    mask = None
    if len(banned):
        allowed = torch.ones((1, -(-model.vocab // 32) * 32), dtype=torch.int64, device=dev)
        allowed[0, list(banned)] = 0
        bits = (allowed.view(1, -1, 32) << torch.arange(32, device=dev)).sum(-1)
        mask = torch.where(bits >= 1 << 31, bits - (1 << 32), bits).int()
    for _ in range(steps):
        if repetition != 1.0 or mask is not None:
            n = logits.shape[0]
            said = torch.cat((before.expand(n, -1), history), dim=1)
            logits = qgkv.adjust_logits(
                logits, history=said, lens=torch.full((n,), said.shape[1], dtype=torch.int32, device=dev),
                repetition=torch.full((n,), repetition, device=dev), mask=mask,
                mask_rows=None if mask is None else torch.zeros(n, dtype=torch.int32, device=dev))
        scores, tokens, parents = qgkv.beam_select(logits, cum, beams, workspace=ws)
        # the beams continue their parents: pages are shared, the partly filled last one is copied
        table, lens, model.refs = qgkv.kv_fork(model.cache, table, lens, parents.view(-1), model.refs, workspace=ws)
        history = torch.cat((history[parents.view(-1).long()], tokens.view(-1, 1)), dim=1)
        cum = scores
        if history.shape[1] == steps:
            break
        qgkv.kv_reserve(model.cache, table, lens, model.refs, workspace=ws)
        logits = model.step(tokens.view(-1), table, lens, groups=groups)
        lens += 1
    qgkv.kv_free(model.cache, table, lens, model.refs)
    if qgemv.qg_device_status() != qgemv.QG_OK:
        raise RuntimeError("the decode ran out of pages or met a bad index")
    return scores[0], history


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    p.add_argument("--layers", type=int, default=22)
    p.add_argument("--steps", type=int, default=32)
    p.add_argument("--beams", type=int, default=4, choices=range(1, 5))
    p.add_argument("--repetition", type=float, default=1.0)
    p.add_argument("--prompt", type=int, default=21, help="tokens of the prompt")
    p.add_argument("--fmt", default="e4m3", choices=sorted(qgkv.FORMATS))
    a = p.parse_args()
    model = Model(layers=a.layers, fmt=a.fmt, pages=512 + a.prompt // 16)
    prompt = [(7 * i * i + 3) % model.vocab for i in range(a.prompt)]
    beam_search(model, prompt, a.beams, 2, a.repetition)  # first use
    begin, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    begin.record()
    scores, tokens = beam_search(model, prompt, a.beams, a.steps, a.repetition)
    end.record()
    torch.cuda.synchronize()
    for s, t in zip(scores.tolist(), tokens.tolist()):
        print(f"{s:10.4f}  {t}")
    print(f"{a.beams} beams x {a.steps} tokens behind a prompt of {len(prompt)} in {begin.elapsed_time(end):.1f} ms")


if __name__ == "__main__":
    main()
