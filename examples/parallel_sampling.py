"""Several continuations of each of a few prompts, sampled side by side, with random weights:

    python examples/parallel_sampling.py [--temperature T] [--top-p P] [--samples N] [--steps N]

A prompt is fed once; its whole pages go into every sample's page table.  Every step then finds pages for one
row of each sample that still runs, appends, attends with the prompts' pages read once for all of their
samples, runs the experts, and draws the next tokens.  A sample that ends gives its pages back.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.abspath(__file__)))
import speculative_step as base  # noqa: E402
from speculative_step import moe, norm  # noqa: E402

PAGE, VOCAB, ROWS = base.PAGE, base.VOCAB, 32  # rows: what one pass of the experts takes


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


class Model(base.Model):
    """The model with pages from a pool that all sequences take from."""

    def __init__(self, seqs, max_tokens, seed=0):
        super().__init__(seqs, max_tokens, seed)
        self.refs = torch.zeros(self.cache.n_pages, dtype=torch.int32, device="cuda")
        self.table.fill_(-1)
        self.lens = torch.zeros(seqs, dtype=torch.int32, device="cuda")
        self.ws_pages = moe.workspace(moe.moe_kv_pages_workspace_size(seqs, self.cache.n_pages))
        self.ws_shared = moe.workspace(moe.moe_kv_attention_shared_workspace_size(self.cache, ROWS, ROWS, ROWS,
                                                                                  base.HEADS * base.GROUP))
        self.ws_sample = moe.workspace(moe.moe_sample_workspace_size(ROWS, VOCAB))

    def feed(self, tokens, new_rows, groups, prefix):
        """Logits after each of `tokens`, of which sequence b takes new_rows[b]."""
        cu, total, *_ = moe.moe_kv_reserve(new_rows, self.lens, self.table, self.refs, PAGE, len(tokens), ws=self.ws_pages)
        x = self.embed[tokens.long()]
        for n in range(base.LAYERS):
            heads = (norm(x) @ self.qkv[n]).view(len(tokens), (base.GROUP + 2) * base.HEADS, base.DIM)
            q, k, v = heads.split([base.GROUP * base.HEADS, base.HEADS, base.HEADS], dim=1)
            moe.moe_kv_append(self.cache, n, k, v, cu, self.lens, self.table, ws=self.ws_append)
            a = moe.moe_kv_attention_shared(self.cache, n, q, cu, total, self.table, groups, prefix, max_rows=ROWS,
                                            max_group_rows=ROWS, ws=self.ws_shared)
            x = x + a.flatten(1) @ self.out[n]
            y = norm(x)
            idx, w = moe.moe_route_topk(y, self.router[n], base.TOP_K)
            x = moe.moe_expert_forward_decode(self.pools[n], y, idx, w, residual=x)
        self.lens = total
        return norm(x) @ self.head

    def feed_one(self, b, tokens, groups, prefix):
        """Feed sequence b its tokens, 32 at a time; logits after the last."""
        new_rows = torch.zeros_like(self.lens)
        for at in range(0, len(tokens), ROWS):
            part = tokens[at:at + ROWS]
            new_rows[b] = len(part)
            logits = self.feed(ints(part), new_rows, groups, prefix)
        return logits[-1:]

    def status(self):
        for ws in (self.ws_pages, self.ws_append, self.ws_shared, self.ws_sample):
            code = moe.moe_check_status(ws)
            if code != moe.MOE_OK:
                raise RuntimeError(moe.status_string(code))


def generate(temperature=0.8, top_p=0.95, samples=4, prompts=(37, 20), steps=24, stop=0.05, seed=0):
    """Returns (model, the sequences' tokens).  A sample stops after any of the first stop * VOCAB tokens."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    seqs = samples * len(prompts)
    m = Model(seqs, max(prompts) + steps + 1, seed)
    groups = ints([i * samples for i in range(len(prompts) + 1)])
    prefix = ints(list(prompts))
    alone, none = torch.arange(seqs + 1, dtype=torch.int32, device="cuda"), torch.zeros(seqs, dtype=torch.int32, device="cuda")
    hist, logits = [], []
    for p, n in enumerate(prompts):
        text, first, whole = torch.randint(0, VOCAB, (n,), generator=g, device="cuda").tolist(), p * samples, n // PAGE
        last = m.feed_one(first, text, alone, none)
        for b in range(first + 1, first + samples):  # the whole pages are shared, the rest is each sample's own
            m.table[b, :whole] = m.table[first, :whole]
            m.refs[m.table[first, :whole].long()] += 1
            m.lens[b] = whole * PAGE
            if n > whole * PAGE:
                m.feed_one(b, text[whole * PAGE:], alone, none)
        logits += [last] * samples
        hist += [list(text) for _ in range(samples)]
    logits = torch.cat(logits)
    runs = torch.ones(seqs, dtype=torch.bool, device="cuda")
    t, tp = torch.full((seqs,), temperature, device="cuda"), torch.full((seqs,), top_p, device="cuda")
    for _ in range(steps):
        # (a sample that has ended has no row: its setting is not used)
        at = runs.nonzero()[:, 0]
        u = torch.rand(seqs, generator=g, device="cuda")
        token = moe.moe_sample(logits, t[at], u[at], top_p=tp[at], ws=m.ws_sample)
        for b, x in zip(at.tolist(), token.tolist()):
            hist[b].append(x)
        ends = token < int(stop * VOCAB)
        runs[at[ends]] = False
        keep = torch.where(runs, m.lens, 0).to(torch.int32)
        moe.moe_kv_release(keep, m.lens, m.table, m.refs, PAGE, ws=m.ws_pages)
        m.lens = keep
        if not bool(runs.any()):
            break
        logits = m.feed(token[~ends], runs.to(torch.int32), groups, prefix)
    m.status()
    return m, hist


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--temperature", type=float, default=0.8)
    ap.add_argument("--top-p", type=float, default=0.95)
    ap.add_argument("--samples", type=int, default=4)
    ap.add_argument("--steps", type=int, default=24)
    a = ap.parse_args()
    m, hist = generate(a.temperature, a.top_p, a.samples, steps=a.steps)
    for b, h in enumerate(hist):
        print(f"sample {b}: {len(h)} tokens, the last {h[-8:]}")
    print(f"{int((m.refs > 0).sum())} pages held by {int((m.lens > 0).sum())} samples that still run")


if __name__ == "__main__":
    main()
