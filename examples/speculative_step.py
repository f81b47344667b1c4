"""Speculative decoding over the library's operators, with random weights:

    python examples/speculative_step.py [--mode greedy|sampled|lookup] [--steps N]

Every step feeds each sequence its last accepted token and a few drafted ones in one pass:
per layer the rows' keys and values are appended to the paged 8-bit cache, attention reads
it, and the routed experts run on all rows; then the drafts are verified, and rejected ones
leave the cache by a shorter length.  The projections around them are plain products.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import mxfp4_routed_expert_topk_gb300 as moe  # noqa: E402

E, H, I, TOP_K = 32, 256, 128, 4                  # routed experts of a layer
LAYERS, HEADS, GROUP, DIM, PAGE = 2, 2, 4, 64, 16  # key/value heads, query heads for each
VOCAB, DRAFTS = 1000, 4


def norm(x):
    f = x.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6)).to(torch.bfloat16)


class Model:
    def __init__(self, seqs, max_tokens, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape, scale=1.0):
            return (torch.randn(shape, generator=g, device="cuda") * scale * shape[0] ** -0.5).to(torch.bfloat16)

        self.embed = torch.randn((VOCAB, H), generator=g, device="cuda").to(torch.bfloat16)
        self.head = weight(H, VOCAB, scale=4.0)
        self.qkv = [weight(H, (GROUP + 2) * HEADS * DIM) for _ in range(LAYERS)]
        self.out = [weight(GROUP * HEADS * DIM, H, scale=0.5) for _ in range(LAYERS)]
        self.router = [weight(H, E).t().contiguous() for _ in range(LAYERS)]
        self.pools = [moe.Pool(E, H, I) for _ in range(LAYERS)]
        for n, pool in enumerate(self.pools):
            moe.moe_pool_fill_synthetic(pool, seed + n)
        # a sequence's pages, one after the other; the cache and what the operators need beside it
        width = -(-max_tokens // PAGE)
        self.cache = moe.KvCache(seqs * width, LAYERS, HEADS, DIM, PAGE)
        self.table = torch.arange(seqs * width, dtype=torch.int32, device="cuda").view(seqs, width)
        rows = seqs * (DRAFTS + 1)
        self.ws_append = moe.workspace(moe.moe_kv_append_workspace_size())
        self.ws_attend = moe.workspace(moe.moe_kv_attention_workspace_size(self.cache, 32, HEADS * GROUP))
        self.ws_verify = moe.workspace(moe.moe_verify_workspace_size(seqs, rows))

    def forward(self, tokens, cu, old, table, max_rows):
        """Logits after each of `tokens` (rows cu[b] .. cu[b+1]-1 are sequence b's, which has old[b]
        tokens in the cache); at most 32 rows."""
        x = self.embed[tokens.long()]
        total = old + (cu[1:] - cu[:-1])
        for n in range(LAYERS):
            heads = (norm(x) @ self.qkv[n]).view(len(tokens), (GROUP + 2) * HEADS, DIM)
            q, k, v = heads.split([GROUP * HEADS, HEADS, HEADS], dim=1)
            moe.moe_kv_append(self.cache, n, k, v, cu, old, table, ws=self.ws_append)
            a = moe.moe_kv_attention(self.cache, n, q, cu, total, table, max_rows=max_rows, ws=self.ws_attend)
            x = x + a.flatten(1) @ self.out[n]
            y = norm(x)
            idx, w = moe.moe_route_topk(y, self.router[n], TOP_K)
            x = moe.moe_expert_forward_decode(self.pools[n], y, idx, w, residual=x)
        return norm(x) @ self.head

    def prompt(self, b, tokens):
        """Feed sequence b a prompt, 32 rows at a time; logits after each token."""
        out = []
        for at in range(0, len(tokens), 32):
            part = torch.tensor(tokens[at:at + 32], dtype=torch.int32, device="cuda")
            cu = torch.tensor([0, len(part)], dtype=torch.int32, device="cuda")
            old = torch.tensor([at], dtype=torch.int32, device="cuda")
            out.append(self.forward(part, cu, old, self.table[b:b + 1], len(part)))
        return torch.cat(out)

    def draft(self, token):
        """The draft model: the next token's distribution from the last token alone."""
        return torch.softmax((norm(self.embed[token]) @ self.head).float(), -1)


def look_up(history, n):
    """What followed the last token the last time it came up (the token itself if it did not)."""
    at = len(history) - 2
    while at >= 0 and history[at] != history[-1]:
        at -= 1
    found = history[at + 1:at + 1 + n] if at >= 0 else []
    return found + [history[-1]] * (n - len(found))


def generate(mode="greedy", seqs=4, prompt=20, steps=12, seed=0):
    """Returns (model, tokens of each sequence, accepted drafts of each step)."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = DRAFTS + 1
    m = Model(seqs, prompt + steps * rows + 1, seed)
    hist = torch.randint(0, VOCAB, (seqs, prompt), generator=g, device="cuda").tolist()
    for b in range(seqs):
        m.prompt(b, hist[b][:-1])
    cu = torch.arange(0, (seqs + 1) * rows, rows, dtype=torch.int32, device="cuda")
    taken = []
    for _ in range(steps):
        old = torch.tensor([len(h) - 1 for h in hist], dtype=torch.int32, device="cuda")  # (the last one is fed now)
        q = torch.zeros((seqs, rows, VOCAB), device="cuda")  # what the drafts were drawn from
        fed = torch.empty((seqs, rows), dtype=torch.int32, device="cuda")
        for b, h in enumerate(hist):
            fed[b, 0] = h[-1]
            if mode == "lookup":
                fed[b, 1:] = torch.tensor(look_up(h, DRAFTS), dtype=torch.int32)
        if mode != "lookup":
            for i in range(DRAFTS):
                q[:, i] = m.draft(fed[:, i].long())
                best = q[:, i].argmax(-1) if mode == "greedy" else torch.multinomial(q[:, i], 1, generator=g)[:, 0]
                fed[:, i + 1] = best.to(torch.int32)
        fed = fed.flatten()
        logits = m.forward(fed, cu, old, m.table, rows)
        if mode == "greedy":
            accepted, after = moe.moe_verify_greedy(logits, fed, cu, ws=m.ws_verify)
        else:
            p = torch.softmax(logits.float(), -1)
            u = torch.rand(seqs * rows, generator=g, device="cuda")
            us = torch.rand(seqs, generator=g, device="cuda")
            drawn_from = q.flatten(0, 1) if mode == "sampled" else None
            accepted, after = moe.moe_verify_sampled(p, drawn_from, fed, cu, u, us, ws=m.ws_verify)
        taken.append(accepted.tolist())
        drafts = fed.view(seqs, rows)[:, 1:].tolist()
        for h, d, n, t in zip(hist, drafts, taken[-1], after.tolist()):
            h.extend(d[:n] + [t])
    for ws in (m.ws_append, m.ws_attend, m.ws_verify):
        status = moe.moe_check_status(ws)
        if status != moe.MOE_OK:
            raise RuntimeError(moe.status_string(status))
    return m, hist, taken


def main():
    ap = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    ap.add_argument("--mode", choices=("greedy", "sampled", "lookup"), default="sampled")
    ap.add_argument("--steps", type=int, default=12)
    a = ap.parse_args()
    _, hist, taken = generate(a.mode, steps=a.steps)
    for n, t in enumerate(taken):
        print(f"step {n}: accepted drafts {t}")
    made = sum(t + 1 for step in taken for t in step)
    print(f"{made} tokens in {len(taken)} steps of {len(hist)} sequences")


if __name__ == "__main__":
    main()
