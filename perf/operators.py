"""The operators of a speculative serving step around the routed-expert layer, as cases to time.

A serving step of a few rows per sequence (one accepted token and its drafts) does, in every layer, what
these cases hold: the new rows' keys and values are appended to a paged cache of E4M3 codes with one fp32
scale per page, head and side; the rows' queries attend over that cache, causally among themselves; and
after the last layer the drafts are verified against the target's probabilities with given random numbers.

Each case runs in a plain form (elementary torch operations in 32 bits) or, with `own` set, through the
package's entry points.  A page holds, for each layer, the codes [2][heads][page][dim] (keys, then values),
then the scales [2][heads] in fp32, padded to 128 bytes.
"""
import math
import random

import torch

own = False

FP8 = torch.float8_e4m3fn
GRID = 38  # probabilities are read as whole multiples of 2^-38


# ------------------------------------------------------------------------------- cases


def listed():
    return [
        # one short conversation, one token: the call's latency
        _attn("attend_1x1_300", 1, 1, 300, 300, 8, 7, 128, 64),
        # ordinary batched decode: 64 conversations of very different lengths, one token each
        _attn("attend_64x1_16k", 64, 1, 1, 16384, 8, 7, 128, 64),
        # drafted rows (one accepted token and four drafts) over odd lengths, small pages
        _attn("attend_24x5_9k", 24, 5, 700, 9001, 8, 7, 128, 32),
        # the widest verification batch over long documents
        _attn("attend_4x17_128k", 4, 17, 120001, 131072, 8, 7, 128, 128),
        # narrow heads, few of them, smallest pages, ragged row counts
        _attn("attend_48x9_64d", 48, 9, 1, 8191, 4, 8, 64, 16, ragged=True),
        # a decode step's rows into the cache
        _append("append_64x1", 64, 1, 1, 16384, 8, 128, 64),
        # a verification batch's rows, crossing page ends
        _append("append_32x17", 32, 17, 0, 9000, 8, 128, 32),
        # several prompts at once, odd lengths
        _append("append_6x8191", 6, 8191, 0, 0, 8, 128, 64, ragged=True),
        # one conversation with four drafts
        _verify("verify_1x5", 1, 5, 32001, "sampled", "fp32"),
        # a batch of conversations with draft probabilities, odd vocabulary
        _verify("verify_64x9", 64, 9, 131071, "sampled", "fp32", ragged=True),
        # drafts without probabilities (looked up, not sampled), 16-bit target
        _verify("verify_96x5_lookup", 96, 5, 65536, "lookup", "bf16"),
        # greedy verification on 16-bit logits: the reference point of identical output
        _verify("verify_8x17_greedy", 8, 17, 131072, "greedy", "bf16"),
    ]


def _attn(name, seqs, rows, lo, hi, heads, group, dim, page, ragged=False, layers=1):
    return {"name": name, "op": "attend", "seqs": seqs, "rows": rows, "lo": lo, "hi": hi, "heads": heads, "group": group,
            "dim": dim, "page": page, "ragged": ragged, "layers": layers}


def _append(name, seqs, rows, lo, hi, heads, dim, page, ragged=False, layers=1):
    return {"name": name, "op": "append", "seqs": seqs, "rows": rows, "lo": lo, "hi": hi, "heads": heads,
            "dim": dim, "page": page, "ragged": ragged, "layers": layers}


def _verify(name, seqs, rows, vocab, mode, dtype, ragged=False):
    return {"name": name, "op": "verify", "seqs": seqs, "rows": rows, "vocab": vocab, "mode": mode, "dtype": dtype,
            "ragged": ragged}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("attend", "attend", "append", "verify", "verify"))
    if op == "verify":
        mode = rng.choice(("sampled", "lookup", "greedy"))
        vocab, rows = _log_int(rng, 1000, 160001), rng.randint(1, 17)
        seqs = _log_int(rng, 1, max(1, min(96, 40_000_000 // (vocab * rows))))
        c = _verify("", seqs, rows, vocab, mode, rng.choice(("fp32", "bf16")), rng.random() < 0.5)
    else:
        heads, dim = rng.choice((1, 2, 4, 8)), rng.choice((64, 128, 128))
        page, layers = rng.choice((16, 32, 64, 128)), rng.choice((1, 1, 2))
        if op == "attend":
            rows, group = rng.choice((1, 1, 2, 5, 9, 17, rng.randint(1, 17))), rng.choice((1, 2, 4, 7, 8, 16))
            hi = _log_int(rng, 17, 131072)
            seqs = _log_int(rng, 1, max(1, min(96, 400_000 // hi)))
            c = _attn("", seqs, rows, rng.choice((1, max(1, hi // 2), hi)), hi, heads, group, dim, page, rng.random() < 0.4, layers)
        else:
            rows = _log_int(rng, 1, 8192)
            seqs = _log_int(rng, 1, max(1, min(96, 40_000 // rows)))
            hi = rng.choice((0, 500, 4001))
            c = _append("", seqs, rows, rng.choice((0, hi)), hi, heads, dim, page, rng.random() < 0.5, layers)
    del c["name"]
    return c


def _shape(case):
    """The lengths a case stands for: (rows of each sequence, tokens cached before them)."""
    r = random.Random("%(op)s %(seqs)d %(rows)d" % case)
    n = [r.randint(1, case["rows"]) if case["ragged"] and b else case["rows"] for b in range(case["seqs"])]
    if case["op"] == "verify":
        return n, None
    lo, hi = case["lo"], case["hi"]
    old = [hi if b == 0 else r.randint(lo, hi) for b in range(case["seqs"])]
    if case["op"] == "attend":  # lo..hi counts the new rows too
        old = [max(0, t - m) for t, m in zip(old, n)]
    return n, old


def work(case):
    n, old = _shape(case)
    rows = sum(n)
    if case["op"] == "verify":
        size = 4 if case["dtype"] == "fp32" else 2
        if case["mode"] == "greedy":  # every row up to a mismatch: all of them at most
            return {"bytes": rows * case["vocab"] * size + 8 * rows, "flops": rows * case["vocab"]}
        sides = 2 if case["mode"] == "sampled" else 1  # one row of the target and one of the draft per sequence
        return {"bytes": case["seqs"] * case["vocab"] * size * sides + 24 * rows, "flops": 4 * case["seqs"] * case["vocab"]}
    H, D, P = case["heads"], case["dim"], case["page"]
    if case["op"] == "append":
        pages = sum((o + m + P - 1) // P - o // P for m, o in zip(n, old))
        return {"bytes": rows * H * D * 2 * 3 + pages * H * 8 + rows * 4, "flops": rows * H * D * 2 * 2}
    Hq = H * case["group"]
    kv = sum(m + o for m, o in zip(n, old))
    pairs = sum(m * o + m * (m + 1) // 2 for m, o in zip(n, old))
    return {"bytes": kv * H * D * 2 + -(-kv // P) * H * 8 + rows * Hq * D * 4, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------------------ inputs


def _offsets(n):
    at = [0]
    for m in n:
        at.append(at[-1] + m)
    return torch.tensor(at, dtype=torch.int32, device="cuda")


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, old = _shape(case)
    s = {"case": case, "n": n, "old": old, "cu": _offsets(n), "max_rows": max(n)}
    return _prepare_verify(s, case, g) if case["op"] == "verify" else _prepare_cache(s, case, g)


def _prepare_cache(s, case, g):
    n, old, P, H, D, L = s["n"], s["old"], case["page"], case["heads"], case["dim"], case["layers"]
    rows, layer = sum(n), case["layers"] - 1
    width = max((o + m + P - 1) // P for o, m in zip(old, n))
    used = [(o + m + P - 1) // P for o, m in zip(old, n)]
    pages = sum(used) + 3
    codes = 2 * H * P * D
    record = -(-(codes + 8 * H) // 128) * 128
    pool = torch.zeros((pages, L * record), dtype=torch.uint8, device="cuda")
    view = pool.view(pages, L, record)[:, layer]
    step = max(1, (1 << 28) // codes)
    for at in range(0, pages, step):  # values of about N(0, 1) times a page's own power of two
        some = view[at:at + step]
        v = torch.randn((some.shape[0], codes), generator=g, device="cuda").mul_(56.0).clamp_(-448, 448)
        some[:, :codes] = v.to(FP8).view(torch.uint8)
    e = torch.randint(-7, -4, (pages, 2 * H), generator=g, device="cuda")
    view[:, codes:codes + 8 * H].view(torch.float32).copy_(torch.exp2(e.float()))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)  # pages lie anywhere in the pool
    at, table = 0, torch.full((len(n), max(width, 1)), -1, dtype=torch.int32, device="cuda")
    for b, u in enumerate(used):
        table[b, :u] = order[at:at + u]
        at += u
    s.update(pool=pool, table=table, layer=layer, record=record, start=torch.tensor(old, dtype=torch.int32, device="cuda"),
             total=torch.tensor([o + m for o, m in zip(old, n)], dtype=torch.int32, device="cuda"))
    if case["op"] == "attend":
        Hq = H * case["group"]
        s["q"] = torch.randn((rows, Hq, D), generator=g, device="cuda").mul_(1.5).to(torch.bfloat16)
        s["scale"] = D ** -0.5
    else:  # keys and values as slices of one projection's output; some heads are much larger than others
        kv = torch.randn((rows, 2 * H, D), generator=g, device="cuda")
        kv *= torch.exp2(torch.randint(-3, 4, (1, 2 * H, 1), generator=g, device="cuda").float())
        s["kv"] = kv.to(torch.bfloat16)
    return s


def _prepare_verify(s, case, g):
    n, V, dt = s["n"], case["vocab"], torch.float32 if case["dtype"] == "fp32" else torch.bfloat16
    R = sum(n)
    x = torch.randn((R, V), generator=g, device="cuda").mul_(3.0)
    s["last"] = s["cu"][1:].long() - 1
    if case["mode"] == "greedy":
        s["p"] = x.to(dt)
        best = _first_max(s["p"].float())
        other = torch.randint(0, V, (R,), generator=g, device="cuda")
        drafted = torch.where(torch.rand(R, generator=g, device="cuda") < 0.9, best, other)
    else:
        s["p"] = torch.softmax(x, -1).to(dt)
        y = torch.softmax(x.add_(torch.randn((R, V), generator=g, device="cuda"), alpha=0.4), -1)
        drafted = torch.multinomial(y, 1, generator=g)[:, 0]
        if case["mode"] == "sampled":
            s["q"] = y.to(dt)
        else:  # a looked-up draft is right most of the time where the target is sure
            drafted = torch.where(torch.rand(R, generator=g, device="cuda") < 0.6, _first_max(s["p"].float()), drafted)
    # row r of a sequence was fed token r; the draft that follows it is token r + 1
    tok = torch.randint(0, V, (R,), generator=g, device="cuda")
    tok[1:] = drafted[:-1]
    s["tok"] = tok.to(torch.int32)
    s["u"] = torch.rand(R, generator=g, device="cuda")
    s["us"] = torch.rand(len(n), generator=g, device="cuda")
    return s


def _first_max(x):
    m = x.amax(-1, keepdim=True)
    at = torch.arange(x.shape[1], device=x.device, dtype=torch.int32)
    return torch.where(x == m, at, x.shape[1]).amin(-1).long()


# -------------------------------------------------------------------------------- runs


def run(s):
    if own:
        return _run_own(s)
    op = s["case"]["op"]
    if op == "attend":
        return _attend_plain(s)
    if op == "append":
        return _append_plain(s)
    return _greedy_plain(s) if s["case"]["mode"] == "greedy" else _verify_plain(s)


def _run_own(s):
    import mxfp4_routed_expert_topk_gb300 as moe

    c = s["case"]
    if "ws" not in s:  # what a program makes once: the cache's view and a workspace
        if c["op"] != "verify":
            s["cache"] = moe.KvCache(s["pool"].shape[0], c["layers"], c["heads"], c["dim"], c["page"], buffer=s["pool"])
        if c["op"] == "attend":
            size = moe.moe_kv_attention_workspace_size(s["cache"], s["max_rows"], c["heads"] * c["group"])
        elif c["op"] == "append":
            size = moe.moe_kv_append_workspace_size()
        else:
            size = moe.moe_verify_workspace_size(c["seqs"], len(s["tok"]))
        s["ws"] = moe.workspace(size)
    if c["op"] == "attend":
        return moe.moe_kv_attention(s["cache"], s["layer"], s["q"], s["cu"], s["total"], s["table"], max_rows=s["max_rows"],
                                    scale=s["scale"], ws=s["ws"])
    if c["op"] == "append":
        H = c["heads"]
        moe.moe_kv_append(s["cache"], s["layer"], s["kv"][:, :H], s["kv"][:, H:], s["cu"], s["start"], s["table"], ws=s["ws"])
        return _cache_out(s)
    if c["mode"] == "greedy":
        return moe.moe_verify_greedy(s["p"], s["tok"], s["cu"], ws=s["ws"])
    return moe.moe_verify_sampled(s["p"], s.get("q"), s["tok"], s["cu"], s["u"], s["us"], ws=s["ws"])


def _cache_view(s):
    """(codes [pages][2][heads][page][dim] as bytes, scales [pages][2][heads]) of the case's layer."""
    c = s["case"]
    H, P, D = c["heads"], c["page"], c["dim"]
    rec = s["pool"].view(-1, c["layers"], s["record"])[:, s["layer"]]
    n = 2 * H * P * D
    return rec[:, :n].unflatten(1, (2, H, P, D)), rec[:, n:n + 8 * H].view(torch.float32).unflatten(1, (2, H))


def _cache_out(s):
    codes, scales = _cache_view(s)
    return {"codes": codes.view(FP8), "scales": scales}


def _attend_plain(s):
    c = s["case"]
    H, P, D, G = c["heads"], c["page"], c["dim"], c["group"]
    codes, scales = _cache_view(s)
    pages = s["table"].clamp(min=0).long()
    B, L, N = pages.shape[0], pages.shape[1] * P, s["max_rows"]
    sc = scales[pages]  # [B][width][2][H]
    k = codes[:, 0][pages].view(FP8).float().mul_(sc[:, :, 0, :, None, None]).transpose(1, 2).reshape(B, H, L, D)
    v = codes[:, 1][pages].view(FP8).float().mul_(sc[:, :, 1, :, None, None]).transpose(1, 2).reshape(B, H, L, D)
    cu, total = s["cu"].long(), s["total"].long()
    i = torch.arange(N, device="cuda")
    n = cu[1:] - cu[:-1]
    row = torch.where(i < n[:, None], cu[:-1, None] + i, 0)  # [B][N]
    q = s["q"].float()[row].view(B, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, N * G, D)
    x = torch.matmul(q, k.transpose(2, 3)).mul_(s["scale"]).view(B, H, N, G, L)
    sees = torch.arange(L, device="cuda") <= (total - n)[:, None, None] + i[:, None]  # [B][N][L]
    x = x.masked_fill_(~sees[:, None, :, None], -math.inf)
    p = torch.exp(x.sub_(x.amax(-1, keepdim=True)))
    o = torch.matmul(p.view(B, H, N * G, L), v).view(B, H, N, G, D) / p.sum(-1, keepdim=True)
    seq = torch.searchsorted(cu[1:], torch.arange(len(s["q"]), device="cuda"), right=True)
    at = torch.arange(len(s["q"]), device="cuda") - cu[seq]
    return o.permute(0, 2, 1, 3, 4).reshape(B, N, H * G, D)[seq, at].to(torch.bfloat16)


def _append_plain(s):
    c = s["case"]
    H, P = c["heads"], c["page"]
    codes, scales = _cache_view(s)
    cu, start, table = s["cu"].long(), s["start"].long(), s["table"].long()
    R = len(s["kv"])
    r = torch.arange(R, device="cuda")
    seq = torch.searchsorted(cu[1:], r, right=True)
    pos = start[seq] + r - cu[seq]
    page, off = table[seq, pos // P], pos % P
    x = s["kv"].float().unflatten(1, (2, H))  # [R][2][H][D]
    amax = torch.zeros_like(scales).index_reduce_(0, page, x.abs().amax(-1), "amax")
    # the smallest power of two 2^e with amax <= 448 * 2^e, no smaller than 2^-126
    m, e = torch.frexp(amax)  # amax = m * 2^e, 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875), -126).clamp(min=-126)
    fresh = torch.ldexp(torch.ones_like(amax), e)
    # a sequence's first page may hold older tokens: its scale only grows, and they follow it
    first = table[torch.arange(len(start), device="cuda"), (start // P).clamp(max=table.shape[1] - 1)].clamp(min=0)
    keep = torch.where((torch.arange(P, device="cuda") < (start % P)[:, None]) & (cu[1:] > cu[:-1])[:, None], 1, 0)
    was = scales[first]
    now = torch.where((keep.sum(1) > 0)[:, None, None], torch.maximum(was, fresh[first]), fresh[first])
    new = fresh.index_put((first,), now)
    olds = codes[first]  # [B][2][H][P][D]
    moved = (olds.view(FP8).float() * (was / now)[..., None, None]).to(FP8).view(torch.uint8)
    codes[first] = torch.where(keep[:, None, None, :, None] > 0, moved, olds)
    touched = torch.zeros(len(scales), dtype=torch.bool, device="cuda").index_fill_(0, page, True)
    scales.copy_(torch.where(touched[:, None, None], new, scales))
    q = (x / new[page][..., None]).clamp_(-448, 448).to(FP8).view(torch.uint8)
    codes[page, :, :, off] = q
    return _cache_out(s)


def _whole(p):
    return (p.float().nan_to_num(0.0, 1.0, 0.0).clamp(0, 1) * 2.0 ** GRID).to(torch.int64)


def _verify_plain(s):
    p, q, tok, cu, V = s["p"], s.get("q"), s["tok"].long(), s["cu"].long(), s["case"]["vocab"]
    R, B = len(tok), len(cu) - 1
    r = torch.arange(R, device="cuda")
    seq = torch.searchsorted(cu[1:], r, right=True)
    last = r == cu[1:][seq] - 1
    draft = tok[(r + 1).clamp(max=R - 1)]
    m = (s["u"] * 2.0 ** 24).to(torch.int64).clamp(0, 2 ** 24 - 1)
    pt = _whole(p.gather(1, draft[:, None])[:, 0])
    qt = _whole(q.gather(1, draft[:, None])[:, 0]) if q is not None else torch.full_like(pt, 1 << GRID)
    ok = (m * qt < (pt << 24)) & ~last
    stop = torch.full((B,), R, device="cuda").scatter_reduce_(0, seq, torch.where(ok, R, r), "amin")
    full = _whole(p[stop])
    left = (full - _whole(q[stop])).clamp(min=0) if q is not None else full.scatter(1, draft[stop][:, None], 0)
    left = torch.where(last[stop][:, None] | (left.sum(-1, keepdim=True) == 0), full, left)
    total = left.sum(-1)
    us = (s["us"] * 2.0 ** 24).to(torch.int64).clamp(0, 2 ** 24 - 1)
    aim = (total >> 24) * us + (((total & (2 ** 24 - 1)) * us) >> 24)
    token = (left.cumsum(-1) <= aim[:, None]).sum(-1)
    token = torch.where(total > 0, token, -1)
    return (stop - cu[:-1]).to(torch.int32), token.to(torch.int32)


def _greedy_plain(s):
    tok, cu = s["tok"].long(), s["cu"].long()
    R, B = len(tok), len(cu) - 1
    best = _first_max(s["p"].float())
    r = torch.arange(R, device="cuda")
    seq = torch.searchsorted(cu[1:], r, right=True)
    ok = (best == tok[(r + 1).clamp(max=R - 1)]) & (r != cu[1:][seq] - 1)
    stop = torch.full((B,), R, device="cuda").scatter_reduce_(0, seq, torch.where(ok, R, r), "amin")
    return (stop - cu[:-1]).to(torch.int32), best[stop].to(torch.int32)


# ------------------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "verify":
        return _exact_verify(s, case)
    P, H, D = case["page"], case["heads"], case["dim"]
    size = 2 * H * P * D
    rec = s["pool"].reshape(-1, case["layers"], s["record"])[:, s["layer"]].contiguous()
    codes = rec[:, :size].contiguous().view(FP8).double().reshape(-1, 2, H, P, D)
    scales = rec[:, size:size + 8 * H].contiguous().view(torch.float32).double().reshape(-1, 2, H)
    table = s["table"].tolist()
    if case["op"] == "append":
        return _exact_append(s, codes, scales, table)
    outs, at = [], 0
    for b, (m, o) in enumerate(zip(s["n"], s["old"])):
        total, ids = o + m, table[b][:(o + m + P - 1) // P]
        kv = (codes[ids] * scales[ids][..., None, None]).permute(1, 2, 0, 3, 4).reshape(2, H, -1, D)[:, :, :total]
        q = s["q"][at:at + m].double().reshape(m, H, case["group"], D)
        x = torch.einsum("mhgd,htd->hgmt", q, kv[0]) * s["scale"]
        x = x + torch.full((m, total), -math.inf, dtype=torch.float64, device="cuda").triu(o + 1)
        outs.append(torch.einsum("hgmt,htd->mhgd", torch.softmax(x, -1), kv[1]).reshape(m, -1, D))
        at += m
    return torch.cat(outs)


def _exact_append(s, codes, scales, table):
    P, at = s["case"]["page"], 0
    x = s["kv"].double().reshape(len(s["kv"]), 2, -1, s["case"]["dim"])
    for b, (m, o) in enumerate(zip(s["n"], s["old"])):
        for first in range(o // P, (o + m - 1) // P + 1):
            lo, hi = max(o, first * P), min(o + m, (first + 1) * P)
            page, part = table[b][first], x[at + lo - o:at + hi - o].permute(1, 2, 0, 3)
            big = part.abs().amax((-1, -2))
            sc = torch.exp2(torch.ceil(torch.log2(big / 448)).clamp(min=-126))
            sc = torch.where(sc * 224 >= big, sc / 2, sc).clamp(min=2.0 ** -126)  # in case the logarithm rounds up
            sc = torch.where(sc * 448 < big, sc * 2, sc)
            if lo % P:
                sc = torch.maximum(sc, scales[page])
                codes[page][:, :, :lo % P] = _round8(codes[page][:, :, :lo % P] * (scales[page] / sc)[..., None, None])
            codes[page][:, :, lo - first * P:hi - first * P] = _round8(part / sc[..., None, None])
            scales[page] = sc
        at += m
    return {"codes": codes, "scales": scales}


def _round8(x):
    """The nearest E4M3 value (ties to even), in 64 bits."""
    step = torch.exp2(torch.floor(torch.log2(x.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(x / step) * step).clamp(-448, 448)


def _exact_verify(s, case):
    tok, cu, V = s["tok"].tolist(), s["cu"].tolist(), case["vocab"]
    whole = lambda x: torch.floor(x.double() * 2.0 ** GRID).to(torch.int64)  # noqa: E731
    took, token = [], []
    for b in range(case["seqs"]):
        r, end = cu[b], cu[b + 1]
        while True:
            if case["mode"] == "greedy":
                x = s["p"][r].double()
                best = int((x == x.max()).nonzero()[0, 0])
                if r + 1 < end and best == tok[r + 1]:
                    r += 1
                    continue
                token.append(best)
                break
            P = whole(s["p"][r])
            if r + 1 == end:
                left = P
            else:
                d, m = tok[r + 1], math.floor(float(s["u"][r].double()) * 2 ** 24)
                Q = whole(s["q"][r]) if "q" in s else None
                if m * (int(Q[d]) if Q is not None else 1 << GRID) < int(P[d]) << 24:
                    r += 1
                    continue
                left = P.clone()
                if Q is None:
                    left[d] = 0
                else:
                    left = torch.clamp(P - Q, min=0)
                left = left if int(left.sum()) else P
            total = int(left.sum())
            aim = total * math.floor(float(s["us"][b].double()) * 2 ** 24) >> 24
            token.append(int(torch.searchsorted(left.cumsum(0), torch.tensor([aim], device="cuda"), right=True)[0]) if total else -1)
            break
        took.append(r - cu[b])
    return torch.tensor(took, dtype=torch.int32), torch.tensor(token, dtype=torch.int32)
