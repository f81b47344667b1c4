"""Operators of a batch that samples several continuations of shared prompts, as cases to time.

Next to the routed experts, a step of such a batch finds pages for the new rows of every sequence and maps
the rows to their places (reserve; pages of dropped tokens go back with release), attends over the paged
E4M3 cache with the pages that a group of sequences shares read once for all of them (share), and draws each
row's next token from its logits under temperature, top-k, top-p and min-p with a given uniform number
(sample), or writes the distribution that is left for the verification of drafts (probs).

Each case runs in a plain form (elementary torch operations, 32 bits, whole numbers in 64) or, with `own` set,
through the package's entry points.  A page of the cache holds, for each layer, the codes
[2][heads][page][dim] (keys, then values), then the scales [2][heads] in fp32, padded to 128 bytes.

Sampling is defined in whole numbers.  With x the row's logits in fp32 (NaN and -infinity take no part), m the
largest, c = log2(e) / temperature, and every operation rounded to fp32: y = (x - m) c, n = rint(y), f = y - n,
p = 2^n (1 + f (C1 + f (C2 + f (C3 + f (C4 + f C5))))), W = floor(2^38 p), 0 unless y > -39.  Tokens stand in
the order of falling x, then rising index.  top-k keeps the first k; of their sum S, top-p keeps a token if
what stands before it is below S floor(2^24 top_p) / 2^24 (the first always); min-p keeps W >= 2^38 min_p, of
min_p's first 24 bits.  The token is the lowest index at which the kept weights, summed in index order, pass
floor(S' floor(2^24 u) / 2^24).  temperature <= 0 takes the first token of the order.
"""
import math
import random

import torch

own = False

FP8 = torch.float8_e4m3fn
GRID = 38  # weights are whole multiples of 2^-38
BITS = 24  # top_p, min_p and uniforms are whole multiples of 2^-24
LOG2E = 1.4426950216293335  # fp32
POLY = (0.6931470036506653, 0.24022242426872253, 0.05550733581185341, 0.009671512991189957, 0.001326472731307149)


# ------------------------------------------------------------------------------- cases


def listed():
    return [
        # four answers to one short question: the call's latency
        _share("share_4x1_500", (4,), 1, (500,), 60, 8, 7, 128, 64),
        # drafted rows of 24 conversations about one document, small pages, odd lengths
        _share("share_24x5_33k", (24,), 5, (32777,), 600, 8, 7, 128, 32),
        # several prompts at once: a single sequence, groups of many sizes, one without a prefix; narrow heads
        _share("share_6g_64d", (1, 13, 40, 5, 2, 29), 2, (9001, 4100, 1777, 0, 20000, 12288), 700, 4, 8, 64, 16, idle=True),
        # the largest: 96 samples over a whole library, each with its own continuation
        _share("share_96x1_128k", (96,), 1, (131072,), 2048, 8, 7, 128, 128),
        # one conversation's next token
        _sample("sample_1x32001", "sample", 1, 32001, "fp32", "mixed"),
        # a large batch, every request with settings of its own
        _sample("sample_256x131072", "sample", 256, 131072, "fp32", "mixed"),
        # the targets' distributions of nine sequences with four drafts each
        _sample("probs_45x65536", "probs", 45, 65536, "bf16", "mixed"),
        # a large verification batch with nucleus sampling alone, odd vocabulary
        _sample("probs_96x131071_p", "probs", 96, 131071, "fp32", "p"),
        # a decode step: one row each, few of them at a page's end
        _pages("reserve_64x1", "reserve", 64, 1, 16384, 64, 40000),
        # prompts of a full scheduler, many sequences, a large pool
        _pages("reserve_512x300", "reserve", 512, 300, 4096, 16, 400000),
        # the rejected ones of eight drafts each
        _pages("release_64x8", "release", 64, 8, 16384, 64, 40000),
        # many sequences are cut back at once, some of which share pages
        _pages("release_512x300", "release", 512, 300, 4096, 16, 400000),
    ]


def _share(name, members, rows, prefix, own_len, heads, group, dim, page, idle=False, layers=1):
    """members[g] sequences share the first prefix[g] tokens; 1..own_len further tokens each, `rows` of them new."""
    return {"name": name, "op": "share", "members": ",".join(map(str, members)), "rows": rows,
            "prefix": ",".join(map(str, prefix)), "own_len": own_len, "heads": heads, "group": group, "dim": dim,
            "page": page, "idle": idle, "layers": layers}


def _sample(name, op, rows, vocab, dtype, cuts):
    return {"name": name, "op": op, "rows": rows, "vocab": vocab, "dtype": dtype, "cuts": cuts}


def _pages(name, op, seqs, rows, hi, page, pages):
    """Sequences of 0..hi tokens take (or give back) 0..rows tokens each."""
    return {"name": name, "op": op, "seqs": seqs, "rows": rows, "hi": hi, "page": page, "pages": pages}


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(("share", "share", "sample", "sample", "probs", "reserve", "release"))
    if op == "share":
        groups = rng.choice((1, 1, 2, rng.randint(1, 6)))
        prefix = [rng.choice((0, _log_int(rng, 17, 131072))) if g else _log_int(rng, 17, 131072) for g in range(groups)]
        rows, page = rng.choice((1, 1, 2, 5, rng.randint(1, 9))), rng.choice((16, 32, 64, 128))
        members = [max(1, min(_log_int(rng, 1, 96 // groups), 10_000_000 // (groups * rows * (p + 1)))) for p in prefix]
        c = _share("", members, rows, prefix, max(rows, _log_int(rng, 1, 2048)), rng.choice((1, 2, 4, 8)),
                   rng.choice((1, 2, 4, 7, 8)), rng.choice((64, 128, 128)), page, rng.random() < 0.4, rng.choice((1, 1, 2)))
    elif op in ("sample", "probs"):
        vocab = _log_int(rng, 1000, 160001)
        rows = _log_int(rng, 1, max(1, min(256 if op == "sample" else 96, 33_000_000 // vocab)))
        c = _sample("", op, rows, vocab, rng.choice(("fp32", "bf16")), rng.choice(("mixed", "mixed", "p", "k", "none")))
    else:
        seqs, page = _log_int(rng, 1, 512), rng.choice((16, 32, 64, 128))
        rows, hi = _log_int(rng, 1, 300), _log_int(rng, 1, 4096)
        need = seqs * (-(-(hi + rows) // page) + 1)
        c = _pages("", op, seqs, rows, hi, page, need + _log_int(rng, 100, 200000))
    del c["name"]
    return c


def _shape(case):
    """The lengths a case stands for: of each sequence, its new rows and the tokens before them; the groups."""
    r = random.Random("%r" % sorted((k, v) for k, v in case.items() if k != "name"))
    if case["op"] == "share":
        members = [int(x) for x in case["members"].split(",")]
        n, old, groups = [], [], [0]
        for m, p in zip(members, map(int, case["prefix"].split(","))):
            for i in range(m):
                idle = case["idle"] and i > 0 and r.random() < 0.15
                rows = 0 if idle else case["rows"] if i == 0 else r.randint(1, case["rows"])
                own_len = max(rows, r.randint(1, case["own_len"]))
                n.append(rows)
                old.append(p + own_len - rows)
            groups.append(len(n))
        return n, old, groups
    n = [r.choice((case["rows"], r.randint(0, case["rows"]))) for _ in range(case["seqs"])]
    n[0] = case["rows"]
    old = [r.randint(0, case["hi"]) for _ in range(case["seqs"])]
    return n, old, None


def _prefixes(case):
    """Of each group: the tokens in whole shared pages."""
    return [int(x) // case["page"] * case["page"] for x in case["prefix"].split(",")]


def work(case):
    if case["op"] in ("sample", "probs"):
        size, n = 4 if case["dtype"] == "fp32" else 2, case["rows"] * case["vocab"]
        return {"bytes": n * size * (2 if case["op"] == "probs" else 1) + case["rows"] * 24, "flops": 20 * n}
    n, old, groups = _shape(case)
    P = case["page"]
    if case["op"] == "reserve":
        need = sum(-(-(o + m) // P) - -(-o // P) for m, o in zip(n, old))
        return {"bytes": case["pages"] * 4 + need * 8 + case["seqs"] * 16 + sum(n) * 16, "flops": case["pages"]}
    if case["op"] == "release":
        drop = sum(-(-(o + m) // P) - -(-o // P) for m, o in zip(n, old))
        return {"bytes": drop * 16 + case["seqs"] * 8, "flops": drop}
    H, D, Hq = case["heads"], case["dim"], case["heads"] * case["group"]
    kv = pairs = 0
    for g, p in enumerate(_prefixes(case)):
        kv += p
        for b in range(groups[g], groups[g + 1]):
            if n[b]:
                kv += old[b] + n[b] - p
                pairs += n[b] * old[b] + n[b] * (n[b] + 1) // 2
    return {"bytes": kv * H * D * 2 + -(-kv // P) * H * 8 + sum(n) * Hq * D * 4, "flops": 4 * pairs * Hq * D}


# ------------------------------------------------------------------------------ inputs


def _ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def _offsets(n):
    at = [0]
    for m in n:
        at.append(at[-1] + m)
    return _ints(at)


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if case["op"] == "share":
        return _prepare_share(case, g)
    if case["op"] in ("sample", "probs"):
        return _prepare_sample(case, g)
    return _prepare_pages(case, g)


def _prepare_share(case, g):
    n, old, groups = _shape(case)
    P, H, D, L = case["page"], case["heads"], case["dim"], case["layers"]
    prefix = _prefixes(case)
    used = [-(-(o + m) // P) for o, m in zip(old, n)]
    shared = [prefix[k] // P for k in range(len(prefix)) for _ in range(groups[k], groups[k + 1])]
    pages = sum(p // P for p in prefix) + sum(u - w for u, w in zip(used, shared)) + 3
    codes = 2 * H * P * D
    record = -(-(codes + 8 * H) // 128) * 128
    pool = torch.zeros((pages, L * record), dtype=torch.uint8, device="cuda")
    view = pool.view(pages, L, record)[:, L - 1]
    step = max(1, (1 << 28) // codes)
    for at in range(0, pages, step):  # values of about N(0, 1) times a page's own power of two
        some = view[at:at + step]
        v = torch.randn((some.shape[0], codes), generator=g, device="cuda").mul_(56.0).clamp_(-448, 448)
        some[:, :codes] = v.to(FP8).view(torch.uint8)
    e = torch.randint(-7, -4, (pages, 2 * H), generator=g, device="cuda")
    view[:, codes:codes + 8 * H].view(torch.float32).copy_(torch.exp2(e.float()))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)  # pages lie anywhere in the pool
    at, table = 0, torch.full((len(n), max(used)), -1, dtype=torch.int32, device="cuda")
    for k in range(len(prefix)):
        w = prefix[k] // P
        table[groups[k]:groups[k + 1], :w] = order[at:at + w]
        at += w
        for b in range(groups[k], groups[k + 1]):
            table[b, w:used[b]] = order[at:at + used[b] - w]
            at += used[b] - w
    q = torch.randn((sum(n), H * case["group"], D), generator=g, device="cuda").mul_(1.5).to(torch.bfloat16)
    return {"case": case, "n": n, "old": old, "groups": groups, "shared": prefix, "cu": _offsets(n), "q": q, "pool": pool,
            "table": table, "record": record, "total": _ints([o + m for o, m in zip(old, n)]), "cu_groups": _ints(groups),
            "prefix": _ints([int(x) for x in case["prefix"].split(",")]), "max_rows": max(n),
            "max_group_rows": max(sum(n[a:b]) for a, b in zip(groups, groups[1:])), "scale": D ** -0.5}


def _prepare_sample(case, g):
    R, V, cuts = case["rows"], case["vocab"], case["cuts"]
    x = torch.randn((R, V), generator=g, device="cuda").mul_(2.5)
    # in half of the rows a few tokens stand out, as where the model is sure
    top = torch.randint(0, V, (R, 6), generator=g, device="cuda")
    lift = torch.rand((R, 6), generator=g, device="cuda") * 14 * (torch.rand((R, 1), generator=g, device="cuda") < 0.5)
    x.scatter_add_(1, top, lift)
    if cuts == "mixed":  # a tenth of each row's vocabulary is masked out
        x.masked_fill_(torch.rand((R, V), generator=g, device="cuda") < 0.1, -math.inf)

    def pick(values, dtype):
        at = torch.randint(0, len(values), (R,), generator=g, device="cuda")
        return torch.tensor(values, dtype=dtype, device="cuda")[at]

    mixed = cuts == "mixed"
    return {"case": case, "x": x.to(torch.float32 if case["dtype"] == "fp32" else torch.bfloat16),
            "t": pick((0.0, 0.6, 0.7, 0.8, 0.9, 1.0, 1.0, 1.2) if mixed else (0.7, 0.8, 1.0, 1.1), torch.float32),
            "k": pick((0, 1, 20, 50, 50, 64, 200, 1000) if mixed else (20, 50, 100), torch.int32) if cuts in ("mixed", "k") else None,
            "p": pick((1.0, 0.5, 0.8, 0.9, 0.95, 0.99) if mixed else (0.8, 0.9, 0.95), torch.float32) if cuts in ("mixed", "p") else None,
            "m": pick((0.0, 0.0, 0.0, 0.02, 0.1), torch.float32) if mixed else None,
            "u": torch.rand(R, generator=g, device="cuda")}


def _prepare_pages(case, g):
    n, old, _ = _shape(case)
    P, N, B = case["page"], case["pages"], case["seqs"]
    full = [-(-(o + m) // P) for o, m in zip(old, n)]
    have = full if case["op"] == "release" else [-(-o // P) for o in old]
    width = max(full) + 1
    order = torch.randperm(N, generator=g, device="cuda").to(torch.int32)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(N, dtype=torch.int32, device="cuda")
    first = _ints(have).cumsum(0) - _ints(have)
    col = torch.arange(width, device="cuda")
    mine = col < _ints(have)[:, None]
    table = torch.where(mine, order[(first[:, None] + col).clamp(max=N - 1).long()], table)
    if case["op"] == "release" and B > 1:  # odd sequences hold their left neighbour's first pages, too
        both = (torch.arange(B, device="cuda") % 2 == 1)[:, None] & (col < torch.minimum(_ints(have), _ints(have).roll(1))[:, None] // 2)
        table = torch.where(both, table.roll(1, 0), table)
    held = table[mine].long()
    refs.scatter_add_(0, held, torch.ones_like(held, dtype=torch.int32))
    return {"case": case, "n": _ints(n), "start": _ints(old), "total": _ints([o + m for o, m in zip(old, n)]),
            "table": table.contiguous(), "refs": refs, "rows": sum(n)}


# -------------------------------------------------------------------------------- runs


def run(s):
    if own:
        return _run_own(s)
    return {"share": _share_plain, "sample": _sample_plain, "probs": _sample_plain, "reserve": _reserve_plain,
            "release": _release_plain}[s["case"]["op"]](s)


def _run_own(s):
    import mxfp4_routed_expert_topk_gb300 as moe

    c = s["case"]
    op = c["op"]
    if "ws" not in s:  # what a program makes once: the cache's view and a workspace
        if op == "share":
            s["cache"] = moe.KvCache(s["pool"].shape[0], c["layers"], c["heads"], c["dim"], c["page"], buffer=s["pool"])
            size = moe.moe_kv_attention_shared_workspace_size(s["cache"], len(s["q"]), s["max_rows"], s["max_group_rows"],
                                                              c["heads"] * c["group"])
        elif op in ("reserve", "release"):
            size = moe.moe_kv_pages_workspace_size(c["seqs"], c["pages"])
        else:
            size = moe.moe_sample_workspace_size(c["rows"], c["vocab"])
        s["ws"] = moe.workspace(size)
    if op == "share":
        return moe.moe_kv_attention_shared(s["cache"], c["layers"] - 1, s["q"], s["cu"], s["total"], s["table"], s["cu_groups"],
                                           s["prefix"], max_rows=s["max_rows"], max_group_rows=s["max_group_rows"],
                                           scale=s["scale"], ws=s["ws"])
    if op == "sample":
        return moe.moe_sample(s["x"], s["t"], s["u"], top_k=s["k"], top_p=s["p"], min_p=s["m"], ws=s["ws"])
    if op == "probs":
        return moe.moe_sample_probs(s["x"], s["t"], top_k=s["k"], top_p=s["p"], min_p=s["m"], ws=s["ws"])
    table, refs = s["table"].clone(), s["refs"].clone()  # (the call changes them in place)
    if op == "release":
        moe.moe_kv_release(s["start"], s["total"], table, refs, c["page"], ws=s["ws"])
        return {"table": table, "refs": refs}
    cu, total, seq, pos, slot = moe.moe_kv_reserve(s["n"], s["start"], table, refs, c["page"], s["rows"], ws=s["ws"])
    return {"table": table, "refs": refs, "cu": cu, "total": total, "seq": seq, "pos": pos, "slot": slot}


def _cache_view(s):
    """(codes [pages][2][heads][page][dim] as bytes, scales [pages][2][heads]) of the case's layer."""
    c = s["case"]
    H, P, D = c["heads"], c["page"], c["dim"]
    rec = s["pool"].view(-1, c["layers"], s["record"])[:, c["layers"] - 1]
    n = 2 * H * P * D
    return rec[:, :n].unflatten(1, (2, H, P, D)), rec[:, n:n + 8 * H].view(torch.float32).unflatten(1, (2, H))


def _rows_of(codes, scales, side, pages):
    """Keys or values of the given pages: [..., heads, tokens, dim] in 32 bits."""
    x = codes[:, side][pages].view(FP8).float().mul_(scales[:, side][pages][..., None, None])
    return x.transpose(-4, -3).flatten(-3, -2)


def _share_plain(s):
    c = s["case"]
    H, P, D, G = c["heads"], c["page"], c["dim"], c["group"]
    codes, scales = _cache_view(s)
    out = torch.empty_like(s["q"])
    cu, total, at = s["cu"].long(), s["total"].long(), 0
    for k, prefix in enumerate(s["shared"]):
        b0, b1 = s["groups"][k], s["groups"][k + 1]
        R, N, w = sum(s["n"][b0:b1]), max(s["n"][b0:b1]), prefix // P
        q = s["q"][at:at + R].float().mul(s["scale"])  # [R][Hq][D]
        r = torch.arange(at, at + R, device="cuda")
        seq = torch.searchsorted(cu[b0 + 1:b1 + 1], r, right=True)
        i = r - cu[b0 + seq]
        # each sequence's own tokens, padded to the longest
        last = max(-(-(o + m) // P) for o, m in zip(s["old"][b0:b1], s["n"][b0:b1]))
        pages = s["table"][b0:b1, w:last].clamp(min=0).long()
        rows = torch.arange(N, device="cuda")
        n = cu[b0 + 1:b1 + 1] - cu[b0:b1]
        padded = torch.where(rows < n[:, None], cu[b0:b1, None] - at + rows, 0)
        qb = q[padded].view(b1 - b0, N, H, G, D).permute(0, 2, 1, 3, 4).reshape(b1 - b0, H, N * G, D)
        x = torch.matmul(qb, _rows_of(codes, scales, 0, pages).transpose(2, 3)).view(b1 - b0, H, N, G, -1)
        t = prefix + torch.arange(x.shape[-1], device="cuda")
        sees = t <= (total[b0:b1] - n)[:, None, None] + rows[:, None]  # [B][N][T]
        x = x.masked_fill_(~sees[:, None, :, None], -math.inf)
        m = x.amax(-1, keepdim=True)
        p = torch.exp(x.sub_(m))
        o = torch.matmul(p.view(b1 - b0, H, N * G, -1), _rows_of(codes, scales, 1, pages)).view(b1 - b0, H, N, G, D)
        pick = lambda y: y.permute(0, 2, 1, 3, 4)[seq, i]  # noqa: E731  [R][H][G][.]
        o, m, l = pick(o), pick(m), pick(p.sum(-1, keepdim=True))
        if w:  # the shared tokens, for all rows of the group at once
            first = s["table"][b0, :w].long()
            qg = q.view(R, H, G, D).transpose(0, 1).reshape(H, R * G, D)
            x = torch.matmul(qg, _rows_of(codes, scales, 0, first).transpose(1, 2))
            m2 = x.amax(-1, keepdim=True)
            p = torch.exp(x.sub_(m2))
            back = lambda y: y.view(H, R, G, -1).transpose(0, 1)  # noqa: E731
            o2, l2 = back(torch.matmul(p, _rows_of(codes, scales, 1, first))), back(p.sum(-1, keepdim=True))
            m2 = back(m2)
            both = torch.maximum(m, m2)
            f, f2 = torch.exp(m - both), torch.exp(m2 - both)
            o, l = o * f + o2 * f2, l * f + l2 * f2
        out[at:at + R] = (o / l).reshape(R, H * G, D).to(torch.bfloat16)
        at += R
    return out


def _bits(v, none):
    """The first 24 bits of numbers in 0..1 as whole numbers (`none` for NaN)."""
    return torch.where(v == v, (v.clamp(0, 1) * 2.0 ** BITS).to(torch.int64), none)


def _share_of(total, m, up):
    """total m / 2^24, rounded down or up, without leaving 64 bits."""
    low = (total & (2 ** BITS - 1)) * m + (2 ** BITS - 1 if up else 0)
    return (total >> BITS) * m + (low >> BITS)


def _kept_plain(s):
    """(kept weights [rows][vocab], first token of the order, rows that take it or have none)."""
    x, V = s["x"].float(), s["x"].shape[1]
    x = x.masked_fill(x != x, -math.inf)
    best, order = torch.sort(x, dim=-1, descending=True, stable=True)
    m = best[:, :1]
    c = (torch.full_like(s["t"], LOG2E) / s["t"]).clamp(max=torch.finfo(torch.float32).max)[:, None]
    y = torch.where(best == m, 0.0, (best - m) * c)
    n = torch.round(y)
    f = y - n
    e = torch.full_like(f, POLY[4])
    for k in (3, 2, 1, 0):
        e = e * f + POLY[k]
    e = e * f + 1.0
    two = ((n.clamp(min=-100).nan_to_num(0.0).to(torch.int32) + 127) << 23).view(torch.float32)
    live = (y > -39.0) & (best > -math.inf)
    w = torch.where(live, e * two, 0.0).mul_(2.0 ** GRID).to(torch.int64)
    if s["k"] is not None:
        k = torch.where(s["k"] > 0, s["k"], V)[:, None]
        w = torch.where(torch.arange(V, device="cuda") < k, w, 0)
    keep = w > 0
    if s["p"] is not None:
        upto = w.cumsum(-1)
        keep &= upto - w < _share_of(upto[:, -1:], _bits(s["p"], 1 << BITS).clamp(min=1)[:, None], True)
    if s["m"] is not None:
        keep &= w >= (_bits(s["m"], 0) << (GRID - BITS))[:, None]
    kept = torch.zeros_like(w).scatter_(1, order, torch.where(keep, w, 0))
    none = m[:, 0] == -math.inf
    first = torch.where(none, -1, order[:, 0])
    return kept, first, none | ~(s["t"] > 0)


def _sample_plain(s):
    kept, first, plain = _kept_plain(s)
    total = kept.sum(-1)
    if s["case"]["op"] == "probs":
        hot = torch.arange(kept.shape[1], device="cuda") == first[:, None]
        p = kept.float() / total.float()[:, None]
        return torch.where(plain[:, None], hot.float(), p).to(s["x"].dtype)
    aim = _share_of(total, _bits(s["u"], 0).clamp(max=2 ** BITS - 1), False)
    token = (kept.cumsum(-1) <= aim[:, None]).sum(-1)
    return torch.where(plain, first, token).to(torch.int32)


def _reserve_plain(s):
    P, N, B = s["case"]["page"], s["case"]["pages"], s["case"]["seqs"]
    table, refs = s["table"].clone(), s["refs"].clone()
    n, start = s["n"].long(), s["start"].long()
    total = start + n
    c0, c1 = (start + P - 1) // P, (total + P - 1) // P
    upto = (c1 - c0).cumsum(0)
    free = refs == 0
    rank = free.cumsum(0) - 1
    pages = torch.arange(N, device="cuda")
    lowest = torch.zeros(N + 1, dtype=torch.int64, device="cuda").scatter_(0, torch.where(free, rank, N), pages)
    col = torch.arange(table.shape[1], device="cuda")
    new = (col >= c0[:, None]) & (col < c1[:, None])
    table = torch.where(new, lowest[((upto - c1)[:, None] + col).clamp(0, N)].to(torch.int32), table)
    refs = torch.where(free & (rank < upto[-1]), 1, refs)
    cu = torch.zeros(B + 1, dtype=torch.int32, device="cuda")
    cu[1:] = n.cumsum(0)
    r = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(cu[1:].long(), r, right=True)
    pos = start[seq] + r - cu[seq]
    slot = table[seq, pos // P].long() * P + pos % P
    return {"table": table, "refs": refs, "cu": cu, "total": total.to(torch.int32), "seq": seq.to(torch.int32),
            "pos": pos.to(torch.int32), "slot": slot}


def _release_plain(s):
    P = s["case"]["page"]
    table, refs = s["table"].clone(), s["refs"].clone()
    c0, c1 = (s["start"].long() + P - 1) // P, (s["total"].long() + P - 1) // P
    col = torch.arange(table.shape[1], device="cuda")
    drop = (col >= c0[:, None]) & (col < c1[:, None])
    refs.scatter_add_(0, table.clamp(min=0).long().flatten(), -drop.to(torch.int32).flatten())
    return {"table": torch.where(drop, -1, table), "refs": refs}


# ------------------------------------------------------------------------------- exact


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "share":
        return _exact_share(s, case)
    if case["op"] in ("sample", "probs"):
        return _exact_sample(s, case)
    return _exact_pages(s, case)


def _exact_share(s, case):
    H, D, G, P, L = case["heads"], case["dim"], case["group"], case["page"], case["layers"]
    size = 2 * H * P * D
    rec = s["pool"].reshape(-1, L, s["record"])[:, L - 1]
    scales = rec[:, size:size + 8 * H].contiguous().view(torch.float32).double().reshape(-1, 2, H)

    def tokens(ids):
        ids = torch.tensor(ids, dtype=torch.long, device="cuda")
        x = rec[ids][:, :size].contiguous().view(FP8).double().reshape(-1, 2, H, P, D) * scales[ids][..., None, None]
        return x.permute(1, 2, 0, 3, 4).reshape(2, H, -1, D)

    outs, at, table = [], 0, s["table"].tolist()
    for k, prefix in enumerate(s["shared"]):
        both = tokens(table[s["groups"][k]][:prefix // P])
        for b in range(s["groups"][k], s["groups"][k + 1]):
            m, total = s["n"][b], s["old"][b] + s["n"][b]
            if not m:
                continue
            kv = torch.cat((both, tokens(table[b][prefix // P:-(-total // P)])), 2)[:, :, :total]
            q = s["q"][at:at + m].double().reshape(m, H, G, D)
            x = torch.matmul(q.permute(1, 2, 0, 3).reshape(H, G * m, D), kv[0].transpose(1, 2)).mul_(s["scale"])
            x = x.view(H, G, m, total)
            hidden = torch.ones((m, total), dtype=torch.bool, device="cuda").triu(s["old"][b] + 1)
            p = torch.softmax(x.masked_fill_(hidden, -math.inf), -1)
            o = torch.matmul(p.view(H, G * m, total), kv[1]).view(H, G, m, D)
            outs.append(o.permute(2, 0, 1, 3).reshape(m, H * G, D))
            at += m
    return torch.cat(outs)


def _exact_sample(s, case):
    """Row by row; products and sums of two fp32 numbers in 64 bits, rounded to fp32, are the rounded ones."""
    r32 = lambda v: v.float().double()  # noqa: E731
    cuts = {k: None if s[k] is None else s[k].double().tolist() for k in ("k", "p", "m", "t", "u")}
    outs = []
    for r in range(case["rows"]):
        x = s["x"][r].double()
        live = ((x == x) & (x > -math.inf)).nonzero()[:, 0]
        out = torch.zeros(case["vocab"], dtype=torch.float64, device="cuda")
        x, by = torch.sort(x[live], descending=True, stable=True)
        ids = live[by]
        T = cuts["t"][r]
        if len(ids) == 0 or not T > 0:
            token = int(ids[0]) if len(ids) else -1
            if token >= 0:
                out[token] = 1.0
        else:
            c = min(float(r32(torch.tensor(LOG2E / T, dtype=torch.float64))), torch.finfo(torch.float32).max)
            y = r32(r32(x - x[0]) * c)
            y[x == x[0]] = 0.0
            i = int((y > -39.0).sum())
            y, ids = y[:i], ids[:i]
            n = torch.round(y)
            f = y - n
            e = torch.zeros_like(f)
            for k in (4, 3, 2, 1, 0):
                e = r32(r32(e * f) + POLY[k])
            w = (r32(r32(e * f) + 1.0) * 2 ** 24).to(torch.int64)  # (a whole number)
            up = n.to(torch.int64) + GRID - 24
            w = (w << up.clamp(min=0)) >> (-up).clamp(min=0)
            if cuts["k"] is not None and cuts["k"][r] > 0:
                w = w[:int(cuts["k"][r])]
            if cuts["p"] is not None:
                part = max(1, math.floor(min(max(cuts["p"][r], 0.0), 1.0) * 2 ** BITS))
                before = torch.cat((torch.zeros(1, dtype=torch.int64, device="cuda"), w.cumsum(0)[:-1]))
                w = w[:int((before < -(-int(w.sum()) * part // 2 ** BITS)).sum())]
            ids = ids[:len(w)]
            if cuts["m"] is not None:
                ok = w >= math.floor(min(max(cuts["m"][r], 0.0), 1.0) * 2 ** BITS) << (GRID - BITS)
                w, ids = w[ok], ids[ok]
            total = int(w.sum())
            out[ids] = w.double() / total
            ids, by = torch.sort(ids)
            aim = total * min(math.floor(cuts["u"][r] * 2 ** BITS), 2 ** BITS - 1) >> BITS
            token = int(ids[torch.searchsorted(w[by].cumsum(0), torch.tensor(aim, device="cuda"), right=True)])
        outs.append(out if case["op"] == "probs" else token)
    return torch.stack(outs) if case["op"] == "probs" else torch.tensor(outs, dtype=torch.int32)


def _exact_pages(s, case):
    P = case["page"]
    n, start = s["n"].tolist(), s["start"].tolist()
    table, refs = s["table"].tolist(), s["refs"].tolist()
    if case["op"] == "release":
        for b, (m, o) in enumerate(zip(n, start)):
            for col in range(-(-o // P), -(-(o + m) // P)):
                refs[table[b][col]] -= 1
                table[b][col] = -1
        return {"table": torch.tensor(table, dtype=torch.int32), "refs": torch.tensor(refs, dtype=torch.int32)}
    cu, seq, pos, slot, at = [0], [], [], [], 0
    for b, (m, o) in enumerate(zip(n, start)):
        for col in range(-(-o // P), -(-(o + m) // P)):
            while refs[at]:
                at += 1
            refs[at], table[b][col] = 1, at
        for t in range(o, o + m):
            seq.append(b)
            pos.append(t)
            slot.append(table[b][t // P] * P + t % P)
        cu.append(cu[-1] + m)
    t32 = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"table": t32(table), "refs": t32(refs), "cu": t32(cu), "total": t32([o + m for m, o in zip(n, start)]),
            "seq": t32(seq), "pos": t32(pos), "slot": torch.tensor(slot, dtype=torch.int64)}
