"""The operators around a speculative-verify pass, as measured cases.

A verify pass of one attention layer runs the quantized wqkv product, adds
low-rank adapters, rotates queries and keys while appending keys and values to
a paged cache, attends from every drafted token over the cache and its own
ancestors, and, once the drafts are judged, moves the accepted rows next to
the context.  Each case is one of these four calls:

  lora       y = base + scale * B (A x), an adapter per request
  rope       per-head norms, rotation, append to the paged cache
  attention  drafted tokens (a tree, a chain or one token) over the cache
  accept     accepted rows moved behind the context, every layer at once

Where ``own`` is false, run() is plain torch in 32 bits (64 for the angles);
where it is true, it calls the library.
"""

import math
import random

import torch

own = False

DEVICE = "cuda"
LORA, ROPE, ATTENTION, ACCEPT = "lora", "rope", "attention", "accept"


def listed():
    return [
        # one request at batch 1 beside the 7B wqkv product: latency
        dict(name="lora 1 token wqkv", op=LORA, requests=1, per=1, bare=0, adapters=8, rank=16, ragged=False, k=4096,
             n=12288, out="bf16"),
        # 32 requests verify 5 drafts each beside the 70B wqkv product, four of them without an adapter
        dict(name="lora 32x5 verify wqkv", op=LORA, requests=32, per=5, bare=4, adapters=64, rank=32, ragged=True,
             k=8192, n=10240, out="f32"),
        # prompts of a few tenants beside the 7B w1|w3 product, rows of the first requests bare
        dict(name="lora 8x128 prompt w13", op=LORA, requests=8, per=128, bare=1, adapters=4, rank=64, ragged=False,
             k=4096, n=22016, out="bf16"),
        # batch-1 decode, every head its own key head: latency
        dict(name="rope 1 token", op=ROPE, requests=1, per=1, heads=32, kv=32, dim=128, rot=128, interleaved=True,
             norm=False, source="bf16", page=16, far=2048),
        # verify of 32 requests at far positions, grouped heads, fp32 products, norms of queries and keys
        dict(name="rope 32x5 verify norms", op=ROPE, requests=32, per=5, heads=64, kv=8, dim=128, rot=128,
             interleaved=False, norm=True, source="f32", page=64, far=131072),
        # a prompt's rows, half of each head rotated
        dict(name="rope 3x1365 prompt", op=ROPE, requests=3, per=1365, heads=32, kv=8, dim=128, rot=64,
             interleaved=False, norm=True, source="bf16", page=128, far=8192),
        # batch-1 decode shortly after the prompt: latency
        dict(name="attention 1 token 500", op=ATTENTION, requests=1, per=1, heads=32, kv=32, dim=128, page=16,
             longest=500, ragged=False, tree=False),
        # one long conversation verifies a chain of 5
        dict(name="attention 1x5 chain 32k", op=ATTENTION, requests=1, per=5, heads=64, kv=8, dim=128, page=64,
             longest=32763, ragged=False, tree=False),
        # a serving batch, trees of 8, lengths of all kinds
        dict(name="attention 32x8 tree ragged", op=ATTENTION, requests=32, per=8, heads=32, kv=8, dim=128, page=64,
             longest=16384, ragged=True, tree=True),
        # wide trees: 64 drafts for each of two requests
        dict(name="attention 2x64 tree 16k", op=ATTENTION, requests=2, per=64, heads=64, kv=8, dim=128, page=128,
             longest=16000, ragged=False, tree=True),
        # one request of a shallow model after its tree of 5
        dict(name="accept 1x5 one layer", op=ACCEPT, layers=1, requests=1, width=4, levels=1, kv=8, dim=128, page=16,
             longest=500),
        # a serving batch after trees of 57, all 32 layers
        dict(name="accept 32x57 all layers", op=ACCEPT, layers=32, requests=32, width=8, levels=7, kv=8, dim=128,
             page=16, longest=100),
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high + 0.49)))))))


def draw(rng):
    largest = max(work(c)["bytes"] for c in listed())
    most = max(work(c)["flops"] for c in listed())
    while True:
        c = _draw(rng)
        w = work(c)
        if w["bytes"] <= 0.8 * largest and w["flops"] <= 0.8 * most:
            return c


def _draw(rng):
    op = rng.choice([LORA, LORA, ROPE, ROPE, ATTENTION, ATTENTION, ATTENTION, ACCEPT])
    if op == LORA:
        requests, per = _log(rng, 1, 128), rng.choice([1, 1, 2, 3, 5, 8, _log(rng, 1, 256)])
        return dict(op=op, requests=requests, per=min(per, 4096 // requests), bare=rng.choice([0, 0, requests // 4]),
                    adapters=_log(rng, 1, 128), rank=rng.choice([8, 16, 24, 32, 64, 128]), ragged=rng.random() < 0.5,
                    k=8 * _log(rng, 32, 1792), n=_log(rng, 64, 28672), out=rng.choice(["bf16", "f32"]))
    kv = rng.choice([1, 2, 4, 8, 8, 32])
    heads = kv if kv == 32 else kv * rng.choice([1, 2, 4, 5, 8])
    dim = rng.choice([64, 128, 128, 128, 256])
    page = rng.choice([16, 64, 128, rng.randint(5, 200)])
    if op == ROPE:
        return dict(op=op, requests=_log(rng, 1, 64), per=rng.choice([1, 2, 5, 8, _log(rng, 1, 256)]), heads=heads,
                    kv=kv, dim=dim, rot=rng.choice([dim, dim, dim // 2, dim // 4]), interleaved=rng.random() < 0.5,
                    norm=rng.random() < 0.5, source=rng.choice(["bf16", "f32"]), page=page, far=_log(rng, 1, 262144))
    if op == ATTENTION:
        return dict(op=op, requests=_log(rng, 1, 64), per=rng.choice([1, 1, 2, 5, 8, 16, rng.randint(1, 64)]),
                    heads=heads, kv=kv, dim=dim, page=page, longest=_log(rng, 1, 40000), ragged=rng.random() < 0.6,
                    tree=rng.random() < 0.6)
    width = rng.randint(2, 8)
    return dict(op=op, layers=_log(rng, 1, 32), requests=_log(rng, 1, 32), width=width,
                levels=rng.randint(1, 63 // width), kv=kv, dim=dim, page=page, longest=_log(rng, 1, 300))


# --- what a case fixes whatever the seed -----------------------------------


def _lengths(case):
    """Context length of each request: all the longest, or spread from nothing on."""
    r = random.Random(case["requests"] * 1000003 + case["longest"])
    if not case.get("ragged", True):
        return [case["longest"]] * case["requests"]
    return [case["longest"]] + [_log(r, 1, case["longest"] + 1) - 1 for _ in range(case["requests"] - 1)]


def _counts(case):
    """Drafted tokens of each request."""
    r = random.Random(case["requests"] * 7919 + case["per"])
    if not case.get("ragged", False):
        return [case["per"]] * case["requests"]
    return [case["per"]] + [r.randint(1, case["per"]) for _ in range(case["requests"] - 1)]


def _ranks(case):
    """Rank of each resident adapter: all the same, or some of them smaller."""
    return [case["rank"] if not case["ragged"] or a % 3 else max(8, case["rank"] // 2) for a in range(case["adapters"])]


def _adapter_of(case):
    """Adapter of each request; -1 for the first `bare` ones."""
    return [-1 if r < case["bare"] else (5 * r + 3) % case["adapters"] for r in range(case["requests"])]


def _paths(case):
    """Accepted drafts of each request: one node of each level of its tree, as many levels as were accepted."""
    r, w = random.Random(case["requests"] * 31 + case["width"]), case["width"]
    paths = []
    for _ in range(case["requests"]):
        n = r.randint(1, min(w, case["levels"] + 1)) if case["requests"] > 1 else min(w, case["levels"] + 1)
        # a node that the move itself does not overwrite, so that the call can be made again
        paths.append([0] + [r.choice([1 + (i - 1) * w + a for a in range(w)
                                      if 1 + (i - 1) * w + a >= n or 1 + (i - 1) * w + a == i])
                            for i in range(1, n)])
    return paths


def work(case):
    op = case["op"]
    if op == LORA:
        t, of, ranks = case["requests"] * case["per"], _adapter_of(case), _ranks(case)
        weights = sum(ranks[a] * (case["k"] + case["n"]) for a in set(of) if a >= 0)
        flops = sum(2 * case["per"] * ranks[a] * (case["k"] + case["n"]) for a in of if a >= 0)
        return {"bytes": 2 * weights + 2 * t * case["k"] + t * case["n"] * (4 + (2 if case["out"] == "bf16" else 4)),
                "flops": flops}
    if op == ROPE:
        t, q, k = case["requests"] * case["per"], case["heads"] * case["dim"], case["kv"] * case["dim"]
        return {"bytes": t * ((q + 2 * k) * (4 if case["source"] == "f32" else 2) + 2 * q + 4 * k),
                "flops": t * (q + k) * (8 if case["norm"] else 4)}
    if op == ATTENTION:
        rows = keys = pairs = 0
        for length, n in zip(_lengths(case), _counts(case)):
            rows, keys, pairs = rows + n, keys + length + n, pairs + n * (length + (n + 1) / 2)
        return {"bytes": 4 * keys * case["kv"] * case["dim"] + 4 * rows * case["heads"] * case["dim"],
                "flops": 4 * pairs * case["heads"] * case["dim"]}
    moved = sum(p != i for path in _paths(case) for i, p in enumerate(path))
    return {"bytes": max(64, 8 * moved * case["layers"] * case["kv"] * case["dim"]), "flops": 0}


# --- inputs ----------------------------------------------------------------


def _ints(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device=DEVICE)


def _starts(counts):
    starts = [0]
    for n in counts:
        starts.append(starts[-1] + n)
    return starts


def _table(generator, spans, page):
    """Page table of requests that use positions [from, to) each, pages in no order, and the number of pages.
    Pages before `from` are not touched by the call and stand for none in the pool; some pages are nobody's."""
    need = [(a // page, -(-b // page)) for a, b in spans]
    pages = sum(-(-(b - a) // page) + 1 for a, b in spans) + 3
    order = torch.randperm(pages, generator=generator, device=DEVICE).to(torch.int32)
    table = torch.zeros(len(need), max(1, max(b for _, b in need)), dtype=torch.int32, device=DEVICE)
    at = 0
    for r, (a, b) in enumerate(need):
        table[r, a:b] = order[at:at + b - a]
        at += b - a
    return table, pages


def _trees(r, counts, tree):
    """Visible drafts of each drafted token as bits, and its depth: a random tree, or a chain."""
    bits, depth = [], []
    for n in counts:
        mask, deep = [], []
        for j in range(n):
            parent = (r.randint(max(0, j - 12), j - 1) if tree else j - 1) if j else -1
            mask.append((mask[parent] if j else 0) | 1 << j)
            deep.append(deep[parent] + 1 if j else 0)
        bits += [m - (1 << 64) if m >> 63 else m for m in mask]
        depth += deep
    return bits, depth


def prepare(case, seed):
    op, r = case["op"], random.Random(seed)
    g = torch.Generator(device=DEVICE)
    g.manual_seed(seed)

    def normal(*shape, sigma=1.0, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device=DEVICE).normal_(0.0, sigma, generator=g)

    s = {"case": case}
    if op == LORA:
        tokens, order = case["requests"] * case["per"], list(range(case["adapters"]))
        r.shuffle(order)  # which resident adapter a request uses
        ranks = [0] * case["adapters"]
        for a, rank in enumerate(_ranks(case)):
            ranks[order[a]] = rank
        s["x"] = normal(tokens, case["k"])
        s["base"] = normal(tokens, case["n"], dtype=torch.float32)
        s["a"] = normal(case["adapters"], case["rank"], case["k"], sigma=case["k"] ** -0.5)
        s["b"] = normal(case["adapters"], case["n"], case["rank"], sigma=case["rank"] ** -0.5)
        s["adapter"] = _ints([-1 if a < 0 else order[a] for a in _adapter_of(case) for _ in range(case["per"])])
        s["ranks"] = _ints(ranks)
        s["scale"] = torch.rand(case["adapters"], generator=g, device=DEVICE) + 0.5
        s["y"] = torch.empty(tokens, case["n"], device=DEVICE,
                             dtype=torch.bfloat16 if case["out"] == "bf16" else torch.float32)
        if own:
            import weight_only_quantized_wq_amd as wq
            s["plan"] = wq.wq_lora_prepare(s["x"], s["a"], s["b"], s["adapter"], s["y"], base=s["base"],
                                           ranks=s["ranks"], scale=s["scale"])
    elif op == ROPE:
        heads, kv, dim, per = case["heads"], case["kv"], case["dim"], case["per"]
        counts = [per] * case["requests"]
        lengths = [r.randint(0, case["far"]) for _ in counts]
        table, pages = _table(g, [(n, n + per) for n in lengths], case["page"])
        _, depth = _trees(r, counts, per <= 64)
        source = torch.float32 if case["source"] == "f32" else torch.bfloat16
        s["qkv"] = normal(sum(counts), (heads + 2 * kv) * dim, dtype=source)
        s["k"], s["v"] = normal(pages, case["page"], kv, dim), normal(pages, case["page"], kv, dim)
        s["table"], s["starts"], s["lengths"] = table, _ints(_starts(counts)), _ints(lengths)
        s["positions"] = _ints([lengths[t // per] + d for t, d in enumerate(depth)])
        s["request"] = _ints([t // per for t in range(len(depth))], torch.int64)
        half = torch.arange(0, case["rot"], 2, dtype=torch.float64, device=DEVICE)
        s["freq"] = (500000.0 ** (-half / case["rot"])).to(torch.float32)
        s["q_norm"] = normal(dim, sigma=0.1) + 1 if case["norm"] else None
        s["k_norm"] = normal(dim, sigma=0.1) + 1 if case["norm"] else None
        s["q"] = torch.empty(sum(counts), heads, dim, dtype=torch.bfloat16, device=DEVICE)
        if own:
            import weight_only_quantized_wq_amd as wq
            s["plan"] = wq.wq_qkv_rope_prepare(
                s["qkv"], s["q"], s["k"], s["v"], s["table"], s["starts"], s["lengths"], s["freq"],
                positions=s["positions"], q_norm=s["q_norm"], k_norm=s["k_norm"], eps=1e-6,
                interleaved=case["interleaved"])
    elif op == ATTENTION:
        counts, lengths = _counts(case), _lengths(case)
        table, pages = _table(g, [(0, n + d) for n, d in zip(lengths, counts)], case["page"])
        bits, _ = _trees(r, counts, case["tree"])
        s["q"] = normal(sum(counts), case["heads"], case["dim"])
        s["k"] = normal(pages, case["page"], case["kv"], case["dim"])
        s["v"] = normal(pages, case["page"], case["kv"], case["dim"])
        s["table"], s["starts"], s["lengths"] = table, _ints(_starts(counts)), _ints(lengths)
        s["tree"] = _ints(bits, torch.int64) if case["tree"] else None
        s["y"] = torch.empty_like(s["q"])
        if own:
            import weight_only_quantized_wq_amd as wq
            s["plan"] = wq.wq_tree_attention_prepare(
                s["q"], s["k"], s["v"], s["table"], s["starts"], s["lengths"], s["y"], tree=s["tree"],
                max_tokens=case["per"], scale=case["dim"] ** -0.5)
    else:
        drafts = 1 + case["width"] * case["levels"]
        lengths, paths = _lengths(case), _paths(case)
        table, pages = _table(g, [(0, n + drafts) for n in lengths], case["page"])
        s["k"] = normal(case["layers"], pages, case["page"], case["kv"], case["dim"])
        s["v"] = normal(case["layers"], pages, case["page"], case["kv"], case["dim"])
        longest = max(len(p) for p in paths)
        s["path"] = _ints([p + [0] * (longest - len(p)) for p in paths])
        s["accepted"], s["table"], s["lengths"] = _ints([len(p) for p in paths]), table, _ints(lengths)
        if own:
            import weight_only_quantized_wq_amd as wq
            s["plan"] = wq.wq_kv_accept_prepare(s["k"], s["v"], s["table"], s["lengths"], s["path"], s["accepted"])
    return s


# --- one pass --------------------------------------------------------------


def run(s):
    op = s["case"]["op"]
    if own:
        import weight_only_quantized_wq_amd as wq
        if op == LORA:
            wq.wq_lora_run(s["plan"])
            return s["y"]
        if op == ROPE:
            wq.wq_qkv_rope_run(s["plan"])
            return {"q": s["q"], "k": s["k"], "v": s["v"]}
        if op == ATTENTION:
            wq.wq_tree_attention_run(s["plan"])
            return s["y"]
        wq.wq_kv_accept_run(s["plan"])
        return {"k": s["k"].view(torch.int16), "v": s["v"].view(torch.int16)}
    if op == LORA:
        return _lora(s)
    if op == ROPE:
        return _rope(s)
    if op == ATTENTION:
        return _attention(s)
    return _accept(s)


def _lora(s):
    adapters, rank, k = s["a"].shape
    slot = torch.arange(adapters, device=DEVICE)
    # products with every resident adapter, those of others (and ranks it has not) masked out
    keep = (s["adapter"][:, None] == slot) * s["scale"]
    keep = keep[:, :, None] * (torch.arange(rank, device=DEVICE) < s["ranks"][:, None])
    h = (s["x"].float() @ s["a"].float().reshape(adapters * rank, k).T) * keep.reshape(-1, adapters * rank)
    y = s["base"] + h @ s["b"].float().permute(0, 2, 1).reshape(adapters * rank, -1)
    return y.to(s["y"].dtype)


def _rope(s):
    c = s["case"]
    heads, kv, dim, rot = c["heads"], c["kv"], c["dim"], c["rot"]
    x = s["qkv"].float().view(-1, heads + 2 * kv, dim)
    qk, v = x[:, :heads + kv], x[:, heads + kv:]
    if c["norm"]:
        weight = torch.cat([s["q_norm"].float().expand(heads, dim), s["k_norm"].float().expand(kv, dim)])
        qk = qk / torch.sqrt((qk * qk).mean(-1, keepdim=True) + 1e-6) * weight
    angle = s["positions"].double()[:, None] * s["freq"].double()
    cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]
    turned, rest = qk[..., :rot], qk[..., rot:]
    if c["interleaved"]:
        a, b = turned[..., 0::2], turned[..., 1::2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = turned[..., :rot // 2], turned[..., rot // 2:]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    qk = torch.cat([turned, rest], -1).to(torch.bfloat16)
    t = torch.arange(qk.shape[0], device=DEVICE)
    at = s["lengths"].long()[s["request"]] + t - s["starts"].long()[s["request"]]
    row = s["table"].long()[s["request"], at // c["page"]] * c["page"] + at % c["page"]
    s["k"].view(-1, kv, dim)[row] = qk[:, heads:]
    s["v"].view(-1, kv, dim)[row] = v.to(torch.bfloat16)
    return {"q": qk[:, :heads], "k": s["k"], "v": s["v"]}


def _attention(s):
    c = s["case"]
    heads, kv, dim, page, most = c["heads"], c["kv"], c["dim"], c["page"], c["per"]
    starts, lengths = s["starts"].long(), s["lengths"].long()
    requests, tokens = lengths.shape[0], s["q"].shape[0]
    j = torch.arange(most, device=DEVICE)
    there = j < (starts[1:] - starts[:-1])[:, None]                      # [requests, most]
    row = torch.where(there, starts[:-1, None] + j, tokens)
    at = torch.arange(min(c["longest"] + most, s["table"].shape[1] * page), device=DEVICE)
    slot = s["table"].long()[:, at // page] * page + at % page           # [requests, positions]
    k = s["k"].view(-1, kv, dim)[slot].float().permute(0, 2, 1, 3)
    v = s["v"].view(-1, kv, dim)[slot].float().permute(0, 2, 1, 3)
    q = s["q"].float()[row.clamp(max=tokens - 1)] * dim ** -0.5          # [requests, most, heads, dim]
    q = q.view(requests, most, kv, heads // kv, dim).permute(0, 2, 1, 3, 4).reshape(requests, kv, -1, dim)
    bits = (2 << j) - 1 if s["tree"] is None else s["tree"][row.clamp(max=tokens - 1)]
    draft = at - lengths[:, None]                                        # [requests, positions]
    seen = (bits.expand(requests, most)[:, :, None] >> draft.clamp(0, 63)[:, None]) & 1 > 0
    seen = (draft < 0)[:, None] | (seen & (draft < (starts[1:] - starts[:-1])[:, None])[:, None])
    score = (q @ k.transpose(-1, -2)).view(requests, kv, most, heads // kv, -1)
    score = score.masked_fill(~seen[:, None, :, None], -math.inf)
    p = torch.exp(score - score.amax(-1, keepdim=True).clamp(min=-3e38))
    p = (p / p.sum(-1, keepdim=True).clamp(min=1e-37)).reshape(requests, kv, -1, at.shape[0])
    y = (p @ v).view(requests, kv, most, heads // kv, dim).permute(0, 2, 1, 3, 4).reshape(-1, heads, dim)
    out = torch.empty(tokens + 1, heads, dim, dtype=torch.bfloat16, device=DEVICE)
    out[row.reshape(-1)] = y.to(torch.bfloat16)
    return out[:tokens]


def _accept(s):
    c = s["case"]
    i = torch.arange(s["path"].shape[1], device=DEVICE)
    keep = i < s["accepted"][:, None]
    source = s["lengths"].long()[:, None] + torch.where(keep, s["path"].long(), i)
    target = s["lengths"].long()[:, None] + i
    # rows past the accepted ones stand for themselves
    target = torch.where(keep, target, source)
    most = s["table"].shape[1] * c["page"] - 1
    source, target = source.clamp(max=most), target.clamp(max=most)
    table = s["table"].long()
    source = table.gather(1, source // c["page"]) * c["page"] + source % c["page"]
    target = table.gather(1, target // c["page"]) * c["page"] + target % c["page"]
    k, v = (s[x].view(c["layers"], -1, c["kv"], c["dim"]) for x in ("k", "v"))
    k[:, target[keep]] = k[:, source[keep]]
    v[:, target[keep]] = v[:, source[keep]]
    return {"k": s["k"].view(torch.int16), "v": s["v"].view(torch.int16)}


# --- in 64 bits, from the definitions --------------------------------------


def exact(case, seed):
    if case["op"] == ACCEPT:
        return None
    s = prepare(case, seed)
    if case["op"] == LORA:
        y = s["base"].double()
        of = s["adapter"].tolist()
        for a in sorted(set(of) - {-1}):
            rows = torch.tensor([t for t, x in enumerate(of) if x == a], device=DEVICE)
            rank = int(s["ranks"][a])
            low = torch.mm(s["x"][rows].double(), s["a"][a, :rank].double().t())
            y[rows] += float(s["scale"][a]) * torch.mm(low, s["b"][a, :, :rank].double().t())
        return y
    if case["op"] == ROPE:
        heads, kv, dim, rot, page = (case[x] for x in ("heads", "kv", "dim", "rot", "page"))
        x = s["qkv"].double().reshape(-1, heads + 2 * kv, dim)
        if case["norm"]:
            for part, weight in ((slice(0, heads), s["q_norm"]), (slice(heads, heads + kv), s["k_norm"])):
                x[:, part] *= torch.rsqrt(x[:, part].square().mean(-1) + 1e-6)[..., None] * weight.double()
        turn = torch.polar(torch.ones((), dtype=torch.float64, device=DEVICE),
                           torch.outer(s["positions"].double(), s["freq"].double()))[:, None]
        i = torch.arange(rot // 2, device=DEVICE)
        first, second = (2 * i, 2 * i + 1) if case["interleaved"] else (i, i + rot // 2)
        z = torch.complex(x[:, :heads + kv, first], x[:, :heads + kv, second]) * turn
        x[:, :heads + kv, first], x[:, :heads + kv, second] = z.real, z.imag
        k, v = s["k"].double(), s["v"].double()
        starts, table = s["starts"].tolist(), s["table"].tolist()
        for r, length in enumerate(s["lengths"].tolist()):
            where = [(table[r][p // page], p % page) for p in range(length, length + starts[r + 1] - starts[r])]
            pages, rows = (torch.tensor(w, device=DEVICE) for w in zip(*where))
            k[pages, rows] = x[starts[r]:starts[r + 1], heads:heads + kv]
            v[pages, rows] = x[starts[r]:starts[r + 1], heads + kv:]
        return {"q": x[:, :heads], "k": k, "v": v}
    heads, kv, dim, page = (case[x] for x in ("heads", "kv", "dim", "page"))
    starts, y = s["starts"].tolist(), torch.zeros(s["q"].shape, dtype=torch.float64, device=DEVICE)
    for r, length in enumerate(s["lengths"].tolist()):
        a, b = starts[r], starts[r + 1]
        pages = s["table"][r, :-(-(length + b - a) // page)].long()
        k, v = (s[x][pages].flatten(0, 1)[:length + b - a].double() for x in ("k", "v"))
        hidden = torch.zeros(b - a, length + b - a, dtype=torch.bool, device=DEVICE)
        for t in range(b - a):
            bits = int(s["tree"][a + t]) if case["tree"] else (2 << t) - 1
            hidden[t, length:] = torch.tensor([not bits >> d & 1 for d in range(b - a)], device=DEVICE)
        for h in range(heads):
            score = torch.mm(s["q"][a:b, h].double(), k[:, h * kv // heads].t()) / math.sqrt(dim)
            score[hidden] = -math.inf
            y[a:b, h] = torch.mm(torch.softmax(score, -1), v[:, h * kv // heads])
    return y
