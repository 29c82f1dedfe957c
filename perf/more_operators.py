"""A step of speculative decoding over the mixed cache, in plain form and as the library's calls.

Three operators, in the order a step that checks a tree of drafted tokens uses them:

  tree     attention of every drafted token of every request over [BF16 sink | 4-bit history | BF16 recent] and over those
           drafted tokens that its mask lets it see, whose keys and values lie behind the cache's last position
  sample   a token per row of logits by temperature, top-k, top-p and min-p, from given uniform numbers
  accept   the path of drafted tokens that the sampled ones confirm, and its rows moved to the end of every layer's cache

A cache is [sink | history | recent]: positions [0, 64) and the last 256 are BF16, what lies between is 4-bit.
"""
import math

import numpy as np
import torch

own = False

DIM, SINK, RECENT = 128, 64, 256
DEV = "cuda"
DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# --------------------------------------------------------------------------- cases
def listed():
    shape_8b = dict(n_kv=8, gqa=4, page=64, group=128)       # 32 query heads, 8 kv heads
    shape_32b = dict(n_kv=8, gqa=8, page=64, group=32)       # 64 query heads, 8 kv heads, small groups
    small = dict(n_kv=2, gqa=4, page=16, group=128)          # 8 query heads, 2 kv heads, 16-token pages
    return [
        # a short conversation on a small model, a small tree: latency only
        dict(name="tree_1k_b1_n8", op="tree", batch=1, context=1024, ragged=False, nodes=8, chain=False, **small),
        # one long conversation: a small tree, and the largest that is drafted
        dict(name="tree_100k_b1_n8", op="tree", batch=1, context=100000, ragged=False, nodes=8, chain=False, **shape_8b),
        dict(name="tree_100k_b1_n64", op="tree", batch=1, context=100000, ragged=False, nodes=64, chain=False, **shape_8b),
        # a serving batch of unequal lengths, each request with a tree of its own size
        dict(name="tree_ragged_b16_n16", op="tree", batch=16, context=100000, ragged=True, nodes=16, chain=False, **shape_8b),
        # 64 query heads, groups of 32 channels
        dict(name="tree_32k_b4_n8_g32", op="tree", batch=4, context=32768, ragged=False, nodes=8, chain=False, **shape_32b),
        # nothing was drafted: the newest token of each request alone
        dict(name="tree_4k_b64_n1", op="tree", batch=64, context=4096, ragged=False, nodes=1, chain=True, **shape_8b),
        # the next token of one conversation, every filter on
        dict(name="sample_b1_filters", op="sample", rows=1, vocab=151936, dtype="bf16", filters="all"),
        # every node of eight trees of 32
        dict(name="sample_r256_filters", op="sample", rows=256, vocab=151936, dtype="bf16", filters="all"),
        # a batch that samples from the whole distribution, logits in 32 bits
        dict(name="sample_r64_plain", op="sample", rows=64, vocab=151936, dtype="fp32", filters="none"),
        # an older vocabulary, top-p alone
        dict(name="sample_r48_top_p", op="sample", rows=48, vocab=32000, dtype="fp16", filters="top_p"),
        # one conversation's tree, all 36 layers; a batch of larger trees on a small model
        dict(name="accept_b1_n16_l36", op="accept", batch=1, context=100000, nodes=16, layers=36, **shape_8b),
        dict(name="accept_b64_n64_l28", op="accept", batch=64, context=4096, nodes=64, layers=28, **shape_8b),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["tree", "tree", "sample", "accept"])
    if op == "sample":
        vocab = log(500, 200000)
        return dict(op=op, rows=min(log(1, 256), max(1, 256 * 151936 // vocab)), vocab=vocab, dtype=rng.choice(list(DTYPES)),
                    filters=rng.choice(["all", "none", "top_k", "top_p", "min_p"]))
    n_kv, gqa = rng.choice([(1, 8), (2, 4), (4, 2), (8, 1), (8, 4), (8, 8), (5, 4)])
    c = dict(op=op, n_kv=n_kv, gqa=gqa, page=rng.choice([16, 32, 64]), group=rng.choice([32, 64, 128, 128]), context=log(1, 100000), nodes=log(1, 100))
    if op == "accept":
        c |= dict(layers=log(1, 36), batch=log(1, 64))
        c["batch"] = min(c["batch"], max(1, 64 * 64 * 28 * 8 // (c["nodes"] * c["layers"] * n_kv)))
        return c
    # as many requests as the largest listed cases' reading and arithmetic allow
    most = min(1300000 // c["context"], 6400000 * 32 // (c["context"] * c["nodes"] * n_kv * gqa))
    return c | dict(batch=min(log(1, 64), max(1, most)), ragged=rng.random() < 0.7, chain=rng.random() < 0.25)


# --------------------------------------------------------------------------- inputs
def _generator(*parts):
    return torch.Generator(device=DEV).manual_seed(int(np.random.SeedSequence([abs(int(p)) for p in parts]).generate_state(1, np.uint64)[0] >> 1))


def _put(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


def _lengths(case, rng):
    T, B = case["context"], case["batch"]
    if not case.get("ragged"):
        return np.full(B, T, np.int64)
    return rng.integers(max(1, T * 2 // 3), T + 1, size=B)


def _pages(case):
    """Pages of the longest context a case can have and its tree: the width of its page tables, whatever lengths a seed draws."""
    return (max(case["context"], SINK + RECENT + 1) + case["nodes"] + case["page"] - 1) // case["page"]


def _table(spans, case, most, rng):
    """Page table that gives every page touching one of a request's spans a physical page, in random order, of a pool
    of `most` pages (or as many as there are)."""
    ps = case["page"]
    t = np.full((len(spans), _pages(case)), -1, np.int32)
    for b, ranges in enumerate(spans):
        for lo, hi in ranges:
            if hi > lo:
                t[b, lo // ps:(hi + ps - 1) // ps] = 0
    n = int((t == 0).sum())
    pool = max(n, 1) if most is None else most
    t[t == 0] = rng.permutation(pool)[:n]
    return t, pool


def _fill_int4(n_pages, case, gen):
    """Pages of 4-bit rows made from normal rows whose channels differ in size, one page set of keys and one of values."""
    H, ps, g = case["n_kv"], case["page"], case["group"]
    sigma = torch.rand((2, H, 1, DIM), generator=gen, device=DEV) * 1.5 + 0.5
    codes = [torch.empty((n_pages, H, ps, DIM // 2), dtype=torch.uint8, device=DEV) for _ in range(2)]
    sz = torch.empty((n_pages, H, ps, DIM // g, 4), dtype=torch.bfloat16, device=DEV)
    step = max(1, (1 << 26) // (H * ps * DIM))
    for i in range(0, n_pages, step):
        n = min(step, n_pages - i)
        for kind in (0, 1):
            x = torch.randn((n, H, ps, DIM // g, g), generator=gen, device=DEV) * sigma[kind].view(H, 1, DIM // g, g)
            lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
            zero, scale = lo.to(torch.bfloat16), ((hi - lo) / 15).to(torch.bfloat16)
            q = ((x - zero.float()) / scale.float()).round_().clamp_(0, 15).to(torch.uint8).view(n, H, ps, DIM // 2, 2)
            codes[kind][i:i + n] = q[..., 0] | (q[..., 1] << 4)
            sz[i:i + n, ..., 2 * kind] = scale[..., 0]
            sz[i:i + n, ..., 2 * kind + 1] = zero[..., 0]
    return codes[0], codes[1], sz


def _trees(case, rng):
    """Each request's number of nodes and their parents: node 0 is the newest token, a node's parent comes before it."""
    B, n = case["batch"], case["nodes"]
    counts = np.full(B, n) if not case.get("ragged") else rng.integers(1, n + 1, size=B)
    parents = []
    for c in counts:
        j = np.arange(1, c)
        near = rng.integers(np.maximum(0, j - 8), j)                 # a few children a node, paths of some length
        parents.append(np.concatenate([[-1], near]).astype(np.int32))
    return counts, parents


def _prepare_tree(case, seed):
    rng, gen = np.random.default_rng(seed), _generator(seed, 1)
    ps, H, B, Hq = case["page"], case["n_kv"], case["batch"], case["n_kv"] * case["gqa"]
    T = _lengths(case, rng)
    he = np.minimum(T, np.maximum(SINK, T - RECENT))
    counts, parents = _trees(case, rng)
    n, begin = int(counts.max()), np.concatenate([[0], np.cumsum(counts)])
    sees = np.zeros((B, n, n), bool)                                 # sees[b, i, j]: node i sees node j
    for b, par in enumerate(parents):
        for i, p in enumerate(par):
            if case["chain"]:
                sees[b, i, :i + 1] = True
            else:
                if p >= 0:
                    sees[b, i] = sees[b, p]
                sees[b, i, i] = True
    words, rows = (case["nodes"] + 31) // 32, B * case["nodes"]      # the buffers of a captured step: rows behind the last node stay as they are
    bits = np.zeros((B, n, words * 32), bool)
    bits[..., :n] = sees
    mask = np.packbits(bits, axis=-1, bitorder="little").view("<i4")             # [B, n, words]
    req, node = np.repeat(np.arange(B), counts), np.concatenate([np.arange(c) for c in counts])
    t4, n4 = _table([[(SINK, int(h))] for h in he], case, None, rng)
    tb, nb = _table([[(0, min(SINK, int(t))), (int(h), int(t + c))] for t, h, c in zip(T, he, counts)], case, None, rng)
    ck, cv, sz = _fill_int4(n4, case, gen)
    row = lambda k: (torch.randn((k, ps, H, DIM), generator=gen, device=DEV) * 1.3).to(torch.bfloat16)  # noqa: E731
    q = torch.randn((rows, Hq, DIM), generator=gen, device=DEV) * (torch.rand((DIM,), generator=gen, device=DEV) * 1.5 + 0.5)
    flat = np.zeros((rows, words), np.int32)
    flat[:len(req)] = mask[req, node]
    # the plain form's gather plan: positions of the sink and recent rows, then of the nodes, -1 where there is none
    win = np.full((B, SINK + RECENT + n), -1, np.int64)
    for b in range(B):
        p = np.concatenate([np.arange(min(SINK, T[b])), np.arange(max(he[b], min(SINK, T[b])), T[b])])
        win[b, :len(p)] = p
        win[b, SINK + RECENT:SINK + RECENT + counts[b]] = T[b] + np.arange(counts[b])
    return dict(T=_put(T.astype(np.int32)), he=_put(he.astype(np.int32)), max_pages=_pages(case), t4=_put(t4), tb=_put(tb), ck=ck, cv=cv, sz=sz,
                bk=row(nb), bv=row(nb), q=q.to(torch.bfloat16), win=_put(win), sees=_put(sees), begin=_put(begin.astype(np.int32)),
                mask=None if case["chain"] else _put(flat), out=torch.zeros((rows, Hq, DIM), dtype=torch.bfloat16, device=DEV),
                lse=torch.zeros((rows, Hq), dtype=torch.float32, device=DEV), req=_put(req), node=_put(node), counts=counts, sm_scale=1 / math.sqrt(DIM))


def _prepare_sample(case, seed):
    rng, gen = np.random.default_rng(seed), _generator(seed, 2)
    n, V, on = case["rows"], case["vocab"], case["filters"]
    # most logits in a broad hump, a few far above it, more or fewer from row to row
    x = torch.randn((n, V), generator=gen, device=DEV) * 2.0
    tall = torch.rand((n, V), generator=gen, device=DEV) < _put(10.0 ** rng.uniform(-4.5, -2.5, (n, 1)))
    x = x + tall * torch.rand((n, V), generator=gen, device=DEV) * _put(rng.uniform(4, 16, (n, 1)))
    x[:, V - V // 200:] = -math.inf                                  # the entries that pad a vocabulary stand for no token
    temp = np.where(rng.random(n) < 0.06, 0.0, rng.uniform(0.3, 1.4, n)).astype(np.float32)
    k = np.where(rng.random(n) < 0.15, 0, np.exp(rng.uniform(0, math.log(min(V, 1000)), n)).astype(np.int64)).astype(np.int32)
    p = np.where(rng.random(n) < 0.15, 1.0, rng.uniform(0.5, 0.999, n)).astype(np.float32)
    m = np.where(rng.random(n) < 0.3, 0.0, np.exp(rng.uniform(math.log(1e-4), math.log(0.3), n))).astype(np.float32)
    pick = lambda name, a: _put(a) if on in ("all", name) else None  # noqa: E731
    return dict(logits=x.to(DTYPES[case["dtype"]]), temperature=_put(temp), top_k=pick("top_k", k), top_p=pick("top_p", p), min_p=pick("min_p", m),
                u=torch.rand((n,), generator=gen, device=DEV), tokens=torch.zeros((n,), dtype=torch.int32, device=DEV))


def _prepare_accept(case, seed):
    rng, gen = np.random.default_rng(seed), _generator(seed, 3)
    ps, H, B, n = case["page"], case["n_kv"], case["batch"], case["nodes"]
    T = np.full(B, case["context"], np.int64) if B == 1 else rng.integers(max(1, case["context"] // 3), case["context"] + 1, size=B)
    counts, parents = _trees(dict(case, ragged=B > 1), rng)
    total = int(counts.sum())
    draft, target = rng.integers(0, 150000, total), rng.integers(0, 150000, total)
    lo = 0
    for c, par in zip(counts, parents):
        for j in range(1, c):                                        # siblings are different tokens
            draft[lo + j] = draft[lo + j] * 256 + j
        for i in range(c):                                           # four sampled tokens in five are one of the node's children
            kids = np.flatnonzero(par == i)
            if len(kids) and rng.random() < 0.8:
                target[lo + i] = draft[lo + rng.choice(kids)]
        lo += c
    spans = [[(int(t), int(t + c))] for t, c in zip(T, counts)]
    tb, nb = _table(spans, case, B * ((n + ps - 1) // ps + 1), rng)
    # every layer's pool, part of one allocation as a server makes it
    rows = lambda: torch.randn((case["layers"], nb, ps, H, DIM), generator=gen, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    longest = n + 1
    i32 = lambda *s: torch.full(s, -1, dtype=torch.int32, device=DEV)  # noqa: E731
    req = np.repeat(np.arange(B), counts)
    return dict(T=_put(T.astype(np.int32)), begin=_put(np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)), parents=_put(np.concatenate(parents)),
                draft=_put(draft.astype(np.int32)), target=_put(target.astype(np.int32)), tb=_put(tb), k=rows(), v=rows(),
                accepted=i32(B), path=i32(B, longest), tokens=i32(B, longest), new_len=i32(B), counts=counts,
                req=_put(req), node=_put(np.concatenate([np.arange(c) for c in counts])))


def prepare(case, seed):
    return dict(case=case, **{"tree": _prepare_tree, "sample": _prepare_sample, "accept": _prepare_accept}[case["op"]](case, seed))


# --------------------------------------------------------------------------- plain forms
def _values(codes, scale, zero, group):
    """The 32-bit values of 4-bit rows [..., 64 bytes] with scale and zero [..., 128 / group]."""
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (DIM // group, group))
    return (zero.float()[..., None] + q * scale.float()[..., None]).flatten(-2)


def _plain_tree(case, s):
    B, H, G, ps = case["batch"], case["n_kv"], case["gqa"], case["page"]
    n = s["sees"].shape[1]
    q = torch.zeros((B, n, H, G, DIM), device=DEV)
    total = len(s["req"])
    q[s["req"], s["node"]] = s["q"][:total].float().view(-1, H, G, DIM) * s["sm_scale"]
    t4 = s["t4"].clamp(min=0).long()
    k = _values(s["ck"][t4], s["sz"][t4][..., 0], s["sz"][t4][..., 1], case["group"])         # [B, P, H, ps, 128]
    hist = torch.einsum("bnhgd,bphsd->bhngps", q, k).flatten(-2)
    del k
    at = torch.arange(hist.shape[-1], device=DEV)
    hist = hist.masked_fill_(((at < SINK) | (at >= s["he"][:, None]))[:, None, None, None], -math.inf)
    w = s["win"].clamp(min=0)
    page = s["tb"].gather(1, w // ps).clamp(min=0).long()
    window = torch.einsum("bnhgd,bwhd->bhngw", q, s["bk"][page, w % ps].float())
    seen = torch.cat([(s["win"][:, None, :SINK + RECENT] >= 0).expand(B, n, -1), s["sees"]], -1)
    window = window.masked_fill(~seen[:, None, :, None], -math.inf)
    m = torch.maximum(hist.amax(-1, keepdim=True), window.amax(-1, keepdim=True)).clamp(min=-1e30)
    hist, window = hist.sub_(m).exp_(), torch.exp(window - m)
    weight = hist.sum(-1, keepdim=True) + window.sum(-1, keepdim=True)
    v = _values(s["cv"][t4], s["sz"][t4][..., 2], s["sz"][t4][..., 3], case["group"])
    out = torch.einsum("bhngps,bphsd->bhngd", hist.unflatten(-1, (-1, ps)), v)
    out = out + torch.einsum("bhngw,bwhd->bhngd", window, s["bv"][page, w % ps].float())
    out = torch.where(weight > 0, out / weight, 0.0).permute(0, 2, 1, 3, 4)[s["req"], s["node"]]
    lse = (m + torch.log(weight))[..., 0].permute(0, 2, 1, 3)[s["req"], s["node"]]
    s["out"][:total] = out.to(torch.bfloat16).reshape(-1, H * G, DIM)
    s["lse"][:total] = lse.reshape(-1, H * G)
    return s["out"], s["lse"]


def _plain_sample(case, s):
    """64 bits from the logits on: sums over a vocabulary decide between neighbours."""
    x = s["logits"].double()
    n, V = x.shape
    t = s["temperature"].double()[:, None]
    top = x.amax(-1, keepdim=True)
    w = torch.exp((x - top) / torch.where(t > 0, t, 1.0))
    order = torch.sort(x, dim=-1, descending=True, stable=True)[1]
    ws = w.gather(1, order)
    rank = torch.arange(V, device=DEV)
    keep = torch.ones((n, V), dtype=torch.bool, device=DEV)
    if s["top_k"] is not None:
        k = s["top_k"][:, None]
        keep &= (k <= 0) | (rank < k)
    if s["top_p"] is not None:
        mass = torch.where(keep, ws, 0.0)
        before = torch.cumsum(mass, -1) - mass
        p = s["top_p"].double()[:, None]
        keep &= (p >= 1) | (before < p * mass.sum(-1, keepdim=True))
    if s["min_p"] is not None:
        keep &= ws >= s["min_p"].double()[:, None]
    kept = torch.zeros((n, V), dtype=torch.float64, device=DEV).scatter_(1, order, torch.where(keep, ws, 0.0))
    sums = torch.cumsum(kept, -1)
    drawn = (sums > s["u"].double()[:, None] * sums[:, -1:]).int().argmax(-1)
    s["tokens"].copy_(torch.where(t[:, 0] > 0, drawn, (x == top).int().argmax(-1)))
    return s["tokens"]


def _plain_accept(case, s):
    B, n, ps = case["batch"], case["nodes"], case["page"]
    T = s["T"]
    parents, draft, target = (torch.full((B, n), -2, dtype=torch.long, device=DEV) for _ in range(3))
    for to, a in ((parents, "parents"), (draft, "draft"), (target, "target")):
        to[s["req"], s["node"]] = s[a].long()
    cur, alive = torch.zeros(B, dtype=torch.long, device=DEV), torch.ones(B, dtype=torch.bool, device=DEV)
    path, tokens = torch.full((B, n + 1), -1, dtype=torch.long, device=DEV), torch.full((B, n + 1), -1, dtype=torch.long, device=DEV)
    accepted = torch.zeros(B, dtype=torch.long, device=DEV)
    for d in range(n):
        tok = target.gather(1, cur[:, None])
        path[:, d], tokens[:, d] = torch.where(alive, cur, -1), torch.where(alive, tok[:, 0], -1)
        accepted += alive
        hit = (parents == cur[:, None]) & (draft == tok) & alive[:, None]
        alive = hit.any(-1)
        cur = torch.where(alive, hit.int().argmax(-1), cur)
    s["accepted"].copy_(accepted)
    s["path"].copy_(path)
    s["tokens"].copy_(tokens)
    s["new_len"].copy_(T + accepted)
    b, j = torch.arange(B, device=DEV)[:, None], torch.arange(n, device=DEV)
    on = (path[:, :n] >= 0) & (path[:, :n] != j)
    src, dst = T[:, None] + path[:, :n].clamp(min=0), T[:, None] + j
    pages = s["tb"].shape[1]
    of = lambda p: s["tb"][b, (p // ps).clamp(max=pages - 1)].long()  # noqa: E731
    src_page, dst_page, src_slot, dst_slot = of(src)[on], of(dst)[on], (src % ps)[on], (dst % ps)[on]
    for rows in (s["k"], s["v"]):
        rows[:, dst_page, dst_slot] = rows[:, src_page, src_slot]
    return s["accepted"], s["path"], s["tokens"], s["new_len"], s["k"], s["v"]


# --------------------------------------------------------------------------- the library's calls
def _handles(case, s):
    """Layout, pool descriptors and workspaces, made on a state's first pass and kept, as a server keeps them."""
    if "lib" not in s:
        from bit_kv_cache_oscar_gb300 import binding as ob
        h = dict(ob=ob)
        if case["op"] != "sample":
            h["L"] = L = ob.Layout(case["n_kv"], case["gqa"], case["page"], case["group"], SINK, RECENT)
        if case["op"] == "tree":
            h["int4"], h["bf16"] = ob.Int4Pool(s["ck"], s["cv"], s["sz"]), ob.Bf16Pool(s["bk"], s["bv"])
            splits = ob.oscar_suggest_splits_tree_int4(L, case["batch"], case["nodes"], case["context"],
                                                       torch.cuda.get_device_properties(0).multi_processor_count)
            h["partials"] = ob.Partials.empty(L, s["q"].shape[0], splits)
        if case["op"] == "accept":
            h["pools"] = [ob.Bf16Pool(k, v) for k, v in zip(s["k"], s["v"])]
        s["lib"] = h
    return s["lib"]


def _run_own(case, s):
    h = _handles(case, s)
    ob, op = h["ob"], case["op"]
    if op == "tree":
        ob.oscar_tree_attention_int4(h["L"], s["q"], s["begin"], s["mask"], case["nodes"], h["bf16"], s["tb"], h["int4"], s["t4"], s["T"], s["he"],
                                     s["sm_scale"], h["partials"], out=s["out"], lse=s["lse"])
        return s["out"], s["lse"]
    if op == "sample":
        ob.oscar_sample(s["logits"], s["temperature"], s["u"], s["tokens"], top_k=s["top_k"], top_p=s["top_p"], min_p=s["min_p"])
        return s["tokens"]
    ob.oscar_tree_accept(h["L"], s["target"], s["draft"], s["parents"], s["begin"], case["nodes"], s["T"], s["accepted"], s["path"], s["tokens"], s["new_len"],
                         pools=h["pools"], page_table=s["tb"])
    return s["accepted"], s["path"], s["tokens"], s["new_len"], s["k"], s["v"]


def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"tree": _plain_tree, "sample": _plain_sample, "accept": _plain_accept}[case["op"]](case, state)


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    if case["op"] == "sample":
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": case["rows"] * (case["vocab"] * size + 24), "flops": case["rows"] * case["vocab"] * 4}
    H, G, B = case["n_kv"], case["gqa"], case["batch"]
    nodes = case["nodes"] if case["op"] == "tree" and not case["ragged"] or B == 1 else (case["nodes"] + 1) / 2
    if case["op"] == "accept":
        moved = B * nodes / 4                                        # about a quarter of the nodes lie on the path
        return {"bytes": case["layers"] * moved * H * 2 * 2 * DIM * 2 + B * nodes * 12, "flops": B * nodes * 4}
    row4 = DIM // 2 + 4 * (DIM // case["group"])                     # bytes of one 4-bit row with its scale and zero
    T = case["context"] * (5 / 6 if case["ragged"] else 1)           # ragged lengths lie between two thirds and all of the context
    hist = max(0.0, min(T, max(SINK, T - RECENT)) - SINK)
    near = min(T, SINK + RECENT) + nodes
    return {"bytes": B * H * (hist * 2 * row4 + near * 2 * DIM * 2 + nodes * G * (DIM * 4 + 4)), "flops": B * H * G * nodes * (hist + near) * DIM * 4}


# --------------------------------------------------------------------------- 64 bits, from the definitions
def _rows64(codes, sz, kind, group):
    """[n, 64] bytes and [n, groups, 4] of one head's rows -> [n, 128] in 64 bits."""
    n = codes.shape[0]
    nib = torch.empty((n, DIM), dtype=torch.float64, device=DEV)
    nib[:, 0::2] = (codes % 16).double()
    nib[:, 1::2] = (codes // 16).double()
    sz = sz.double()
    return (nib.view(n, -1, group) * sz[..., 2 * kind, None] + sz[..., 2 * kind + 1, None]).reshape(n, DIM)


def _cache64(case, s, b, h, kind):
    """All rows of (request, kv head) in position order, its nodes' behind them, in 64 bits."""
    ps, T, he = case["page"], int(s["T"][b]), int(s["he"][b])
    p = torch.arange(T + int(s["counts"][b]), device=DEV)
    rows = torch.zeros((len(p), DIM), dtype=torch.float64, device=DEV)
    far = (p >= SINK) & (p < he)
    pf, pn = p[far], p[~far]
    if len(pf):
        pg = s["t4"][b, pf // ps].long()
        rows[far] = _rows64(s["cv" if kind else "ck"][pg, h, pf % ps], s["sz"][pg, h, pf % ps], kind, case["group"])
    rows[~far] = s["bv" if kind else "bk"][s["tb"][b, pn // ps].long(), pn % ps, h].double()
    return rows


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "sample":
        got = np.zeros(case["rows"], np.int32)
        for r in range(case["rows"]):
            x = s["logits"][r].double().cpu().numpy()
            t = float(s["temperature"][r])
            if t == 0:
                got[r] = int(np.argmax(x))
                continue
            best = np.argsort(-x, kind="stable")
            w = np.exp((x[best] - x[best[0]]) / t)
            if s["top_k"] is not None and int(s["top_k"][r]) > 0:
                w = w[:int(s["top_k"][r])]
            cut = len(w)
            if s["top_p"] is not None and float(s["top_p"][r]) < 1:
                sums = np.cumsum(w)
                cut = min(cut, int(np.searchsorted(sums, float(s["top_p"][r]) * sums[-1], side="left")) + 1)
            if s["min_p"] is not None:
                cut = min(cut, int(np.count_nonzero(w >= float(s["min_p"][r]))))
            ids = np.sort(best[:cut])
            sums = np.cumsum(np.exp((x[ids] - x[best[0]]) / t))
            got[r] = ids[int(np.searchsorted(sums, float(s["u"][r]) * sums[-1], side="right"))]
        return _put(got)
    H, G, ps, B = case["n_kv"], case["gqa"], case["page"], case["batch"]
    if case["op"] == "accept":
        begin, T = s["begin"].cpu().numpy(), s["T"].cpu().numpy()
        par, draft, target = (s[k].cpu().numpy() for k in ("parents", "draft", "target"))
        accepted, path, tokens = (s[k].cpu().numpy() for k in ("accepted", "path", "tokens"))
        before = s["k"], s["v"]
        after = [a.double() for a in before]
        for b in range(B):
            lo, hi = int(begin[b]), int(begin[b + 1])
            child = {(int(par[j]), int(draft[j])): j - lo for j in range(hi - 1, lo, -1)}
            way = [0]
            while (way[-1], int(target[lo + way[-1]])) in child:
                way.append(child[way[-1], int(target[lo + way[-1]])])
            accepted[b] = len(way)
            path[b, :len(way)], tokens[b, :len(way)] = way, target[lo + np.array(way)]
            src, dst = _put(T[b] + np.array(way)).long(), _put(T[b] + np.arange(len(way))).long()
            for x, y in zip(before, after):
                y[:, s["tb"][b, dst // ps].long(), dst % ps] = x[:, s["tb"][b, src // ps].long(), src % ps].double()
        return _put(accepted), _put(path), _put(tokens), _put((T + accepted).astype(np.int32)), *after
    out, lse = s["out"].double(), s["lse"].double()
    for b in range(B):
        T, lo, hi = int(s["T"][b]), int(s["begin"][b]), int(s["begin"][b + 1])
        hidden = torch.cat([torch.zeros((hi - lo, T), dtype=torch.bool, device=DEV), ~s["sees"][b, :hi - lo, :hi - lo]], 1)
        for h in range(H):
            z = s["q"][lo:hi, h * G:(h + 1) * G].double() @ _cache64(case, s, b, h, 0).T * s["sm_scale"]
            z = z.masked_fill_(hidden[:, None], -math.inf)
            lse[lo:hi, h * G:(h + 1) * G] = torch.logsumexp(z, -1)
            out[lo:hi, h * G:(h + 1) * G] = torch.softmax(z, -1) @ _cache64(case, s, b, h, 1)
    return out, lse
