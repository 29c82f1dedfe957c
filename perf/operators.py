"""The serving operators around a 4-bit key/value history, in plain form and as the library's calls.

Five operators, in the order a decode step and a cache manager use them:

  append   per-head RMS norm and rotary position of new queries and keys, keys and values written to the paged BF16 pool
  demote   BF16 rows of the paged cache to 4 bits with a scale and zero per group, and back to BF16 (promote)
  decode   attention of one new token per request over the 4-bit history and the BF16 sink and recent rows
  mass     the attention weight each cached position received in that step, added to a running sum
  evict    the positions of largest running weight of each kv head kept, moved to new pages, read back in BF16

A cache is [sink | history | recent]: positions [0, 64) and the last 256 are BF16, what lies between is 4-bit.
"""
import math

import numpy as np
import torch

own = False

DIM, SINK, RECENT = 128, 64, 256
EPS = 1e-6
DEV = "cuda"


# --------------------------------------------------------------------------- cases
def listed():
    shape_8b = dict(n_kv=8, gqa=4, page=64, group=128)       # 32 query heads, 8 kv heads
    shape_32b = dict(n_kv=8, gqa=8, page=64, group=32)       # 64 query heads, 8 kv heads, small groups
    small = dict(n_kv=2, gqa=4, page=16, group=128)          # 8 query heads, 2 kv heads, 16-token pages
    return [
        # one new token of a single conversation deep into its context: latency only
        dict(name="append_step_b1", op="append", batch=1, tokens=1, pad=0, context=100000, rot=128, pairs=False, **shape_8b),
        # a prompt's chunk, its last rows padding
        dict(name="append_prompt_8k", op="append", batch=1, tokens=8192, pad=77, context=32768, rot=128, pairs=False, **shape_8b),
        # every request's oldest recent token leaves the BF16 window
        dict(name="demote_step_b32", op="demote", batch=32, rows=1, context=32768, ragged=True, **shape_8b),
        # the whole history of a long prompt after its prefill
        dict(name="demote_prompt_100k", op="demote", batch=1, rows=99680, context=100000, ragged=False, **shape_8b),
        # a short conversation on a small model: latency only
        dict(name="decode_1k_b1", op="decode", batch=1, context=1024, ragged=False, **small),
        # one long conversation
        dict(name="decode_100k_b1", op="decode", batch=1, context=100000, ragged=False, **shape_8b),
        # a full serving batch of unequal lengths
        dict(name="decode_ragged_b32", op="decode", batch=32, context=100000, ragged=True, **shape_8b),
        # 64 query heads, groups of 32 channels
        dict(name="decode_131k_b4_g32", op="decode", batch=4, context=131072, ragged=False, **shape_32b),
        # the weights of one step, one conversation and a batch
        dict(name="mass_32k_b1", op="mass", batch=1, context=32768, ragged=False, **shape_8b),
        dict(name="mass_ragged_b8", op="mass", batch=8, context=100000, ragged=True, **shape_8b),
        # a short history cut to a quarter, a long one cut to half
        dict(name="evict_4k_b1", op="evict", batch=1, context=4096, ragged=False, keep=0.25, **small),
        dict(name="evict_100k_b2", op="evict", batch=2, context=100000, ragged=True, keep=0.5, **shape_8b),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    op = rng.choice(["append", "demote", "decode", "mass", "evict"])
    n_kv, gqa = rng.choice([(1, 8), (2, 4), (4, 2), (8, 1), (8, 4), (8, 8), (5, 4)])
    c = dict(op=op, n_kv=n_kv, gqa=gqa, page=rng.choice([16, 32, 64]), group=rng.choice([32, 64, 128]))
    if op == "append":
        tokens = log(1, 8192)
        c |= dict(batch=min(tokens, log(1, 64)), tokens=tokens, pad=rng.choice([0, tokens // 9]), context=log(tokens + 1, 100000),
                  rot=rng.choice([32, 64, 128]), pairs=rng.random() < 0.3)
        return c
    context = log(1 if op == "decode" or op == "mass" else 400, 100000)
    batch = min(log(1, 64), max(1, 1600000 // context))
    c |= dict(batch=batch, context=context, ragged=rng.random() < 0.7)
    if op == "demote":
        hist = max(1, context // 2 - SINK - RECENT)
        c["rows"] = min(log(1, hist), max(1, 99680 // batch))
    if op == "evict":
        c |= dict(batch=min(batch, max(1, 100000 // context)), keep=round(rng.uniform(0.05, 0.95), 3))
    return c


# --------------------------------------------------------------------------- inputs
def _generator(*parts):
    return torch.Generator(device=DEV).manual_seed(int(np.random.SeedSequence([abs(int(p)) for p in parts]).generate_state(1, np.uint64)[0] >> 1))


def _lengths(case, rng):
    T, B = case["context"], case["batch"]
    if not case.get("ragged"):
        return np.full(B, T, np.int64)
    return rng.integers(max(1, T * 2 // 3), T + 1, size=B)


def _hist_end(T):
    return np.minimum(T, np.maximum(SINK, T - RECENT))


def _pages(case):
    """Pages of the longest context a case can have: the width of its page tables, whatever lengths a seed draws."""
    return (max(case["context"], SINK + RECENT + 1) + case["page"] - 1) // case["page"]


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


def _put(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


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


def _cache(case, seed):
    """A batch's mixed cache: lengths, page tables, the 4-bit pool of its history, the BF16 pool of its sink and recent rows, a query."""
    rng, gen = np.random.default_rng(seed), _generator(seed, 1)
    ps, H, B = case["page"], case["n_kv"], case["batch"]
    T = _lengths(case, rng)
    he = _hist_end(T)
    t4, n4 = _table([[(SINK, int(h))] for h in he], case, None, rng)
    tb, nb = _table([[(0, min(SINK, int(t))), (int(h), int(t))] for t, h in zip(T, he)], case, None, rng)
    ck, cv, sz = _fill_int4(n4, case, gen)
    row = lambda n: (torch.randn((n, ps, H, DIM), generator=gen, device=DEV) * 1.3).to(torch.bfloat16)  # noqa: E731
    q = torch.randn((B, H * case["gqa"], DIM), generator=gen, device=DEV) * (torch.rand((DIM,), generator=gen, device=DEV) * 1.5 + 0.5)
    # positions of the sink and recent rows, -1 behind the last: the plain form's gather plan
    win = np.full((B, SINK + RECENT), -1, np.int64)
    for b in range(B):
        p = np.concatenate([np.arange(min(SINK, T[b])), np.arange(max(he[b], min(SINK, T[b])), T[b])])
        win[b, :len(p)] = p
    return dict(T=_put(T.astype(np.int32)), he=_put(he.astype(np.int32)), max_pages=_pages(case), t4=_put(t4), tb=_put(tb), ck=ck, cv=cv, sz=sz,
                bk=row(nb), bv=row(nb), q=q.to(torch.bfloat16), win=_put(win), sm_scale=1 / math.sqrt(DIM))


def _rope_table(n):
    """cos (64) and sin (64) of position x frequency, angles in 64 bits."""
    inv = 1e6 ** (-torch.arange(0, DIM, 2, dtype=torch.float64, device=DEV) / DIM)
    a = torch.arange(n, dtype=torch.float64, device=DEV)[:, None] * inv
    return torch.cat([a.cos(), a.sin()], 1).float()


def _prepare_append(case, seed):
    rng, gen = np.random.default_rng(seed), _generator(seed, 2)
    H, Hq, ps, B, n = case["n_kv"], case["n_kv"] * case["gqa"], case["page"], case["batch"], case["tokens"]
    valid = n - case["pad"]
    # each request's run of new tokens ends at its context: token i belongs to request req[i], at position pos[i]
    per = np.diff(np.concatenate([[0], np.sort(rng.integers(0, valid + 1, B - 1)), [valid]])) if B < valid else np.array([1] * valid + [0] * (B - valid))
    ends = np.minimum(np.maximum(_lengths(dict(case, ragged=B > 1), rng), per), case["context"])
    req = np.concatenate([np.repeat(np.arange(B), per), np.zeros(case["pad"], np.int64)])
    pos = np.concatenate([np.arange(e - c, e) for e, c in zip(ends, per)] + [np.full(case["pad"], -1)])
    table, n_pages = _table([[(int(e - c), int(e))] for e, c in zip(ends, per)], case, valid // ps + 2 * B, rng)
    # queries, keys and values as they leave one projection: slices of a row, not tensors of their own
    qkv = torch.randn((n, (Hq + 2 * H) * DIM), generator=gen, device=DEV) * 2
    weight = lambda: (1 + 0.2 * torch.randn(DIM, generator=gen, device=DEV)).to(torch.bfloat16)  # noqa: E731
    pool = lambda: torch.zeros((n_pages, ps, H, DIM), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    return dict(qkv=qkv.to(torch.bfloat16), wq=weight(), wk=weight(), rope=_rope_table(case["context"]), req=_put(req.astype(np.int32)), pos=_put(pos.astype(np.int32)),
                table=_put(table), k=pool(), v=pool(), q_out=torch.zeros((n, Hq, DIM), dtype=torch.bfloat16, device=DEV), valid=valid)


def _prepare_demote(case, seed):
    rng, gen = np.random.default_rng(seed), _generator(seed, 3)
    H, ps, B = case["n_kv"], case["page"], case["batch"]
    T = np.maximum(_lengths(case, rng), SINK + RECENT + 1)
    end = T - RECENT
    begin = np.maximum(SINK, end - case["rows"])
    spans = [[(int(b), int(e))] for b, e in zip(begin, end)]
    most = B * (case["rows"] // ps + 2)
    tb, nb = _table(spans, case, most, rng)
    t4, n4 = _table(spans, case, most, rng)
    to, no = _table(spans, case, most, rng)
    sigma = torch.rand((2, H, DIM), generator=gen, device=DEV) * 1.5 + 0.5
    row = lambda s: (torch.randn((nb, ps, H, DIM), generator=gen, device=DEV) * s).to(torch.bfloat16)  # noqa: E731
    zeros = lambda: torch.zeros((no, ps, H, DIM), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    n4_shape = (n4, H, ps)
    return dict(bk=row(sigma[0]), bv=row(sigma[1]), tb=_put(tb), t4=_put(t4), to=_put(to), ok=zeros(), ov=zeros(),
                ck=torch.zeros(n4_shape + (DIM // 2,), dtype=torch.uint8, device=DEV), cv=torch.zeros(n4_shape + (DIM // 2,), dtype=torch.uint8, device=DEV),
                sz=torch.zeros(n4_shape + (DIM // case["group"], 4), dtype=torch.bfloat16, device=DEV),
                begin=_put(begin.astype(np.int32)), end=_put(end.astype(np.int32)),
                req=_put(np.repeat(np.arange(B), end - begin)), pos=_put(np.concatenate([np.arange(b, e) for b, e in zip(begin, end)])))


def _prepare_mass(case, seed):
    s = _cache(case, seed)
    B, H, G, N = case["batch"], case["n_kv"], case["gqa"], s["max_pages"] * case["page"]
    hist, window = _scores(case, s)
    s["lse"] = torch.logsumexp(torch.cat([hist, window], -1).double(), -1).float().view(B, H * G)
    # what earlier steps left: most positions saw little, a few a lot
    s["mass"] = torch.exp(torch.randn((B, H, N), generator=_generator(seed, 4), device=DEV) * 2 - 6)
    return s


def _prepare_evict(case, seed):
    rng, gen = np.random.default_rng(seed), _generator(seed, 5)
    H, ps, B = case["n_kv"], case["page"], case["batch"]
    T = np.maximum(_lengths(case, rng), SINK + RECENT + 1)
    he = T - RECENT
    keep = np.maximum(1, ((he - SINK) * case["keep"]).astype(np.int64))
    longest = max(1, int(max(1, case["context"] - SINK - RECENT) * case["keep"]))
    t4, n4 = _table([[(SINK, int(h))] for h in he], case, None, rng)
    kept_spans = [[(SINK, SINK + int(k))] for k in keep]
    tn, nn = _table(kept_spans, case, B * (longest // ps + 1), rng)
    to, no = _table(kept_spans, case, B * (longest // ps + 1), rng)
    ck, cv, sz = _fill_int4(n4, case, gen)
    mass = torch.exp(torch.randn((B, H, _pages(case) * ps), generator=gen, device=DEV) * 2 - 6)
    mass[torch.rand(mass.shape, generator=gen, device=DEV) < 0.05] = 0                       # positions that no query has reached yet
    like = lambda a: torch.zeros((nn,) + tuple(a.shape[1:]), dtype=a.dtype, device=DEV)  # noqa: E731
    zeros = lambda: torch.zeros((no, ps, H, DIM), dtype=torch.bfloat16, device=DEV)  # noqa: E731
    end = SINK + keep
    return dict(T=_put(T.astype(np.int32)), he=_put(he.astype(np.int32)), keep=_put(keep.astype(np.int32)), t4=_put(t4), tn=_put(tn), to=_put(to), ck=ck, cv=cv, sz=sz,
                mass=mass, nck=like(ck), ncv=like(cv), nsz=like(sz), ok=zeros(), ov=zeros(), mass_out=torch.zeros_like(mass),
                kept=torch.full((B, H, longest), -1, dtype=torch.int32, device=DEV), begin=_put(np.full(B, SINK, np.int32)), end=_put(end.astype(np.int32)),
                req=_put(np.repeat(np.arange(B), keep)), row=_put(np.concatenate([np.arange(k) for k in keep])))


def prepare(case, seed):
    op = case["op"]
    if op == "append":
        return dict(case=case, **_prepare_append(case, seed))
    if op == "demote":
        return dict(case=case, **_prepare_demote(case, seed))
    if op == "decode":
        return dict(case=case, **_cache(case, seed))
    if op == "mass":
        return dict(case=case, **_prepare_mass(case, seed))
    return dict(case=case, **_prepare_evict(case, seed))


# --------------------------------------------------------------------------- plain forms
def _norm_rotate(x, weight, cos, sin, rot, pairs):
    """x [n, heads, 128] in 32 bits: RMS norm of each head, then the rotation of its first `rot` channels."""
    x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS) * weight.float()
    r = x[..., :rot]
    cos, sin = cos[:, None], sin[:, None]
    if pairs:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = r[..., :rot // 2], r[..., rot // 2:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([r, x[..., rot:]], -1)


def _plain_append(case, s):
    H, G, ps, n, rot = case["n_kv"], case["gqa"], case["page"], s["valid"], case["rot"]
    x = s["qkv"][:n].float().view(n, -1, DIM)
    pos, req = s["pos"][:n].long(), s["req"][:n].long()
    rope = s["rope"][pos]
    cos, sin = rope[:, :rot // 2], rope[:, DIM // 2:DIM // 2 + rot // 2]
    s["q_out"][:n] = _norm_rotate(x[:, :H * G], s["wq"], cos, sin, rot, case["pairs"]).to(torch.bfloat16)
    page, slot = s["table"][req, pos // ps].long(), pos % ps
    s["k"][page, slot] = _norm_rotate(x[:, H * G:H * G + H], s["wk"], cos, sin, rot, case["pairs"]).to(torch.bfloat16)
    s["v"][page, slot] = s["qkv"][:n].view(n, -1, DIM)[:, H * G + H:]
    return s["q_out"], s["k"], s["v"]


def _restore(x, group):
    """4-bit rounding of rows [..., 128] and the values the codes stand for; the code's border is decided in 64 bits."""
    x = x.float().unflatten(-1, (DIM // group, group))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    zero, scale = lo.to(torch.bfloat16).float(), ((hi - lo) / 15).to(torch.bfloat16).float()
    code = ((x.double() - zero.double()) / torch.where(scale == 0, 1.0, scale.double())).round().clamp(0, 15).float()
    code = torch.where(scale == 0, 0.0, code)
    return (zero + code * scale).flatten(-2).to(torch.bfloat16)


def _plain_demote(case, s):
    ps = case["page"]
    req, pos = s["req"], s["pos"]
    src, dst = s["tb"][req, pos // ps].long(), s["to"][req, pos // ps].long()
    s["ok"][dst, pos % ps] = _restore(s["bk"][src, pos % ps], case["group"])
    s["ov"][dst, pos % ps] = _restore(s["bv"][src, pos % ps], case["group"])
    return s["ok"], s["ov"]


def _values(codes, scale, zero, group):
    """The 32-bit values of 4-bit rows [..., 64 bytes] with scale and zero [..., 128 / group]."""
    q = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).float().unflatten(-1, (DIM // group, group))
    return (zero.float()[..., None] + q * scale.float()[..., None]).flatten(-2)


def _scores(case, s):
    """Logits of the history [B, Hkv, G, N] and of the sink and recent rows [B, Hkv, G, 320], -inf where there is no row."""
    B, H, G, ps = case["batch"], case["n_kv"], case["gqa"], case["page"]
    t4 = s["t4"].clamp(min=0).long()
    q = s["q"].float().view(B, H, G, DIM) * s["sm_scale"]
    k = _values(s["ck"][t4], s["sz"][t4][..., 0], s["sz"][t4][..., 1], case["group"])         # [B, P, H, ps, 128]
    hist = torch.einsum("bhgd,bphsd->bhgps", q, k).flatten(-2)
    n = torch.arange(hist.shape[-1], device=DEV)
    hist = hist.masked_fill(((n < SINK) | (n >= s["he"][:, None]))[:, None, None], -math.inf)
    w = s["win"].clamp(min=0)
    page = s["tb"].gather(1, w // ps).clamp(min=0).long()
    window = torch.einsum("bhgd,bwhd->bhgw", q, s["bk"][page, w % ps].float())
    return hist, window.masked_fill((s["win"] < 0)[:, None, None], -math.inf)


def _plain_decode(case, s):
    B, H, G, ps = case["batch"], case["n_kv"], case["gqa"], case["page"]
    hist, window = _scores(case, s)
    m = torch.maximum(hist.amax(-1, keepdim=True), window.amax(-1, keepdim=True))
    hist, window = torch.exp(hist - m), torch.exp(window - m)
    total = hist.sum(-1, keepdim=True) + window.sum(-1, keepdim=True)
    t4, w = s["t4"].clamp(min=0).long(), s["win"].clamp(min=0)
    v = _values(s["cv"][t4], s["sz"][t4][..., 2], s["sz"][t4][..., 3], case["group"])
    out = torch.einsum("bhgps,bphsd->bhgd", hist.unflatten(-1, (-1, ps)), v)
    page = s["tb"].gather(1, w // ps).clamp(min=0).long()
    out = out + torch.einsum("bhgw,bwhd->bhgd", window, s["bv"][page, w % ps].float())
    return (out / total).to(torch.bfloat16).view(B, H * G, DIM), (m + torch.log(total)).view(B, H * G)


def _plain_mass(case, s):
    B, H, G = case["batch"], case["n_kv"], case["gqa"]
    hist, window = _scores(case, s)
    lse = s["lse"].view(B, H, G, 1)
    s["mass"] += torch.exp(hist - lse).sum(2)
    w = s["win"].clamp(min=0)[:, None].expand(B, H, -1)
    s["mass"].scatter_add_(2, w, torch.exp(window - lse).sum(2))
    return s["mass"]


def _plain_evict(case, s):
    H, ps = case["n_kv"], case["page"]
    B, _, N = s["mass"].shape
    n = torch.arange(N, device=DEV)
    he, keep, T = s["he"][:, None, None], s["keep"][:, None, None], s["T"][:, None, None]
    rank = torch.where((n >= SINK) & (n < he), s["mass"], -1.0)
    best = torch.sort(rank, dim=-1, descending=True, stable=True)[1][..., :s["kept"].shape[-1]]
    j = torch.arange(best.shape[-1], device=DEV)
    best = torch.sort(torch.where(j < keep, best, N))[0]
    s["kept"].copy_(torch.where(j < keep, best, -1))
    # the running weights move with their rows: sink, kept history, recent rows, nothing behind them
    moved = torch.cat([n[:SINK].expand(B, H, SINK), best, torch.zeros((B, H, N), dtype=torch.long, device=DEV)], -1)[..., :N]
    at = torch.where(n < SINK + keep, moved, n - keep - SINK + he)
    s["mass_out"].copy_(torch.where(n < T - he + SINK + keep, s["mass"].gather(2, at.clamp(0, N - 1)), 0.0))
    req, row = s["req"], s["row"]
    src = best[req, :, row]                                                                    # [rows, Hkv]: the old position of each kept row
    head = torch.arange(H, device=DEV)
    page, slot = s["t4"][req[:, None], src // ps].long(), src % ps
    to, at = s["to"][req, (SINK + row) // ps].long(), (SINK + row) % ps
    sz = s["sz"][page, head, slot]
    s["ok"][to, at] = _values(s["ck"][page, head, slot], sz[..., 0], sz[..., 1], case["group"]).to(torch.bfloat16)
    s["ov"][to, at] = _values(s["cv"][page, head, slot], sz[..., 2], sz[..., 3], case["group"]).to(torch.bfloat16)
    return s["kept"], s["mass_out"], s["ok"], s["ov"]


# --------------------------------------------------------------------------- the library's calls
def _handles(case, s):
    """Layout, pool descriptors and workspaces, made on a state's first pass and kept, as a server keeps them."""
    if "lib" not in s:
        from bit_kv_cache_oscar_gb300 import binding as ob
        L = ob.Layout(case["n_kv"], case["gqa"], case["page"], case["group"], SINK, RECENT)
        h = dict(ob=ob, L=L)
        if "ck" in s:
            h["int4"] = ob.Int4Pool(s["ck"], s["cv"], s["sz"])
        if "bk" in s:
            h["bf16"] = ob.Bf16Pool(s["bk"], s["bv"])
        if case["op"] == "append":
            h["bf16"] = ob.Bf16Pool(s["k"], s["v"])
        if case["op"] == "decode":
            B, Hq = case["batch"], case["n_kv"] * case["gqa"]
            splits = ob.oscar_suggest_splits_int4(L, B, case["context"], torch.cuda.get_device_properties(0).multi_processor_count)
            h["partials"] = ob.Partials.empty(L, B, splits)
            h["counters"] = torch.zeros(B * case["n_kv"], dtype=torch.int32, device=DEV)
            h["out"] = torch.empty((B, Hq, DIM), dtype=torch.bfloat16, device=DEV)
            h["lse"] = torch.empty((B, Hq), dtype=torch.float32, device=DEV)
        if case["op"] in ("demote", "evict"):
            h["back"] = ob.Bf16Pool(s["ok"], s["ov"])
        if case["op"] == "evict":
            h["new"] = ob.Int4Pool(s["nck"], s["ncv"], s["nsz"])
        s["lib"] = h
    return s["lib"]


def _run_own(case, s):
    h = _handles(case, s)
    ob, L, op = h["ob"], h["L"], case["op"]
    if op == "append":
        Hq, H = L.n_q_heads, L.n_kv_heads
        x = s["qkv"].view(-1, Hq + 2 * H, DIM)
        ob.oscar_append_kv(L, x[:, :Hq], x[:, Hq:Hq + H], x[:, Hq + H:], h["bf16"], s["table"], s["req"], s["pos"], s["q_out"],
                           q_weight=s["wq"], k_weight=s["wk"], eps=EPS, rope=s["rope"], rot_dim=case["rot"], interleaved=case["pairs"])
        return s["q_out"], s["k"], s["v"]
    if op == "demote":
        ob.oscar_demote_int4(L, h["bf16"], s["tb"], h["int4"], s["t4"], s["begin"], s["end"], 1.0, 1.0)
        ob.oscar_promote_int4(L, h["int4"], s["t4"], h["back"], s["to"], s["begin"], s["end"])
        return s["ok"], s["ov"]
    if op == "decode":
        ob.oscar_decode_attention_int4(L, s["q"], h["bf16"], s["tb"], h["int4"], s["t4"], s["T"], s["he"], s["sm_scale"], h["partials"],
                                       out=h["out"], lse=h["lse"], merge_counters=h["counters"])
        return h["out"], h["lse"]
    if op == "mass":
        ob.oscar_attention_mass_int4(L, s["q"], h["bf16"], s["tb"], h["int4"], s["t4"], s["T"], s["he"], s["sm_scale"], s["lse"], s["mass"])
        return s["mass"]
    ob.oscar_evict_int4(L, h["int4"], s["t4"], h["new"], s["tn"], s["T"], s["he"], s["keep"], s["mass"], s["mass_out"], s["kept"])
    ob.oscar_promote_int4(L, h["new"], s["tn"], h["back"], s["to"], s["begin"], s["end"])
    return s["kept"], s["mass_out"], s["ok"], s["ov"]


def run(state):
    case = state["case"]
    if own:
        return _run_own(case, state)
    return {"append": _plain_append, "demote": _plain_demote, "decode": _plain_decode, "mass": _plain_mass, "evict": _plain_evict}[case["op"]](case, state)


# --------------------------------------------------------------------------- what a pass cannot do without
def work(case):
    H, G, B, ps = case["n_kv"], case["gqa"], case["batch"], case["page"]
    row4 = DIM // 2 + 4 * (DIM // case["group"])                    # bytes of one 4-bit row with its scale and zero
    if case["op"] == "append":
        n = case["tokens"] - case["pad"]
        return {"bytes": n * ((G + 2) * H * DIM * 2 * 2 + 4 * case["rot"] + 8), "flops": n * (G + 1) * H * DIM * 8}
    T = case["context"] * (5 / 6 if case.get("ragged") else 1)      # ragged lengths lie between two thirds and all of the context
    hist = max(0.0, min(T, max(SINK, T - RECENT)) - SINK)
    if case["op"] == "demote":
        rows = B * min(case["rows"], max(1, hist)) * H * 2
        return {"bytes": rows * (2 * DIM * 2 + 2 * row4), "flops": rows * DIM * 8}
    near = min(T, SINK + RECENT)
    if case["op"] == "decode":
        return {"bytes": B * H * (hist * 2 * row4 + near * 2 * DIM * 2 + G * DIM * 4), "flops": B * H * G * (hist + near) * DIM * 4}
    if case["op"] == "mass":
        return {"bytes": B * H * (hist * (row4 + 8) + near * (DIM * 2 + 8) + G * DIM * 2), "flops": B * H * G * (hist + near) * DIM * 2}
    keep = max(1, hist * case["keep"])
    # each weight once, the kept rows out of the old pages and into the new ones, their positions, and all of it again for reading them back
    return {"bytes": B * H * (hist * 4 + keep * (4 * row4 + 8) + keep * (2 * row4 + 4 * DIM)), "flops": B * H * (hist * 4 + keep * DIM * 4)}


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
    """All rows of (request, kv head) in position order, in 64 bits."""
    ps, T, he = case["page"], int(s["T"][b]), int(s["he"][b])
    p = torch.arange(T, device=DEV)
    rows = torch.zeros((T, DIM), dtype=torch.float64, device=DEV)
    far = (p >= SINK) & (p < he)
    pf, pn = p[far], p[~far]
    if len(pf):
        pg = s["t4"][b, pf // ps].long()
        rows[far] = _rows64(s["cv" if kind else "ck"][pg, h, pf % ps], s["sz"][pg, h, pf % ps], kind, case["group"])
    rows[~far] = s["bv" if kind else "bk"][s["tb"][b, pn // ps].long(), pn % ps, h].double()
    return rows


def exact(case, seed):
    s = prepare(case, seed)
    H, G, ps, B = case["n_kv"], case["gqa"], case["page"], case["batch"]
    op, f64 = case["op"], torch.float64
    if op == "append":
        n, rot = s["valid"], case["rot"]
        x = s["qkv"].double().view(-1, (G + 2) * H, DIM)
        y = x.clone()
        for lo, hi, w in ((0, G * H, s["wq"]), (G * H, G * H + H, s["wk"])):
            z = x[:, lo:hi]
            z = z / torch.sqrt(z.square().sum(-1, keepdim=True) / DIM + EPS) * w.double()
            c, i = torch.arange(rot // 2, device=DEV), s["pos"].clamp(min=0).long()
            first, second = (2 * c, 2 * c + 1) if case["pairs"] else (c, c + rot // 2)
            turn = torch.complex(s["rope"][i][:, :rot // 2].double(), s["rope"][i][:, DIM // 2:DIM // 2 + rot // 2].double())
            r = torch.complex(z[..., first].contiguous(), z[..., second].contiguous()) * turn[:, None]
            z[..., first], z[..., second] = r.real, r.imag
            y[:, lo:hi] = z
        q, k, v = s["q_out"].double(), s["k"].double(), s["v"].double()
        q[:n] = y[:n, :G * H]
        page, slot = s["table"][s["req"][:n].long(), s["pos"][:n].long() // ps].long(), s["pos"][:n].long() % ps
        k[page, slot], v[page, slot] = y[:n, G * H:G * H + H], y[:n, G * H + H:]
        return q, k, v
    if op == "demote":
        got = []
        for src, dst in ((s["bk"], s["ok"]), (s["bv"], s["ov"])):
            out = dst.double()
            for b in range(B):
                p = torch.arange(int(s["begin"][b]), int(s["end"][b]), device=DEV)
                x = src[s["tb"][b, p // ps].long(), p % ps].double().view(len(p), H, -1, case["group"])
                least, most = x.min(-1)[0], x.max(-1)[0]
                zero, scale = least.to(torch.bfloat16).double(), ((most - least) / 15).to(torch.bfloat16).double()
                steps = torch.round((x - zero[..., None]) / scale[..., None]).clamp(0, 15)
                x = torch.where(scale[..., None] > 0, zero[..., None] + steps * scale[..., None], zero[..., None])
                out[s["to"][b, p // ps].long(), p % ps] = x.view(len(p), H, DIM)
            got.append(out)
        return tuple(got)
    if op in ("decode", "mass"):
        out, lse = torch.empty((B, H * G, DIM), dtype=f64, device=DEV), torch.empty((B, H * G), dtype=f64, device=DEV)
        mass = s["mass"].double() if op == "mass" else None
        for b in range(B):
            for h in range(H):
                z = s["q"][b, h * G:(h + 1) * G].double() @ _cache64(case, s, b, h, 0).T * s["sm_scale"]
                if op == "mass":
                    mass[b, h, :z.shape[1]] += torch.exp(z - s["lse"][b, h * G:(h + 1) * G, None].double()).sum(0)
                    continue
                lse[b, h * G:(h + 1) * G] = torch.logsumexp(z, 1)
                out[b, h * G:(h + 1) * G] = torch.softmax(z, 1) @ _cache64(case, s, b, h, 1)
        return mass if op == "mass" else (out, lse)
    kept, mass, k, v = s["kept"].clone(), torch.zeros_like(s["mass_out"]).double(), s["ok"].double(), s["ov"].double()
    for b in range(B):
        T, he, n = int(s["T"][b]), int(s["he"][b]), int(s["keep"][b])
        to, at = s["to"][b, torch.arange(SINK, SINK + n, device=DEV) // ps].long(), torch.arange(SINK, SINK + n, device=DEV) % ps
        for h in range(H):
            m = s["mass"][b, h].cpu().numpy()
            pick = np.sort(np.lexsort((np.arange(SINK, he), -m[SINK:he]))[:n]) + SINK
            p = _put(pick)
            kept[b, h, :n] = p.int()
            mass[b, h, :T - he + SINK + n] = torch.cat([s["mass"][b, h, :SINK], s["mass"][b, h, p], s["mass"][b, h, he:T]]).double()
            page = s["t4"][b, p // ps].long()
            k[to, at, h] = _rows64(s["ck"][page, h, p % ps], s["sz"][page, h, p % ps], 0, case["group"])
            v[to, at, h] = _rows64(s["cv"][page, h, p % ps], s["sz"][page, h, p % ps], 1, case["group"])
    return kept, mass, k, v
