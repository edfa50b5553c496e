"""Cases of the paged-cache operators for drafted tokens, and their plain forms.

A sequence i holds ``ctx`` tokens in the paged cache; its drafted tokens (a
tree, given by each token's parent) follow at positions ctx, ctx + 1, ...
The five operators are the ShortConv K/V step of a drafted tree, the tree's
attention over the cache, the accumulation of attention weights per cache
row, the eviction of the rows with the least weight, and the acceptance of
one path of the tree.

With ``own`` false ``run`` computes them from elementary torch operations in
32 bits; with ``own`` true it calls ``short_conv_kv_b200.binding``.
"""
import math
import random

import torch

own = False

EPS = 1e-6
MX_BLOCK = 32


# ------------------------------------------------------------------- cases

def _case(name, op, **kw):
    c = dict(op=op, seqs=1, ctx_lo=1, ctx_hi=1, n_lo=1, n_hi=1, heads_q=64, heads_kv=8, dim=128,
             page=64, mx=False, width=4, keep=0, sinks=4, recent=64, chain=False)
    c.update(kw)
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # one user, one new token over an 8192-token context: the plain decode read, where latency counts
        _case("attend_one", "attend", seqs=1, ctx_lo=8192, ctx_hi=8192, chain=True),
        # a batch of ragged contexts, each with a small ragged tree: ordinary speculative serving
        _case("attend_batch", "attend", seqs=32, ctx_lo=512, ctx_hi=8192, n_lo=2, n_hi=16, heads_q=32),
        # the 1M-token context of the chunked prefill, four drafted tokens: the cache read bounds it
        _case("attend_long", "attend", seqs=1, ctx_lo=1048573, ctx_hi=1048573, n_lo=4, n_hi=4),
        # wide trees over an MXFP8 cache: products and exponentials bound it
        _case("attend_wide_mx", "attend", seqs=8, ctx_lo=12000, ctx_hi=20000, n_lo=48, n_hi=64, mx=True),
        # weights of one decode step of a serving batch, kept for a later eviction
        _case("weigh_batch", "weigh", seqs=64, ctx_lo=1024, ctx_hi=4096, chain=True, heads_q=32),
        # a long MXFP8 context weighed by the last tokens of a prompt
        _case("weigh_long_mx", "weigh", seqs=1, ctx_lo=262139, ctx_hi=262139, n_lo=8, n_hi=8, mx=True, chain=True),
        # the K/V step of one user's small tree: latency
        _case("step_one", "step", seqs=1, ctx_lo=900, ctx_hi=900, n_lo=8, n_hi=8),
        # a serving batch's trees into an MXFP8 cache
        _case("step_batch_mx", "step", seqs=256, ctx_lo=10, ctx_hi=190, n_lo=24, n_hi=40, mx=True),
        # pruning a batch of contexts to half of the longest
        _case("evict_batch", "evict", seqs=16, ctx_lo=3000, ctx_hi=8192, keep=4096),
        # pruning one long MXFP8 context to a quarter
        _case("evict_long_mx", "evict", seqs=1, ctx_lo=131071, ctx_hi=131071, keep=32768, recent=1024, mx=True),
        # one user's accepted path: latency
        _case("accept_one", "accept", seqs=1, ctx_lo=900, ctx_hi=900, n_lo=8, n_hi=8),
        # a serving batch's accepted paths
        _case("accept_batch", "accept", seqs=512, ctx_lo=1, ctx_hi=190, n_lo=1, n_hi=24),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "weigh", "step", "evict", "accept"])
    dim = rng.choice([64, 128, 128, 128, 256])
    heads_kv = rng.choice([1, 2, 4, 8, 8])
    group = rng.choice([1, 2, 3, 4, 5, 8, 8, 16])
    mx = rng.random() < 0.4
    page = rng.choice([16, 48, 64, 64, 100, 128])
    c = dict(dim=dim, heads_kv=heads_kv, heads_q=heads_kv * group, mx=mx, page=page, chain=rng.random() < 0.3,
             width=rng.choice([1, 2, 3, 4, 4, 8]))
    if op in ("attend", "weigh"):
        c["n_hi"] = _log_int(rng, 1, 128)
        c["n_lo"] = rng.randint(1, c["n_hi"])
        # cached values in all, and query-by-key products, within the largest listed case
        rows = _log_int(rng, 1, (1 << 28) // (dim * heads_kv))
        rows = max(1, min(rows, (1 << 34) // (dim * heads_kv * group * c["n_hi"])))
        c["seqs"] = _log_int(rng, 1, min(128, rows))
        c["ctx_hi"] = max(1, rows // c["seqs"])
        c["ctx_lo"] = rng.randint(1, c["ctx_hi"])
    elif op == "evict":
        rows = _log_int(rng, 64, 1 << 17)
        c["seqs"] = _log_int(rng, 1, min(64, rows // 32))
        c["ctx_hi"] = max(8, rows // c["seqs"])
        c["ctx_lo"] = rng.randint(1, c["ctx_hi"])
        c["keep"] = rng.randint(max(1, c["ctx_hi"] // 8), c["ctx_hi"])
        c["sinks"] = rng.randint(0, min(4, c["keep"]))
        c["recent"] = rng.randint(0, (c["keep"] - c["sinks"]) // 2)
    else:
        c["n_hi"] = _log_int(rng, 1, 64)
        c["n_lo"] = rng.randint(1, c["n_hi"])
        c["seqs"] = _log_int(rng, 1, max(1, min(512, (1 << 24) // (c["n_hi"] * dim * heads_kv))))
        c["ctx_hi"] = _log_int(rng, 1, 500)
        c["ctx_lo"] = rng.randint(1, c["ctx_hi"])
    return _case(None, op, **c)


# ------------------------------------------------------------------ inputs

def _lens(case, seed):
    """Host-side lengths of the case: (contexts, drafted counts).  The case fixes the set of
    sequences, so that every seed's buffers have one size; the seed orders them."""
    rng = random.Random(case["seqs"] * 1000003 + case["ctx_hi"] * 1009 + case["n_hi"])
    both = []
    for _ in range(case["seqs"]):
        n = rng.randint(case["n_lo"], case["n_hi"])
        both.append((rng.randint(case["ctx_lo"], case["ctx_hi"]), 0 if case["op"] == "evict" else n))
    random.Random(seed * 7919 + 17).shuffle(both)
    return [c for c, _ in both], [n for _, n in both]


def _tree(rng, n, chain):
    """Parents of n drafted tokens: a chain, or a tree whose nodes hang on recent ones, the last
    tokens of a larger one unused padding."""
    if chain:
        return [j - 1 for j in range(n)]
    pad = rng.randint(0, n // 8)
    used = n - pad
    par = [-1] + [rng.randint(max(-1, j - 6), j - 1) for j in range(1, used)]
    return par + [-2] * pad


def _quantise(z):
    """MXFP8 codes (uint8) and E8M0 scale bytes of z [..., D], blocks of 32: shared exponent
    floor(log2 amax) - 8, codes rounded to nearest even and saturated."""
    b = z.unflatten(-1, (-1, MX_BLOCK))
    amax = b.abs().amax(-1, keepdim=True)
    e = torch.frexp(amax)[1] - 9
    e = torch.where(amax < 2.0 ** -126, torch.full_like(e, -127), e.clamp(-127, 127))
    u = (b * torch.exp2(-e.to(z.dtype))).clamp(-448, 448)
    codes = u.float().to(torch.float8_e4m3fn).view(torch.uint8).flatten(-2)
    return codes, (e.squeeze(-1) + 127).to(torch.uint8)


def prepare(case, seed):
    ctx, n = _lens(case, seed)
    rng = random.Random(seed * 104729 + 3)
    dev = torch.device("cuda")
    gen = torch.Generator(device=dev).manual_seed(seed)
    S, H, D, P, W = case["seqs"], case["heads_kv"], case["dim"], case["page"], case["width"]
    HQ, C = case["heads_q"], case["heads_kv"] * case["dim"]
    op = case["op"]
    bf = torch.bfloat16

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=dev, dtype=torch.float32)

    pages = [-(-max(1, c + m) // P) for c, m in zip(ctx, n)]
    wide, total_pages = max(pages), sum(pages)
    perm = torch.randperm(total_pages, generator=gen, device=dev).to(torch.int32)
    at = torch.tensor([0] + pages, dtype=torch.int64).cumsum(0)[:-1]
    col = torch.arange(wide)
    idx = at[:, None] + torch.minimum(col[None], torch.tensor(pages)[:, None] - 1)
    table = perm[idx.to(dev)].contiguous()
    cu = torch.tensor([0] + n, dtype=torch.int64).cumsum(0)
    T = int(cu[-1])
    parents = [p for m in n for p in _tree(rng, m, case["chain"])]
    s = dict(case=case, ctx=ctx, n=n, lmax=max(ctx), nmax=max(n), tmax=max(c + m for c, m in zip(ctx, n)),
             table=table, cu=cu.to(torch.int32).to(dev), lens=torch.tensor(ctx, dtype=torch.int32, device=dev),
             parents=torch.tensor(parents, dtype=torch.int32, device=dev), scale=D ** -0.5)

    # the cache: K and V halves of one buffer per page, filled with normalised rows
    shape = (total_pages, 2, P, H, D)
    if case["mx"]:
        codes = torch.empty(shape, dtype=torch.uint8, device=dev)
        scales = torch.empty(shape[:-1] + (D // MX_BLOCK,), dtype=torch.uint8, device=dev)
        step = max(1, (1 << 26) // (2 * P * C))
        for a in range(0, total_pages, step):
            m = min(step, total_pages - a)
            codes[a:a + m], scales[a:a + m] = _quantise(randn(m, *shape[1:]))
        s.update(kd=codes[:, 0], vd=codes[:, 1], ks=scales[:, 0], vs=scales[:, 1])
    else:
        kv = torch.empty(shape, dtype=bf, device=dev)
        step = max(1, (1 << 27) // (2 * P * C))
        for a in range(0, total_pages, step):
            m = min(step, total_pages - a)
            kv[a:a + m] = randn(m, *shape[1:])
        s.update(kc=kv[:, 0], vc=kv[:, 1])
    if op in ("attend", "weigh"):
        s["q"] = (1.5 * randn(T, HQ, D)).to(bf)
    if op == "attend":
        s["out"] = torch.empty(T, HQ, D, dtype=bf, device=dev)
        s["lse"] = torch.empty(T, HQ, dtype=torch.float32, device=dev)
    if op == "weigh":
        # ln of the sum over about ctx + n keys of exp(N(0, 1.5)), as the attention left it
        full = torch.tensor([c + m for c, m in zip(ctx, n) for _ in range(m)], dtype=torch.float32, device=dev)
        s["lse"] = (full.log() + 1.125)[:, None] + 0.05 * randn(T, HQ)
    if op in ("weigh", "evict", "accept"):
        # accumulated weights: heavy-tailed, many small ones equal
        u = torch.rand(S, H, s["tmax"] + 3, generator=gen, device=dev)
        s["weights"] = ((-torch.log(u + 1e-7)) ** 3 * 64).floor() / 1024
    if op in ("step", "accept"):
        qkv = randn(T, 2 * C + 64).to(bf)  # k and v as column slices of a projection's output
        s["k"], s["v"] = qkv[:, :C], qkv[:, C:2 * C]
        s["state"] = randn(S, max(W - 1, 0), 2 * C).to(bf)
        s["state_rows"] = torch.randperm(S, generator=gen, device=dev).to(torch.int32)
    if op == "step":
        s["wk"], s["wv"] = (randn(W, C) * W ** -0.5).to(bf), (randn(W, C) * W ** -0.5).to(bf)
        s["gk"], s["gv"] = 1 + 0.1 * randn(D), 1 + 0.1 * randn(D)
        pos = torch.cat([torch.arange(c, c + m) for c, m in zip(ctx, n)])
        seq = torch.repeat_interleave(torch.arange(S), torch.tensor(n))
        tc = table.cpu().long()
        slot = tc[seq, pos // P] * P + pos % P
        slot[torch.tensor(parents) < -1] = -1
        s["slots"] = slot.to(dev)
    if op == "accept":
        leaves = []
        for c, m, a in zip(ctx, n, cu.tolist()):
            par = parents[a:a + m]
            used = [j for j in range(m) if par[j] > -2]
            leaves.append(rng.choice([-1] + used[len(used) // 2:]) if rng.random() < 0.2 else used[-1])
        s["leaves"] = torch.tensor(leaves, dtype=torch.int32, device=dev)
    if op in ("evict", "accept"):
        s["new_lens"] = torch.empty(S, dtype=torch.int32, device=dev)
    if op == "evict":
        s["kept"] = torch.empty(S, H, case["keep"], dtype=torch.int32, device=dev)
        s["weights_out"] = torch.zeros_like(s["weights"])
    return s


# ------------------------------------------------------------- plain forms

def _value(s, which, page, off):
    """Cache rows as 32-bit numbers, at index tensors (page, off): [..., H, D]."""
    if "kc" in s:
        return s[which + "c"][page, off].float()
    codes = s[which + "d"][page, off].view(torch.float8_e4m3fn).float()
    scale = torch.exp2(s[which + "s"][page, off].float() - 127)
    return (codes.unflatten(-1, (-1, MX_BLOCK)) * scale[..., None]).flatten(-2)


def _place(s, pos):
    """(page, offset) of positions pos [S, ...]."""
    P = s["case"]["page"]
    page = s["table"].long().gather(1, (pos // P).flatten(1)).view(pos.shape)
    return page, pos % P


def _square(a):
    return ((a @ a) > 0).float()


def _padded(s):
    """Drafted tokens as [S, n] (n the largest count): packed index, who is there, parent."""
    cu, n = s["cu"].long(), s["nmax"]
    j = torch.arange(n, device=cu.device)
    count = cu[1:] - cu[:-1]
    there = j[None] < count[:, None]
    idx = cu[:-1, None] + torch.minimum(j[None], count[:, None] - 1)
    par = torch.where(there, s["parents"].long()[idx], -2)
    return idx, there, par


def _ancestors(par):
    """[S, n, n]: whether a is j or an ancestor of j (j used)."""
    n = par.shape[1]
    used = par > -2
    eye = torch.eye(n, device=par.device)
    up = (par[..., None] == torch.arange(n, device=par.device)).float() + eye
    a = _square(_square(_square(_square(_square(_square(_square(up)))))))
    return (a > 0) & used[..., None] & used[:, None, :]


def _seen(s):
    """Positions [L], whether drafted token j of sequence i sees position p [S, n, L], and the
    position's place in the cache."""
    idx, there, par = _padded(s)
    anc = _ancestors(par)
    ctx = s["lens"].long()
    p = torch.arange(s["tmax"], device=ctx.device)
    rel = p[None] - ctx[:, None]
    n = par.shape[1]
    own_part = anc.gather(2, rel.clamp(0, n - 1)[:, None].expand(-1, n, -1)) & ((rel >= 0) & (rel < n))[:, None]
    vis = (own_part | (rel < 0)[:, None]) & (par > -2)[..., None]
    last = ctx + (s["cu"][1:] - s["cu"][:-1]).long() - 1
    page, off = _place(s, torch.minimum(p[None], last[:, None]))
    return idx, there, vis, page, off


def _logits(s, idx, page, off):
    H, D = s["case"]["heads_kv"], s["case"]["dim"]
    q = s["q"][idx].float().unflatten(2, (H, -1))  # [S, n, H, g, D]
    q = q.permute(0, 2, 3, 1, 4).flatten(2, 3)  # [S, H, g*n, D]
    k = _value(s, "k", page, off).transpose(1, 2)  # [S, H, L, D]
    return (q @ k.transpose(2, 3)) * s["scale"]


def _attend(s):
    idx, there, vis, page, off = _seen(s)
    H, D = s["case"]["heads_kv"], s["case"]["dim"]
    S, n, L = vis.shape
    x = _logits(s, idx, page, off).view(S, H, -1, n, L)
    x = x.masked_fill_(~vis[:, None, None], -math.inf)
    m = x.amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = x.sub_(m).exp_()
    den = p.sum(-1, keepdim=True)
    v = _value(s, "v", page, off).transpose(1, 2)
    v = torch.where(vis.any(1)[:, None, :, None], v, torch.zeros_like(v))
    o = (p.flatten(2, 3) @ v).view(S, H, -1, n, D)
    o = torch.where(den > 0, o / den, torch.zeros_like(o))
    lse = (m + den.log()).squeeze(-1)
    T = s["q"].shape[0]
    flat = _flat_index(s, T)
    o = o.permute(0, 3, 1, 2, 4).flatten(0, 1).flatten(1, 2)[flat]
    lse = lse.permute(0, 3, 1, 2).flatten(0, 1).flatten(1, 2)[flat]
    return {"out": o.to(torch.bfloat16), "lse": lse}


def _flat_index(s, T):
    """Where each packed token is in the padded [S * n]."""
    cu = s["cu"].long()
    t = torch.arange(T, device=cu.device)
    seq = torch.searchsorted(cu, t, right=True) - 1
    return seq * s["nmax"] + t - cu[seq]


def _weigh(s):
    idx, there, vis, page, off = _seen(s)
    H = s["case"]["heads_kv"]
    S, n, L = vis.shape
    x = _logits(s, idx, page, off).view(S, H, -1, n, L)
    lse = s["lse"][idx].unflatten(2, (H, -1)).permute(0, 2, 3, 1)  # [S, H, g, n]
    p = torch.where(vis[:, None, None], (x - lse[..., None]).exp(), torch.zeros_like(x))
    add = p.sum((2, 3))  # [S, H, L]
    rel = torch.arange(L, device=add.device)[None] - s["lens"].long()[:, None]
    count = (s["cu"][1:] - s["cu"][:-1]).long()
    w = s["weights"]
    old = w[..., :L]
    new = torch.where((rel < 0)[:, None], old + add, torch.where((rel < count[:, None])[:, None], add, old))
    w[..., :L] = new
    return {"weights": w}


def _step(s):
    case = s["case"]
    W, H, D, P = case["width"], case["heads_kv"], case["dim"], case["page"]
    idx, there, par = _padded(s)
    S, n = par.shape
    anc = _ancestors(par)
    depth = anc.sum(2) - 1  # 0: a child of the context
    dev = par.device
    back = torch.arange(W - 1, -1, -1, device=dev)  # distance of tap 0 .. W-1
    want = depth[..., None] - back  # [S, n, W]: the depth of the ancestor that the tap meets
    hit = anc[:, :, None, :] & (depth[:, None, None, :] == want[..., None])
    node = hit.float().argmax(-1)
    token = idx.gather(1, node.flatten(1)).view(S, n, W)
    x = torch.cat([s["k"], s["v"]], 1).float()[token]  # [S, n, W, 2C]
    if W > 1:
        rows = s["state"][s["state_rows"].long()].float()
        old = rows[torch.arange(S, device=dev)[:, None, None], (W - 1 + want).clamp(0, W - 2)]
        x = torch.where((want < 0)[..., None], old, x)
    y = (x * torch.cat([s["wk"], s["wv"]], 1).float()).sum(2).view(S, n, 2, H, D)
    gamma = torch.stack([s["gk"], s["gv"]])[:, None]
    z = y / torch.sqrt((y * y).mean(-1, keepdim=True) + EPS) * gamma
    T = s["k"].shape[0]
    # tokens without a slot write their sequence's first token once more
    first = s["cu"].long()[:-1][:, None].expand(S, n)
    use = (par > -2).flatten()
    flat = _flat_index(s, T)
    src = torch.where(use, torch.arange(S * n, device=dev), torch.arange(S, device=dev).repeat_interleave(n) * n)[flat]
    slot = torch.where(use[flat], s["slots"], s["slots"][first.flatten()[flat]])
    z = z.flatten(0, 1)[src]
    page, off = slot // P, slot % P
    if case["mx"]:
        codes, scale = _quantise(z)
        s["kd"][page, off], s["vd"][page, off] = codes[:, 0], codes[:, 1]
        s["ks"][page, off], s["vs"][page, off] = scale[:, 0], scale[:, 1]
    else:
        s["kc"][page, off], s["vc"][page, off] = z[:, 0].to(torch.bfloat16), z[:, 1].to(torch.bfloat16)
    return _caches(s)


def _caches(s):
    """The cache buffers, 8-bit ones as the numbers they stand for."""
    if "kc" in s:
        return {"k": s["kc"], "v": s["vc"]}
    f8, e8 = torch.float8_e4m3fn, torch.float8_e8m0fnu
    return {"k": s["kd"].view(f8), "v": s["vd"].view(f8), "k_scale": s["ks"].view(e8), "v_scale": s["vs"].view(e8)}


def _parts(s):
    return ("kc", "vc") if "kc" in s else ("kd", "vd", "ks", "vs")


def _move(s, part, to, frm, head=None):
    """Rows of one cache part from positions frm to positions to (read whole before written)."""
    (pf, of), (pt, ot) = _place(s, frm), _place(s, to)
    if head is None:
        s[part][pt, ot] = s[part][pf, of]
    else:
        s[part][pt, ot, head] = s[part][pf, of, head]


def _accept(s):
    case = s["case"]
    W, S, n = case["width"], case["seqs"], s["nmax"]
    idx, there, par = _padded(s)
    dev = par.device
    leaf = s["leaves"].long()
    on = _ancestors(par).gather(1, leaf.clamp(min=0)[:, None, None].expand(-1, 1, n)).squeeze(1) & (leaf >= 0)[:, None]
    m = on.sum(1)
    j = torch.arange(n, device=dev)
    order = torch.where(on, j, j + n).argsort(1)  # the path first, in order
    src = torch.where(j < m[:, None], order, j.expand(S, n))
    count = (s["cu"][1:] - s["cu"][:-1]).long()
    j2 = torch.minimum(j[None], count[:, None] - 1)
    src = src.gather(1, j2)
    ctx = s["lens"].long()[:, None]
    to, frm = ctx + j2, ctx + src
    for part in _parts(s):
        _move(s, part, to, frm)
    w = s["weights"]
    seq = torch.arange(S, device=dev)[:, None]
    w[seq, :, to] = w[seq, :, frm]
    if W > 1:
        rows = s["state_rows"].long()
        x = torch.cat([s["k"], s["v"]], 1)
        both = torch.cat([s["state"][rows], x[idx.gather(1, src)]], 1)
        s["state"][rows] = both[seq, m[:, None] + torch.arange(W - 1, device=dev)]
    s["new_lens"] = (s["lens"] + m).to(torch.int32)
    return {**_caches(s), "weights": w, "state": s["state"], "new_lens": s["new_lens"]}


def _evict(s):
    case = s["case"]
    S, H, K, sinks, recent = case["seqs"], case["heads_kv"], case["keep"], case["sinks"], case["recent"]
    w = s["weights"][..., :s["lmax"]]
    dev = w.device
    L = w.shape[2]
    ctx = s["lens"].long()
    p = torch.arange(L, device=dev)
    held = (p[None] < sinks) | (p[None] >= ctx[:, None] - recent)
    key = torch.where(held[:, None], torch.full_like(w, math.inf), w)
    key = torch.where((p[None] >= ctx[:, None])[:, None], torch.full_like(w, -math.inf), key)
    order = key.sort(dim=-1, descending=True, stable=True)[1]
    K2 = min(K, L)
    best = order[..., :K2].sort(dim=-1)[0]
    slot = torch.arange(K2, device=dev)
    small = (ctx <= K)[:, None, None]
    best = torch.where(small, torch.where(slot < ctx[:, None, None], slot, -1), best)
    s["kept"].fill_(-1)
    s["kept"][..., :K2] = best
    new = ctx.clamp(max=K)
    to = torch.minimum(slot.expand(S, K2), new[:, None] - 1)[:, None].expand(S, H, K2)
    frm = best.gather(2, to)
    head = torch.arange(H, device=dev)[None, :, None]
    for part in _parts(s):
        _move(s, part, to, frm, head)
    s["weights_out"].scatter_(2, to, s["weights"].gather(2, frm))
    s["new_lens"] = new.to(torch.int32)
    return {**_caches(s), "kept": s["kept"], "weights": s["weights_out"], "new_lens": s["new_lens"]}


# --------------------------------------------------------- the framework's

def _own(s):
    from short_conv_kv_b200 import binding as b

    case = s["case"]
    op, mx = case["op"], case["mx"]
    kv = (s["kd"], s["ks"], s["vd"], s["vs"]) if mx else (s["kc"], s["vc"])
    if op == "attend":
        if "workspace" not in s:
            s["workspace"] = b.tree_attention_workspace(s["q"], kv[0], s["lens"].shape[0], s["nmax"])
        call = b.tree_attention_mxfp8 if mx else b.tree_attention
        call(s["q"], s["cu"], s["parents"], s["lens"], s["table"], *kv, s["scale"], s["nmax"], s["out"],
             s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    if op == "weigh":
        call = b.attention_weights_mxfp8 if mx else b.attention_weights
        call(s["q"], s["lse"], s["cu"], s["parents"], s["lens"], s["table"], *kv[:2 if mx else 1], s["scale"],
             s["nmax"], s["weights"])
        return {"weights": s["weights"]}
    if op == "step":
        call = b.tree_step_mxfp8 if mx else b.tree_step
        call(s["k"], s["v"], s["cu"], s["parents"], s["wk"], s["wv"], s["gk"], s["gv"], EPS, s["state"],
             s["slots"], *kv, state_indices=s["state_rows"])
        return _caches(s)
    if op == "accept":
        call = b.tree_accept_mxfp8 if mx else b.tree_accept
        call(s["k"], s["v"], s["cu"], s["parents"], s["leaves"], s["lens"], s["table"], case["width"], s["state"],
             *kv, s["new_lens"], weights=s["weights"], state_indices=s["state_rows"])
        return {**_caches(s), "weights": s["weights"], "state": s["state"], "new_lens": s["new_lens"]}
    call = b.evict_mxfp8 if mx else b.evict
    call(s["weights"], s["lens"], s["table"], *kv, case["sinks"], case["recent"], s["kept"], s["new_lens"],
         s["weights_out"])
    return {**_caches(s), "kept": s["kept"], "weights": s["weights_out"], "new_lens": s["new_lens"]}


def run(s):
    if own:
        return _own(s)
    return {"attend": _attend, "weigh": _weigh, "step": _step, "evict": _evict, "accept": _accept}[s["case"]["op"]](s)


# ------------------------------------------------------------ work of a pass

def work(case):
    # mean lengths of the case's ranges
    S, H, D, HQ, W = case["seqs"], case["heads_kv"], case["dim"], case["heads_q"], case["width"]
    ctx, n = (case["ctx_lo"] + case["ctx_hi"]) / 2, (case["n_lo"] + case["n_hi"]) / 2
    row = H * D * (1 + 1 / MX_BLOCK if case["mx"] else 2)  # one position of K (or of V)
    op = case["op"]
    if op == "attend":
        return {"bytes": S * ((ctx + n) * 2 * row + n * HQ * (D * 4 + 4)), "flops": S * n * (ctx + n) * HQ * D * 4}
    if op == "weigh":
        return {"bytes": S * ((ctx + n) * (row + 8 * H) + n * HQ * (D * 2 + 4)), "flops": S * n * (ctx + n) * HQ * D * 2}
    if op == "step":
        return {"bytes": S * (n * (H * D * 4 + 2 * row) + (W - 1) * H * D * 4), "flops": S * n * 2 * H * D * (2 * W + 4)}
    if op == "accept":
        return {"bytes": S * (n / 4 * 4 * row + 2 * (W - 1) * H * D * 4), "flops": S * n}
    moved = max(0, min(case["keep"], ctx))
    return {"bytes": S * (ctx * H * 4 + moved * 4 * row + moved * H * 12), "flops": S * H * ctx}


# ------------------------------------------------- from the definition, in 64 bits

def _rows64(s, which, i, count):
    """Positions 0 .. count-1 of sequence i as 64-bit numbers [count, H, D]."""
    P = s["case"]["page"]
    tab = s["table"][i].long()
    out = []
    for a in range(0, count, P):
        m = min(P, count - a)
        pg = tab[a // P]
        if "kc" in s:
            out.append(s[which + "c"][pg, :m].double())
        else:
            v = s[which + "d"][pg, :m].view(torch.float8_e4m3fn).double()
            e = s[which + "s"][pg, :m].double() - 127
            out.append(v * torch.repeat_interleave(torch.pow(2.0, e), MX_BLOCK, dim=-1))
    return torch.cat(out)


def _paths(par):
    """Each token's list of ancestors, root first, itself last; [] for an unused one."""
    path = []
    for j, p in enumerate(par):
        path.append([] if p < -1 else ([] if p < 0 else path[p]) + [j])
    return path


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    H, D, HQ, W = case["heads_kv"], case["dim"], case["heads_q"], case["width"]
    g = HQ // H
    cu, parents = s["cu"].tolist(), s["parents"].tolist()
    if op == "attend" or op == "weigh":
        if op == "attend":
            out = torch.zeros(cu[-1], HQ, D, dtype=torch.float64, device="cuda")
            lse = torch.full((cu[-1], HQ), -math.inf, dtype=torch.float64, device="cuda")
        else:
            weights = s["weights"].double()
        for i, (c, n) in enumerate(zip(s["ctx"], s["n"])):
            k = _rows64(s, "k", i, c + n)
            v = _rows64(s, "v", i, c + n) if op == "attend" else None
            path = _paths(parents[cu[i]:cu[i + 1]])
            hide = torch.ones(n, n, dtype=torch.bool)
            for j, a in enumerate(path):
                hide[j, a] = False
            hide = hide.cuda()
            dead = [j for j, a in enumerate(path) if not a]
            add = torch.zeros(H, c + n, dtype=torch.float64, device="cuda")
            for h in range(H):
                q = s["q"][cu[i]:cu[i + 1], h * g:(h + 1) * g].double()  # [n, g, D]
                x = torch.einsum("jgd,pd->jgp", q, k[:, h]) * D ** -0.5
                x[:, :, c:].masked_fill_(hide[:, None], -math.inf)
                x[dead] = -math.inf
                at = slice(cu[i], cu[i + 1])
                if op == "weigh":
                    add[h] = torch.exp(x - s["lse"][at, h * g:(h + 1) * g].double()[..., None]).sum((0, 1))
                    continue
                l = torch.logsumexp(x, -1)
                x -= torch.where(l.isinf(), torch.zeros_like(l), l)[..., None]
                lse[at, h * g:(h + 1) * g] = l
                out[at, h * g:(h + 1) * g] = torch.einsum("jgp,pd->jgd", x.exp_(), v[:, h])
            if op == "weigh":
                weights[i, :, :c] += add[:, :c]
                weights[i, :, c:c + n] = add[:, c:]
        return {"out": out, "lse": lse} if op == "attend" else {"weights": weights}
    if op == "step":
        x = torch.cat([s["k"], s["v"]], 1).double()
        taps = torch.cat([s["wk"], s["wv"]], 1).double()
        gamma = torch.stack([s["gk"], s["gv"]]).double()[:, None]
        tokens, window = [], []
        state = s["state"].double()
        pool = torch.cat([x, state.flatten(0, 1)]) if W > 1 else x
        rows = s["state_rows"].tolist()
        for i in range(case["seqs"]):
            for j, a in enumerate(_paths(parents[cu[i]:cu[i + 1]])):
                if a:
                    line = [cu[-1] + rows[i] * (W - 1) + r for r in range(W - 1)] + [cu[i] + t for t in a]
                    tokens.append(cu[i] + j)
                    window.append(line[-W:])
        z = torch.empty(len(tokens), 2, H, D, dtype=torch.float64, device="cuda")
        for a in range(0, len(tokens), 1024):
            y = (pool[torch.tensor(window[a:a + 1024], device="cuda")] * taps).sum(1).view(-1, 2, H, D)
            z[a:a + 1024] = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * gamma
        slot = s["slots"][torch.tensor(tokens, device="cuda")]
        got = {a: b.double() for a, b in _caches(s).items()}
        page, off = slot // case["page"], slot % case["page"]
        if case["mx"]:
            # codes as the unrounded values, in units of the block's scale
            blocks = z.unflatten(-1, (-1, MX_BLOCK))
            e = (torch.floor(torch.log2(blocks.abs().amax(-1))) - 8).clamp(-127, 127)
            u = (blocks / torch.pow(2.0, e)[..., None]).clamp(-448, 448).flatten(-2)
            for q, name in enumerate("kv"):
                got[name][page, off] = u[:, q]
                got[name + "_scale"][page, off] = torch.pow(2.0, e[:, q])
        else:
            got["k"][page, off], got["v"][page, off] = z[:, 0], z[:, 1]
        return got
    P = case["page"]
    got = {a: b.clone() for a, b in _caches(s).items()}
    table = s["table"].tolist()
    lens = []
    if op == "accept":
        old, w, state = {a: b.clone() for a, b in got.items()}, s["weights"].double(), s["state"].clone()
        w0 = w.clone()
        x = torch.cat([s["k"], s["v"]], 1)
        rows, leaves = s["state_rows"].tolist(), s["leaves"].tolist()
        at = [[], [], [], []]
        wi = [[], [], []]
        for i, c in enumerate(s["ctx"]):
            a = _paths(parents[cu[i]:cu[i + 1]])[leaves[i]] if leaves[i] >= 0 else []
            lens.append(c + len(a))
            for r, j in enumerate(a):
                for v, b in zip(at, (table[i][(c + r) // P], (c + r) % P, table[i][(c + j) // P], (c + j) % P)):
                    v.append(b)
                for v, b in zip(wi, (i, c + r, c + j)):
                    v.append(b)
            if W > 1:
                state[rows[i]] = torch.cat([state[rows[i]]] + [x[cu[i] + j:cu[i] + j + 1] for j in a])[-(W - 1):]
        tp, to, fp, fo = (torch.tensor(v, dtype=torch.int64, device="cuda") for v in at)
        i, t, f = (torch.tensor(v, dtype=torch.int64, device="cuda") for v in wi)
        for a in got:
            _raw(got[a])[tp, to] = _raw(old[a])[fp, fo]
        w[i, :, t] = w0[i, :, f]
        return {**{a: b.double() for a, b in got.items()}, "weights": w, "state": state.double(),
                "new_lens": torch.tensor(lens, dtype=torch.int32)}
    K, sinks, recent = case["keep"], case["sinks"], case["recent"]
    kept = torch.full((case["seqs"], H, K), -1, dtype=torch.int32, device="cuda")
    wout = s["weights_out"].double()
    for i, c in enumerate(s["ctx"]):
        lens.append(min(c, K))
        tab = torch.tensor(table[i], device="cuda")
        for h in range(H):
            if c <= K:
                pick = torch.arange(c, device="cuda")
            else:
                # rank by (weight downwards, position upwards) among what is not held anyway
                mid = s["weights"][i, h, sinks:c - recent].double().cpu().numpy()
                best = (-mid).argsort(kind="stable")[:K - sinks - recent]
                flag = torch.zeros(c, dtype=torch.bool)
                flag[:sinks] = True
                flag[c - recent:] = True
                flag[sinks + torch.from_numpy(best)] = True
                pick = flag.nonzero().flatten().cuda()
            m = pick.shape[0]
            kept[i, h, :m] = pick
            wout[i, h, :m] = s["weights"][i, h, pick].double()
            d = torch.arange(m, device="cuda")
            for a, b in _caches(s).items():
                _raw(got[a])[tab[d // P], d % P, h] = _raw(b)[tab[pick // P], pick % P, h]
    return {**{a: b.double() for a, b in got.items()}, "kept": None, "weights": wout,
            "new_lens": torch.tensor(lens, dtype=torch.int32)}


def _raw(t):
    """The same storage as plain bytes, where the type is an 8-bit one."""
    return t.view(torch.uint8) if t.element_size() == 1 else t
