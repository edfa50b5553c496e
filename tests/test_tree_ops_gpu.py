"""The drafted-tree step, attention weights, acceptance and eviction against
their definitions, and a serving step of all of them together."""
import numpy as np
import pytest
import torch

import oracle
from oracle import tree as ot
from short_conv_kv_b200 import binding as b
from short_conv_kv_b200 import workloads as wl
from tests import gpu_util as gu
from tests.tree_util import Scene, check_attention, logit_error

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------ attention weights

@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("lens, drafts, H, D, group, page, kind", [
    ([0, 1], [1, 1], 1, 64, 1, 16, "chain"),
    ([100, 16, 15], [1, 2, 3], 2, 128, 4, 64, "padded"),
    ([700], [8], 2, 128, 8, 48, "padded"),
    ([65, 300], [9, 40], 2, 64, 5, 7, "padded"),
    ([130], [128], 1, 128, 3, 64, "tree"),
    ([200, 3], [50, 2], 1, 256, 2, 64, "padded"),
])
def test_weights(lens, drafts, H, D, group, page, kind, mx):
    sc = Scene(lens, drafts, H, D, group, page, mx, kind, seed=21)
    d = sc.device()
    lse = torch.empty(sc.T, sc.HQ, device="cuda")
    sc.attend(d, lse=lse)
    room = max(c + n for c, n in zip(lens, drafts)) + 5
    w0 = torch.rand(sc.S, H, room + 2, device="cuda")
    w = w0.clone()[:, :, 1:-1]
    _weigh(sc, d, lse, w)
    torch.cuda.synchronize()
    assert int(d["err"]) == 0
    with np.errstate(invalid="ignore"):
        want, size = ot.weights(sc.q.double().numpy(), lse.double().cpu().numpy(), sc.cu, sc.parents,
                                lens, sc.table, sc.values(0), sc.scale, w0[:, :, 1:-1].cpu().numpy())
    old = w0[:, :, 1:-1].double().cpu().numpy()
    got = w.double().cpu().numpy()
    # every term's exponent: the score's error, lse * log2(e)'s rounding and the
    # subtraction's (2^-23 |lse| each at most), ex2's 2^-22; then up to 2^9 additions
    e = logit_error(size, D) + 2.0 ** -22 * (2 + np.abs(lse[lse > -1e30].cpu().numpy()).max()) + 2.0 ** -15
    bound = e * np.abs(want - old) + e * np.abs(want) * (want != old) + 2.0 ** -23 * np.abs(want)
    assert (np.abs(got - want) <= bound).all(), (np.abs(got - want) / bound).max()
    for i, (c, n) in enumerate(zip(lens, drafts)):
        assert np.array_equal(got[i, :, c + n:], old[i, :, c + n:])


def _weigh(sc, d, lse, w):
    if sc.mx:
        b.attention_weights_mxfp8(d["q"], lse, d["cu"], d["parents"], d["lens"], d["table"],
                                  *d["kv"][:2], sc.scale, sc.max_draft, w, d["err"])
    else:
        b.attention_weights(d["q"], lse, d["cu"], d["parents"], d["lens"], d["table"], d["kv"][0],
                            sc.scale, sc.max_draft, w, d["err"])


def test_weights_row_too_short_is_flagged():
    sc = Scene([100, 20], [2, 2], 2, 64, 2, 16, kind="chain", seed=22)
    d = sc.device()
    lse = torch.empty(sc.T, sc.HQ, device="cuda")
    sc.attend(d, lse=lse)
    store = torch.zeros(2, 2, 60, device="cuda")
    _weigh(sc, d, lse, store[:, :, :40])
    assert int(d["err"]) == b.FLAG_CONTEXT
    assert (store[0] == 0).all() and (store[1, :, :22] > 0).all() and (store[1, :, 22:] == 0).all()


# ----------------------------------------------------------------------- the step

def _step_inputs(sc, W, pool_extra=2, seed=0, ring=False, per_head=False):
    gen = torch.Generator().manual_seed(seed)
    C = sc.H * sc.D
    rnd = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16)  # noqa: E731
    wide = rnd(sc.T, 2 * C + 8)
    x = dict(k=wide[:, :C], v=wide[:, C:2 * C], wk=rnd(W, C), wv=rnd(W, C),
             gk=1 + 0.1 * torch.randn(*((sc.H,) if per_head else ()), sc.D, generator=gen),
             gv=1 + 0.1 * torch.randn(*((sc.H,) if per_head else ()), sc.D, generator=gen),
             state=rnd(sc.S + pool_extra, max(W - 1, 0), 2 * C),
             rows=torch.randperm(sc.S + pool_extra, generator=gen)[:sc.S].to(torch.int32),
             pos=torch.randint(0, 50, (sc.S,), generator=gen, dtype=torch.int64) if ring else None)
    slots = np.full(sc.T, -1, np.int64)
    for i in range(sc.S):
        for j, path in enumerate(ot.paths(sc.parents[sc.cu[i]:sc.cu[i + 1]])):
            if path:
                pg, off = ot.place(sc.table[i], sc.lens[i] + j, sc.page)
                slots[sc.cu[i] + j] = pg * sc.page + off
    x["slots"] = torch.from_numpy(slots)
    return x


def _linear_state(x, W, i):
    st = x["state"][x["rows"][i]]
    if x["pos"] is not None and W > 1:
        st = st[(int(x["pos"][i]) + np.arange(W - 1)) % (W - 1)]
    return st


def _oracle_step(sc, x, W):
    """z of every used token: decoded on its own from the rows its window holds."""
    C = sc.H * sc.D
    win = ot.windows(sc.cu, sc.parents, W)
    toks = sorted(win)
    raw = torch.cat([x["k"], x["v"]], 1)
    st = np.zeros((len(toks), max(W - 1, 0), 2 * C), np.uint16)
    for r, t in enumerate(toks):
        i, line = win[t]
        own = _linear_state(x, W, i)
        for q, e in enumerate(line[:-1]):
            st[r, q] = wl.bits(raw[e] if e >= 0 else own[W - 1 + e])
    n = len(toks)
    kc = np.zeros((n, 1, sc.H, sc.D), np.uint16)
    out = oracle.decode(wl.bits(x["k"][toks].contiguous()).reshape(n, sc.H, sc.D),
                        wl.bits(x["v"][toks].contiguous()).reshape(n, sc.H, sc.D), wl.bits(x["wk"]), wl.bits(x["wv"]),
                        x["gk"].numpy(), x["gv"].numpy(), 1e-6, st, np.arange(n, dtype=np.int64),
                        kc, kc.copy())
    return toks, out["z_k"], out["z_v"]


def _run_step(sc, d, x):
    dx = {k: None if v is None else v.cuda() for k, v in x.items()}
    wide = torch.cat([x["k"], x["v"]], 1).cuda()
    C = sc.H * sc.D
    fn = b.tree_step_mxfp8 if sc.mx else b.tree_step
    fn(wide[:, :C], wide[:, C:], d["cu"], d["parents"], dx["wk"], dx["wv"], dx["gk"], dx["gv"], 1e-6,
       dx["state"], dx["slots"], *d["kv"], state_indices=dx["rows"], err_flag=d["err"],
       state_positions=dx["pos"])
    torch.cuda.synchronize()
    assert torch.equal(dx["state"].cpu(), x["state"])
    return wide, dx


STEPS = [
    ([0], [1], 1, 64, 16, "chain", 4),
    ([3, 30, 0], [5, 16, 2], 2, 128, 64, "padded", 4),
    ([9, 1], [7, 30], 3, 64, 7, "padded", 2),
    ([20], [128], 1, 256, 48, "tree", 8),
    ([2, 2, 2, 2], [1, 2, 3, 4], 2, 64, 16, "padded", 1),
    ([5, 6], [12, 9], 8, 128, 64, "tree", 3),
]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("variant", ["plain", "ring", "heads"])
@pytest.mark.parametrize("case", range(len(STEPS)))
def test_step(case, variant, mx):
    lens, drafts, H, D, page, kind, W = STEPS[case]
    sc = Scene(lens, drafts, H, D, 1, page, mx, kind, seed=40 + case)
    x = _step_inputs(sc, W, seed=case, ring=variant == "ring", per_head=variant == "heads")
    d = sc.device()
    before = [t.clone() for t in d["kv"]]
    _run_step(sc, d, x)
    assert int(d["err"]) == 0
    toks, zk, zv = _oracle_step(sc, x, W)
    sm = x["slots"].numpy()[toks]
    if mx:
        for q, z in ((0, zk), (2, zv)):
            data, scale = d["kv"][q].cpu().numpy(), d["kv"][q + 1].cpu().numpy()
            pg, off = sm // page, sm % page
            # only the named rows: copied into sentinel caches, the rest compared below
            gd, gs = np.full_like(data, gu.MX_SENTINEL), np.full_like(scale, gu.MX_SENTINEL)
            gd[pg, off], gs[pg, off] = data[pg, off], scale[pg, off]
            gu.check_mx(gd, gs, sm, z, "step")
    else:
        for q, z in ((0, zk), (1, zv)):
            bits = wl.bits(d["kv"][q].cpu().contiguous()).reshape(-1, H * D)
            gu.assert_close(bits[sm], z.reshape(len(toks), -1), "step")
    mask = np.ones(sc.pages * page, bool)
    mask[sm] = False
    for t, t0 in zip(d["kv"], before):
        a = t.contiguous().view(torch.uint8).cpu().numpy().reshape(sc.pages * page, -1)
        a0 = t0.contiguous().view(torch.uint8).cpu().numpy().reshape(sc.pages * page, -1)
        assert np.array_equal(a[mask], a0[mask])


@pytest.mark.parametrize("W", [1, 4, 8])
@pytest.mark.parametrize("mx", [False, True])
def test_chain_step_equals_prefill_bitwise(W, mx):
    """A tree that is a chain, then its acceptance: cache and state as the
    prefill of the same tokens leaves them, bit for bit."""
    sc = Scene([5, 17, 0], [6, 1, 20], 2, 128, 1, 16, mx, "chain", seed=50)
    x = _step_inputs(sc, W, seed=3)
    d, e = sc.device(), sc.device()
    wide, dx = _run_step(sc, d, x)
    C = sc.H * sc.D
    k, v = wide[:, :C], wide[:, C:]
    st = x["state"].cuda()
    if mx:
        b.prefill_varlen_mxfp8(k, v, e["cu"], dx["wk"], dx["wv"], dx["gk"], dx["gv"], 1e-6, st,
                               dx["slots"], *e["kv"], state_indices=dx["rows"])
    else:
        b.prefill_varlen(k, v, e["cu"], dx["wk"], dx["wv"], dx["gk"], dx["gv"], 1e-6, st, dx["slots"],
                         *e["kv"], state_indices=dx["rows"])
    for t, u in zip(d["kv"], e["kv"]):
        assert torch.equal(t.contiguous().view(torch.uint8), u.contiguous().view(torch.uint8))
    leaves = torch.tensor([n - 1 for n in sc.drafts], dtype=torch.int32, device="cuda")
    new = torch.empty(sc.S, dtype=torch.int32, device="cuda")
    fn = b.tree_accept_mxfp8 if mx else b.tree_accept
    fn(k, v, d["cu"], d["parents"], leaves, d["lens"], d["table"], W, dx["state"] if W > 1 else None,
       *d["kv"], new, state_indices=dx["rows"], err_flag=d["err"])
    assert int(d["err"]) == 0
    assert new.tolist() == [c + n for c, n in zip(sc.lens, sc.drafts)]
    assert torch.equal(dx["state"], st)
    for t, u in zip(d["kv"], e["kv"]):
        assert torch.equal(t.contiguous().view(torch.uint8), u.contiguous().view(torch.uint8))


def test_step_malformed():
    sc = Scene([5, 6], [4, 4], 2, 64, 1, 16, kind="chain", seed=52)
    x = _step_inputs(sc, 3, seed=3)
    good = sc.device()
    _run_step(sc, good, x)

    def run(change, xx=x):
        d = sc.device()
        change(d)
        before = d["kv"][0].clone()
        y = dict(xx)
        _run_step(sc, d, y)
        changed = (d["kv"][0].contiguous().view(torch.int16) != before.contiguous().view(torch.int16)).any(-1).any(-1).cpu().numpy()
        wrote = [bool(changed[ot.place(sc.table[i], sc.lens[i] + j, 16)]) for i in range(2) for j in range(4)]
        return wrote, int(d["err"])

    def par(d):
        d["parents"][1] = 1
    wrote, flag = run(par)  # draft 1 follows itself; 2 meets that in its window
    assert flag == b.FLAG_TREE and wrote[4:] == [True] * 4 and wrote[0] and not wrote[1] and not wrote[2]

    def cu(d):
        d["cu"][2] = 9
    wrote, flag = run(cu)
    assert flag == b.FLAG_CU_SEQLENS and wrote == [True] * 4 + [False] * 4
    y = dict(x)
    y["rows"] = torch.tensor([-1, int(x["rows"][1])], dtype=torch.int32)
    wrote, flag = run(lambda d: None, y)
    assert flag == b.FLAG_STATE_INDEX and wrote == [False] * 4 + [True] * 4
    y = dict(x)
    y["slots"] = x["slots"].clone()
    y["slots"][2] = sc.pages * 16
    wrote, flag = run(lambda d: None, y)
    assert flag == b.FLAG_SLOT_RANGE and wrote == [True, True, False] + [True] * 5


# --------------------------------------------------------------------- acceptance

@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("ring", [False, True])
@pytest.mark.parametrize("lens, drafts, H, D, page, kind, W", [
    ([0], [1], 1, 64, 16, "chain", 4),
    ([10, 15, 0, 31], [9, 4, 16, 2], 2, 128, 16, "padded", 4),
    ([100, 3], [128, 60], 1, 256, 48, "tree", 8),
    ([5, 5, 5], [6, 12, 3], 3, 64, 7, "padded", 2),
    ([5, 8], [6, 12], 2, 64, 1, "tree", 1),
])
def test_accept(lens, drafts, H, D, page, kind, W, ring, mx):
    sc = Scene(lens, drafts, H, D, 1, page, mx, kind, seed=60)
    x = _step_inputs(sc, W, seed=5, ring=ring)
    d = sc.device()
    rng = np.random.default_rng(9)
    leaves, weights = [], torch.rand(sc.S, H, max(c + n for c, n in zip(lens, drafts)))
    for i in range(sc.S):
        used = [j for j, p in enumerate(ot.paths(sc.parents[sc.cu[i]:sc.cu[i + 1]])) if p]
        leaves.append(used[-1] if i != 1 else int(rng.choice(used)))
    if sc.S > 2:
        leaves[2] = -1
    raw = torch.cat([x["k"], x["v"]], 1)
    dk, C = raw.cuda(), H * D
    state, w, new = x["state"].cuda(), weights.cuda(), torch.empty(sc.S, dtype=torch.int32, device="cuda")
    before = [t.cpu().contiguous().view(torch.uint8).numpy() for t in d["kv"]]
    fn = b.tree_accept_mxfp8 if mx else b.tree_accept
    fn(dk[:, :C], dk[:, C:], d["cu"], d["parents"], torch.tensor(leaves, dtype=torch.int32, device="cuda"),
       d["lens"], d["table"], W, state if W > 1 else None, *d["kv"], new, weights=w,
       state_indices=x["rows"].cuda(), state_positions=None if x["pos"] is None else x["pos"].cuda(),
       err_flag=d["err"])
    torch.cuda.synchronize()
    assert int(d["err"]) == 0
    want = [a.copy() for a in before]
    want_w, want_st, want_len = weights.clone(), x["state"].clone(), []
    for i in range(sc.S):
        path = ot.paths(sc.parents[sc.cu[i]:sc.cu[i + 1]])[leaves[i]] if leaves[i] >= 0 else []
        want_len.append(lens[i] + len(path))
        for r, j in enumerate(path):
            to, frm = ot.place(sc.table[i], lens[i] + r, page), ot.place(sc.table[i], lens[i] + j, page)
            for a, a0 in zip(want, before):
                a[to] = a0[frm]
            want_w[i, :, lens[i] + r] = weights[i, :, lens[i] + j]
        if W > 1 and path:
            row = x["rows"][i]
            if ring:
                pos = int(x["pos"][i])
                for r, j in enumerate(path):
                    want_st[row, (pos + r) % (W - 1)] = raw[sc.cu[i] + j]
            else:
                own = torch.cat([x["state"][row]] + [raw[sc.cu[i] + j][None] for j in path])
                want_st[row] = own[-(W - 1):]
    assert new.tolist() == want_len
    assert torch.equal(state.cpu(), want_st) and torch.equal(w.cpu(), want_w)
    for t, a in zip(d["kv"], want):
        assert np.array_equal(t.cpu().contiguous().view(torch.uint8).numpy(), a)


def test_accept_malformed():
    sc = Scene([5, 6], [4, 4], 2, 64, 1, 16, kind="chain", seed=62)
    x = _step_inputs(sc, 3, seed=3)
    C = sc.H * sc.D

    def run(leaves, change=lambda d: None, rows=x["rows"]):
        d = sc.device()
        change(d)
        state, new = x["state"].cuda(), torch.full((2,), -7, dtype=torch.int32, device="cuda")
        raw = torch.cat([x["k"], x["v"]], 1).cuda()
        b.tree_accept(raw[:, :C], raw[:, C:], d["cu"], d["parents"],
                      torch.tensor(leaves, dtype=torch.int32, device="cuda"), d["lens"], d["table"], 3,
                      state, *d["kv"], new, state_indices=rows.cuda(), err_flag=d["err"])
        same = [torch.equal(state[x["rows"][i]].cpu(), x["state"][x["rows"][i]]) for i in range(2)]
        return new.tolist(), same, int(d["err"])

    assert run([4, 1]) == ([5, 8], [True, False], b.FLAG_TREE)
    assert run([-2, 1]) == ([5, 8], [True, False], b.FLAG_TREE)

    def par(d):
        d["parents"][2] = -3
    assert run([3, 1], par) == ([5, 8], [True, False], b.FLAG_TREE)
    assert run([1, 1], par) == ([7, 8], [False, False], 0)

    def lens(d):
        d["lens"][0] = 1 << 30
    assert run([1, 1], lens) == ([-7, 8], [True, False], b.FLAG_CONTEXT)
    bad = torch.tensor([99, int(x["rows"][1])], dtype=torch.int32)
    assert run([1, 1], rows=bad) == ([7, 8], [True, False], b.FLAG_STATE_INDEX)


# ----------------------------------------------------------------------- eviction

EVICTS = [
    # lens, H, D, page, keep, sinks, recent
    ([10], 1, 64, 16, 4, 1, 1),
    ([0, 1, 5, 6, 7], 2, 64, 16, 6, 2, 2),
    ([300, 41, 1000], 2, 128, 64, 128, 4, 20),
    ([77, 500], 3, 64, 7, 33, 0, 0),
    ([2500], 1, 256, 48, 2000, 3, 500),
    ([400], 2, 128, 16, 50, 20, 30),
    ([5000, 1200], 2, 128, 64, 1025, 0, 1),
    ([64, 64], 1, 64, 16, 63, 63, 0),
]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("values", ["random", "ties", "special"])
@pytest.mark.parametrize("case", range(len(EVICTS)))
def test_evict(case, values, mx):
    lens, H, D, page, keep, sinks, recent = EVICTS[case]
    sc = Scene(lens, [0] * len(lens), H, D, 1, page, mx, "chain", seed=70 + case)
    d = sc.device()
    gen = torch.Generator().manual_seed(case)
    room = max(lens) + 2
    w = torch.rand(sc.S, H, room, generator=gen) ** 8 * 50
    if values == "ties":
        w = (w * 2).floor()
    elif values == "special":
        pick = torch.randint(0, 9, w.shape, generator=gen)
        for q, v in enumerate((0.0, -0.0, float("inf"), float("-inf"), float("nan"), 1e-42, -3.0)):
            w[pick == q] = v
    before = [t.cpu().contiguous().view(torch.uint8).numpy() for t in d["kv"]]
    kept = torch.full((sc.S, H, keep), 77, dtype=torch.int32, device="cuda")
    new = torch.empty(sc.S, dtype=torch.int32, device="cuda")
    out = torch.full((sc.S, H, max(room, keep)), 5.0, device="cuda")
    fn = b.evict_mxfp8 if mx else b.evict
    fn(w.cuda(), d["lens"], d["table"], *d["kv"], sinks, recent, kept, new, out, err_flag=d["err"])
    torch.cuda.synchronize()
    assert int(d["err"]) == 0
    assert new.tolist() == [min(c, keep) for c in lens]
    want = [a.copy() for a in before]
    for i in range(sc.S):
        for h in range(H):
            pick = ot.evict_pick(w[i, h].numpy(), lens[i], keep, sinks, recent)
            assert kept[i, h].tolist() == pick + [-1] * (keep - len(pick))
            got = out[i, h].cpu().numpy()
            assert np.array_equal(got[:len(pick)], w[i, h].numpy()[pick], equal_nan=True)
            assert (got[len(pick):] == 5).all()
            for r, p in enumerate(pick):
                to, frm = ot.place(sc.table[i], r, page), ot.place(sc.table[i], p, page)
                for a, a0 in zip(want, before):
                    a[to + (h,)] = a0[frm + (h,)]
    for t, a in zip(d["kv"], want):
        assert np.array_equal(t.cpu().contiguous().view(torch.uint8).numpy(), a)


def test_evict_flags():
    sc = Scene([50, 60], [0, 0], 2, 64, 1, 16, kind="chain", seed=80)
    d = sc.device()
    d["lens"][0] = 1000
    before = [t.clone() for t in d["kv"]]
    kept = torch.full((2, 2, 20), 77, dtype=torch.int32, device="cuda")
    new = torch.full((2,), -7, dtype=torch.int32, device="cuda")
    b.evict(torch.rand(2, 2, 64, device="cuda"), d["lens"], d["table"], *d["kv"], 1, 2, kept, new,
            err_flag=d["err"])
    assert int(d["err"]) == b.FLAG_CONTEXT
    assert new.tolist() == [-7, 20] and (kept[0] == 77).all()
    rows = torch.from_numpy(sc.table[0, :4].astype(np.int64))
    assert torch.equal(d["kv"][0][rows].view(torch.int16), before[0][rows].view(torch.int16))


# --------------------------------------------------------------------- all together

@pytest.mark.parametrize("mx", [False, True])
def test_serving_steps(mx):
    """Prefill, then rounds of drafting, attention, weights and acceptance with an
    eviction between, all enqueued without a synchronisation; then the last
    attention against the definition on the cache that came out."""
    H, D, page, W, g = 2, 64, 16, 4, 4
    S, rounds, room = 3, 4, 200
    gen = torch.Generator().manual_seed(1)
    C, HQ = H * D, H * g
    lens0 = [60, 33, 5]
    pages = -(-room // page) * S
    table = torch.randperm(pages, generator=gen).to(torch.int32).view(S, -1)
    rnd = lambda *s: torch.randn(*s, generator=gen).to(torch.bfloat16)  # noqa: E731
    wk, wv = rnd(W, C).cuda(), rnd(W, C).cuda()
    gk, gv = torch.ones(D, device="cuda"), torch.ones(D, device="cuda")
    state = torch.zeros(S, W - 1, 2 * C, dtype=torch.bfloat16, device="cuda")
    if mx:
        kv = (*gu.mx_caches(pages, page, H, D), *gu.mx_caches(pages, page, H, D))
    else:
        kv = tuple(torch.full((pages, page, H, D), float("nan"), dtype=torch.bfloat16, device="cuda")
                   for _ in range(2))
    fn = {n: getattr(b, n + ("_mxfp8" if mx else "")) for n in
          ("prefill_varlen", "tree_step", "tree_attention", "attention_weights", "tree_accept", "evict")}
    err = torch.zeros(1, dtype=torch.int32, device="cuda")
    cu = torch.tensor(np.concatenate([[0], np.cumsum(lens0)]), dtype=torch.int32)
    T = int(cu[-1])
    slots = torch.cat([table[i].long()[torch.arange(c) // page] * page + torch.arange(c) % page
                       for i, c in enumerate(lens0)])
    fn["prefill_varlen"](rnd(T, H, D).cuda(), rnd(T, H, D).cuda(), cu.cuda(), wk, wv, gk, gv, 1e-6, state,
                         slots.cuda(), *kv, err_flag=err)
    lens, dtab = torch.tensor(lens0, dtype=torch.int32, device="cuda"), table.cuda()
    weights, spare = (torch.zeros(S, H, room, device="cuda") for _ in range(2))
    host = list(lens0)
    dcu = torch.tensor([0, 6, 12, 18], dtype=torch.int32, device="cuda")
    parents = [-1, 0, 0, 2, 2, -1]
    dpar = torch.tensor(parents * S, dtype=torch.int32, device="cuda")
    leaves = torch.tensor([3, 1, 5], dtype=torch.int32, device="cuda")
    path_len = [3, 2, 1]
    paths = ot.paths(parents)
    on = [paths[3], paths[1], paths[5]]
    dacc = torch.tensor([p if j in on[i] else -2 for i in range(S) for j, p in enumerate(parents)],
                        dtype=torch.int32, device="cuda")
    lse = torch.empty(6 * S, HQ, device="cuda")
    for r in range(rounds):
        k, v, q = rnd(6 * S, H, D).cuda(), rnd(6 * S, H, D).cuda(), rnd(6 * S, HQ, D).cuda()
        slots = torch.cat([table[i].long()[(host[i] + torch.arange(6)) // page] * page +
                           (host[i] + torch.arange(6)) % page for i in range(S)]).cuda()
        fn["tree_step"](k, v, dcu, dpar, wk, wv, gk, gv, 1e-6, state, slots, *kv, err_flag=err)
        out = fn["tree_attention"](q, dcu, dpar, lens, dtab, *kv, D ** -0.5, 6, lse=lse, err_flag=err)
        if r == rounds - 1:
            break
        fn["attention_weights"](q, lse, dcu, dacc, lens, dtab, *kv[:2 if mx else 1], D ** -0.5, 6, weights,
                                err_flag=err)
        new = torch.empty_like(lens)
        fn["tree_accept"](k, v, dcu, dpar, leaves, lens, dtab, W, state, *kv, new, weights=weights,
                          err_flag=err)
        lens, host = new, [c + m for c, m in zip(host, path_len)]
        if r == 1:
            kept, new = torch.empty(S, H, 40, dtype=torch.int32, device="cuda"), torch.empty_like(lens)
            fn["evict"](weights, lens, dtab, *kv, 2, 8, kept, new, spare, err_flag=err)
            lens, weights, spare = new, spare, weights
            host = [min(c, 40) for c in host]
    torch.cuda.synchronize()
    assert int(err) == 0 and lens.tolist() == host
    # the weight that a round's accepted tokens gave: g a token and head, spread over what it saw
    if mx:
        vals = [ot.mx_values(kv[i].cpu().numpy(), kv[i + 1].cpu().numpy()) for i in (0, 2)]
    else:
        vals = [t.double().cpu().numpy() for t in kv]
    ref = ot.attention(q.double().cpu().numpy(), dcu.tolist(), parents * S, host, table.numpy(), *vals,
                       D ** -0.5)
    check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), ref, D)
