"""The drafted-tree operators at the edges of what their documentation allows."""
import numpy as np
import pytest
import torch

from short_conv_kv_b200 import binding as b
from tests.tree_util import Scene, check_attention, logit_error

pytestmark = pytest.mark.gpu


# ------------------------------------------- non-finite rows at the context's end

@pytest.mark.parametrize("mx, what", [(False, "nan"), (False, "inf"), (True, "nan"), (True, "scale")])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [1, 2, 20])  # 4, 8 and 80 rows a K/V head
@pytest.mark.parametrize("ctx", [401, 415])
def test_nonfinite_rows_at_the_end_of_the_context(ctx, n, D, mx, what):
    """NaN or an infinity in V of a cached row reaches all tokens (a padding token: none), also when the
    row is among the last ctx % 16, whose keys share a step with the drafted ones."""
    sc = Scene([ctx], [n], 2, D, 4, 16, mx, "padded", seed=500 + n)
    d = sc.device()
    clean = sc.attend(d)
    used = torch.tensor([p > -2 for p in sc.parents.tolist()], device="cuda")
    v = d["kv"][3 if what == "scale" else 2 if mx else 1]
    bad = 0xFF if what == "scale" else 0x7F if mx else float(what)
    at = 1 if what == "scale" else 37
    cols = slice(32, 64) if what == "scale" else slice(37, 38)
    for p in (ctx // 16 * 16 - 1, ctx // 16 * 16, ctx - 1):
        pg, off = int(sc.table[0, p // 16]), p % 16
        keep = v[pg, off, 0, at].clone()
        v[pg, off, 0, at] = bad
        got = sc.attend(d)
        v[pg, off, 0, at] = keep
        hit = got[:, :4, cols][used].float()
        assert (torch.isinf(hit) & (hit > 0) if what == "inf" else torch.isnan(hit)).all(), p
        rest = torch.ones_like(got, dtype=torch.bool)
        rest[:, :4, cols] = ~used[:, None, None]
        assert torch.equal(got[rest], clean[rest]), p
    assert int(d["err"]) == 0


# -------------------------------------------------- scales that overflow

@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("n", [2, 20])
@pytest.mark.parametrize("scale, codes", [(247, (0x78, 0xF8)), (250, (0x7E, 0x60)), (254, (0x40, 0xFE)), (254, (0x3F, 0xBF))])
def test_overflowing_scales_reach_nobody_else(scale, codes, n, D):
    """A drafted row whose V codes times their scale pass the largest float: infinite for the token itself,
    and no trace in its siblings.  (254, 0x3F) is 1.875 * 2^127: large, and finite."""
    sc = Scene([50], [n], 2, D, 4, 16, True, "star", seed=520)
    d = sc.device()
    clean = sc.attend(d).clone()
    p = 50 + n - 1
    pg, off = int(sc.table[0, p // 16]), p % 16
    d["kv"][2][pg, off, 1, 32:64] = codes[0]
    d["kv"][2][pg, off, 1, 40] = codes[1]
    d["kv"][3][pg, off, 1, 1] = scale
    got = sc.attend(d)
    assert torch.equal(got[:n - 1], clean[:n - 1])
    assert torch.equal(got[n - 1, :4], clean[n - 1, :4])
    own = got[n - 1, 4:].float()
    code = torch.tensor(codes, dtype=torch.uint8).view(torch.float8_e4m3fn).double() * 2.0 ** (scale - 127)
    for c, col in ((code[0], 33), (code[1], 40)):
        if abs(float(c)) >= 2.0 ** 128:
            assert (own[:, col] == float(c) * float("inf")).all()
        else:
            assert torch.isfinite(own[:, col]).all() and (own[:, col] * float(c) > 0).all()
    rest = torch.ones(D, dtype=torch.bool)
    rest[32:64] = False
    assert torch.equal(got[n - 1, 4:][:, rest], clean[n - 1, 4:][:, rest])


# --------------------------------------------- tensors allocated within a call

def _segment_stream(t):
    """The stream whose pool of the caching allocator holds t."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]
    raise AssertionError("not the caching allocator's")


@pytest.mark.parametrize("given", ["neither", "out", "workspace"])
@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("mx", [False, True])
def test_allocations_belong_to_the_calls_stream(mx, handle, given, monkeypatch):
    """What a call on another stream allocates for itself comes from that stream's memory: a block of the
    current stream may still be in use by kernels that nothing orders before the call."""
    sc = Scene([300, 20], [3, 9], 2, 64, 4, 16, mx, seed=530)
    d = sc.device()
    want = sc.attend(d)
    made = []
    make = b.tree_attention_workspace

    def keep(*a):
        made.append(make(*a))
        return made[-1]
    monkeypatch.setattr(b, "tree_attention_workspace", keep)
    for stream in (torch.cuda.Stream(), torch.cuda.default_stream()):
        made.clear()
        out = torch.empty_like(want) if given == "out" else None
        ws = make(d["q"], d["kv"][0], sc.S, sc.max_draft) if given == "workspace" else None
        torch.cuda.synchronize()
        current = torch.cuda.current_stream()
        got = sc.attend(d, out=out, workspace=ws, stream=stream.cuda_stream if handle else stream)
        assert torch.cuda.current_stream() == current
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        if given != "out":
            assert _segment_stream(got) == stream.cuda_stream
        if given != "workspace":
            assert [_segment_stream(w) for w in made] == [stream.cuda_stream]


# ------------------------------------------------ batches with nothing drafted

@pytest.mark.parametrize("W", [1, 4])
@pytest.mark.parametrize("mx", [False, True])
def test_batch_without_drafted_tokens(mx, W):
    """T = 0: the lengths are written all the same, and nothing else changes."""
    sc = Scene([30, 0, 17], [0, 0, 0], 2, 64, 4, 16, mx, seed=540)
    d = sc.device()
    before = [t.clone() for t in d["kv"]]
    raw = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    state = torch.randn(3, W - 1, 256, device="cuda").to(torch.bfloat16)
    state0 = state.clone()
    w = torch.rand(3, 2, 40, device="cuda")
    w0 = w.clone()
    new = torch.full((3,), -7, dtype=torch.int32, device="cuda")
    leaves = torch.full((3,), -1, dtype=torch.int32, device="cuda")
    fn = b.tree_accept_mxfp8 if mx else b.tree_accept
    fn(raw, raw, d["cu"], d["parents"], leaves, d["lens"], d["table"], W, state if W > 1 else None, *d["kv"], new,
       weights=w, err_flag=d["err"])
    assert new.tolist() == [30, 0, 17] and int(d["err"]) == 0
    assert torch.equal(state, state0) and torch.equal(w, w0)
    for t, t0 in zip(d["kv"], before):
        assert torch.equal(t.contiguous().view(torch.uint8), t0.contiguous().view(torch.uint8))
    leaves[1] = 0  # a leaf that is no token
    fn(raw, raw, d["cu"], d["parents"], leaves, d["lens"], d["table"], W, state if W > 1 else None, *d["kv"], new,
       weights=w, err_flag=d["err"])
    assert new.tolist() == [30, 0, 17] and int(d["err"]) == b.FLAG_TREE
    assert sc.attend(d).shape == (0, 8, 64)
    lse = torch.empty(0, 8, device="cuda")
    (b.attention_weights_mxfp8 if mx else b.attention_weights)(
        d["q"], lse, d["cu"], d["parents"], d["lens"], d["table"], *d["kv"][:2 if mx else 1], sc.scale, 1, w)
    assert torch.equal(w, w0)


# --------------------------------------------------- the largest head groups

@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("H, group, n, D", [(2, 16384, 65, 64), (2, 16384, 65, 256), (1, 32768, 128, 64)])
def test_weights_of_a_million_query_rows(H, group, n, D, mx):
    """More than 2^20 query rows a K/V head, up to the largest that is taken: every head's own rows are
    weighed, and nothing else is written."""
    sc = Scene([20], [n], H, D, 1, 16, mx, "chain", seed=550)
    d = sc.device()
    gen = torch.Generator(device="cuda").manual_seed(5)
    q = torch.randn(n, H * group, D, generator=gen, device="cuda").to(torch.bfloat16)
    lse = 14 + torch.rand(n, H * group, generator=gen, device="cuda")
    w0 = torch.rand(1, H + 2, 20 + n + 3, generator=gen, device="cuda")
    w = w0.clone()
    fn = b.attention_weights_mxfp8 if mx else b.attention_weights
    fn(q, lse, d["cu"], d["parents"], d["lens"], d["table"], *d["kv"][:2 if mx else 1], sc.scale, n,
       w[:, 1:-1, :-3], d["err"])
    assert int(d["err"]) == 0
    p = np.arange(20 + n)
    k = torch.from_numpy(sc.values(0)[sc.table[0, p // 16], p % 16]).cuda()  # [20 + n, H, D]
    add = torch.zeros(H, 20 + n, dtype=torch.float64, device="cuda")
    size = 0.0
    for j in range(n):
        x = q[j].double().view(H, group, D)
        s = torch.einsum("hgd,phd->hgp", x, k[:21 + j]) * sc.scale
        add[:, :21 + j] += torch.exp(s - lse[j].double().view(H, group, 1)).sum(1)
        size = max(size, float(torch.einsum("hgd,phd->hgp", x.abs(), k[:21 + j].abs()).max() * sc.scale))
    want = w0.double()
    want[0, 1:-1, :20] += add[:, :20]
    want[0, 1:-1, 20:-3] = add[:, 20:]
    # a term's exponent: the score's error, lse * log2(e)'s rounding and the subtraction's, ex2's 2^-22; sums
    # of positive terms: at most 2^6 additions in a pass of 64 rows or more, then one a pass, 2^-24 each of what
    # is there
    e = logit_error(size, D) + 2.0 ** -22 * (2 + 15) + (2 ** 6 + n * group / 64) * 2.0 ** -24
    err = (w.double() - want).abs()
    assert (err[0, 1:-1, :-3] <= e * want[0, 1:-1, :-3]).all(), (err[0, 1:-1, :-3] / want[0, 1:-1, :-3]).max() / e
    rest = torch.ones_like(w, dtype=torch.bool)
    rest[0, 1:-1, :-3] = False
    assert torch.equal(w[rest], w0[rest])


# --------------------------------- masked rows, where several CTAs share a unit

@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("ctx, n", [(2000, 2), (2003, 2), (2000, 20), (1985, 50), (1900, 128)])
def test_masked_nonfinite_rows_in_cut_units(ctx, n, D, mx):
    """A drafted row with NaN in K and V, in a context that is cut into parts: its own token is NaN, its
    siblings' bits and the padding's zeros are as they were."""
    sc = Scene([ctx], [n], 1, D, 4, 16, mx, "star", seed=560)
    d = sc.device()
    if n > 8:
        d["parents"][n - 3] = -2  # padding among them
    clean = sc.attend(d).clone()
    p = ctx + n - 2
    pg, off = int(sc.table[0, p // 16]), p % 16
    for t in d["kv"]:
        t[pg, off] = 0xFF if t.dtype == torch.uint8 else float("nan")
    got = sc.attend(d)
    assert torch.isnan(got[n - 2]).all()
    others = torch.arange(n, device="cuda") != n - 2
    assert torch.equal(got[others], clean[others]) and torch.isfinite(got[others]).all()
    assert int(d["err"]) == 0


# ------------------------------------------------- one step under other layouts

def _five_calls(sc, d, seed):
    """Step, attention, weights, acceptance and eviction on the scene's cache; everything they leave."""
    H, D, W, T, S, g = sc.H, sc.D, 4, sc.T, sc.S, sc.group
    C = H * D
    fn = {n: getattr(b, n + ("_mxfp8" if sc.mx else ""))
          for n in ("tree_step", "tree_attention", "attention_weights", "tree_accept", "evict")}
    gen = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    raw, taps, state = rnd(2, T, C), rnd(2, W, C), rnd(S, W - 1, 2 * C)
    gamma = torch.ones(D, device="cuda")
    pos = np.concatenate([c + np.arange(n) for c, n in zip(sc.lens, sc.drafts)])
    seq = np.repeat(np.arange(S), sc.drafts)
    slots = torch.from_numpy(sc.table[seq, pos // sc.page].astype(np.int64) * sc.page + pos % sc.page).cuda()
    at = (d["cu"], d["parents"])
    fn["tree_step"](raw[0], raw[1], *at, taps[0], taps[1], gamma, gamma, 1e-6, state, slots, *d["kv"],
                    err_flag=d["err"])
    lse = torch.full((T, H * g), 7.0, device="cuda")
    out = fn["tree_attention"](d["q"], *at, d["lens"], d["table"], *d["kv"], sc.scale, sc.max_draft, lse=lse,
                               err_flag=d["err"])
    w = torch.rand(S, H, sc.table.shape[1] * sc.page, generator=gen, device="cuda")
    fn["attention_weights"](d["q"], lse, *at, d["lens"], d["table"], *d["kv"][:2 if sc.mx else 1], sc.scale,
                            sc.max_draft, w, err_flag=d["err"])
    leaves = torch.tensor([n - 1 for n in sc.drafts], dtype=torch.int32, device="cuda")
    new, last = (torch.empty(S, dtype=torch.int32, device="cuda") for _ in range(2))
    fn["tree_accept"](raw[0], raw[1], *at, leaves, d["lens"], d["table"], W, state, *d["kv"], new, weights=w,
                      err_flag=d["err"])
    kept, wo = torch.empty(S, H, 40, dtype=torch.int32, device="cuda"), torch.zeros_like(w)
    fn["evict"](w, new, d["table"], *d["kv"], 2, 8, kept, last, wo, err_flag=d["err"])
    torch.cuda.synchronize()
    assert int(d["err"]) == 0
    return [out, lse, w, state, new, kept, last, wo] + [t.contiguous() for t in d["kv"]]


@pytest.mark.parametrize("layout, mx", [("heads first", False), ("heads first", True), ("far pages", False),
                                        ("far pages", True), ("odd scales", True)])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("drafts", [[3, 1], [40, 9]])
def test_layouts_give_the_same_bits(layout, drafts, D, mx):
    """The five calls on the same rows in another layout: head-major pages, pages that lie past 2^32 elements,
    scale bytes at odd addresses."""
    # the tables' last pages are full to the last slot
    sc = Scene([128 - drafts[0], 96 - drafts[1]], drafts, 2, D, 4, 16, mx, "chain", seed=570, width_extra=0)
    d, e = sc.device(), sc.device()

    def place(t, scales):
        P, page, H, n = t.shape
        if layout == "heads first":
            return t.permute(0, 2, 1, 3).contiguous().permute(0, 2, 1, 3)
        if layout == "far pages":  # the last page begins at 2^32 elements or behind (their scales: at 1/32 of that)
            stride = (2 ** 32 // (P - 1) // 1024 + 1) * 1024 // (32 if scales else 1)
            room = torch.empty((P - 1) * stride + page * H * n, dtype=t.dtype, device="cuda")
            far = room.as_strided(t.shape, (stride, H * n, n, 1))
            assert scales or (P - 1) * stride >= 2 ** 32
            return far.copy_(t)
        if not scales:
            return t.contiguous()
        room = torch.empty(t.numel() + 16, dtype=torch.uint8, device="cuda")
        return room[odd.pop():][:t.numel()].view(t.shape).copy_(t)
    odd = [3, 1]
    e["kv"] = tuple(place(t, sc.mx and i % 2 == 1) for i, t in enumerate(d["kv"]))
    if layout == "odd scales":
        d["kv"] = tuple(t.contiguous() for t in d["kv"])
    for x, y in zip(_five_calls(sc, d, 6), _five_calls(sc, e, 6)):
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8))


# ----------------------------------------------------------- counts at their ends

@pytest.mark.parametrize("mx", [False, True])
def test_no_sequence_at_all(mx):
    """S = 0: every call returns, and nothing is written."""
    sc = Scene([20], [2], 2, 64, 4, 16, mx, seed=580)
    d = sc.device()
    i32 = dict(dtype=torch.int32, device="cuda")
    none, cu, table = torch.empty(0, **i32), torch.zeros(1, **i32), torch.empty(0, 4, **i32)
    q, lse = torch.empty(0, 8, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 8, device="cuda")
    raw = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda")
    w, kept = torch.empty(0, 2, 30, device="cuda"), torch.empty(0, 2, 9, **i32)
    state = torch.empty(0, 3, 256, dtype=torch.bfloat16, device="cuda")
    taps = torch.ones(4, 128, dtype=torch.bfloat16, device="cuda")
    gamma = torch.ones(64, device="cuda")
    before = [t.clone() for t in d["kv"]]
    fn = {n: getattr(b, n + ("_mxfp8" if mx else ""))
          for n in ("tree_step", "tree_attention", "attention_weights", "tree_accept", "evict")}
    fn["tree_step"](raw, raw, cu, none, taps, taps, gamma, gamma, 1e-6, state,
                    torch.empty(0, dtype=torch.int64, device="cuda"), *d["kv"])
    assert fn["tree_attention"](q, cu, none, none, table, *d["kv"], 0.1, 3, lse=lse).shape == (0, 8, 64)
    fn["attention_weights"](q, lse, cu, none, none, table, *d["kv"][:2 if mx else 1], 0.1, 3, w)
    fn["tree_accept"](raw, raw, cu, none, none, none, table, 4, state, *d["kv"], torch.empty(0, **i32), weights=w)
    fn["evict"](w, none, table, *d["kv"], 1, 2, kept, torch.empty(0, **i32))
    torch.cuda.synchronize()
    for t, t0 in zip(d["kv"], before):
        assert torch.equal(t.contiguous().view(torch.uint8), t0.contiguous().view(torch.uint8))


@pytest.mark.parametrize("max_draft", [1, 128])
def test_seventy_thousand_sequences(max_draft):
    """More sequences than a grid's smaller dimensions hold, some without a token: each one's result is its
    own, with the few-row kernels and with the tensor cores'."""
    S, H, D, g, page = 70001, 1, 64, 2, 4
    gen = torch.Generator(device="cuda").manual_seed(8)
    lens = torch.randint(0, 7, (S,), generator=gen, device="cuda").to(torch.int32)
    n = (torch.rand(S, generator=gen, device="cuda") < 0.9).to(torch.int32)
    cu = torch.cat([torch.zeros(1, dtype=torch.int32, device="cuda"), n.cumsum(0).to(torch.int32)])
    T = int(cu[-1])
    table = torch.randint(0, 500, (S, 2), generator=gen, device="cuda").to(torch.int32)  # shared pages
    kc, vc = (torch.randn(500, page, H, D, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(T, g, D, generator=gen, device="cuda").to(torch.bfloat16)
    par = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    lse, err = torch.empty(T, g, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = b.tree_attention(q, cu, par, lens, table, kc, vc, 0.125, max_draft, lse=lse, err_flag=err)
    w = torch.ones(S, H, 8, device="cuda")
    b.attention_weights(q, lse, cu, par, lens, table, kc, 0.125, max_draft, w, err)
    assert int(err) == 0
    seq = n.nonzero().flatten()
    p = torch.arange(8, device="cuda")
    page_of = table[seq].long().gather(1, (p // page).expand(T, 8))
    k, v = (t[page_of, p % page, 0].double() for t in (kc, vc))  # [T, 8, D]
    c = lens[seq].long()[:, None]
    s = torch.einsum("tgd,tpd->tgp", q.double(), k) * 0.125
    s.masked_fill_((p[None] > c)[:, None], -float("inf"))
    prob = s.softmax(-1)
    # as in tree_util.check_attention: roundings of the output and of the probabilities, then the fp32 parts
    size = float(torch.einsum("tgd,tpd->tgp", q.double().abs(), k.abs()).max()) * 0.125
    mag = torch.einsum("tgp,tpd->tgd", prob, v.abs())
    want = torch.einsum("tgp,tpd->tgd", prob, v)
    e = logit_error(size, D) + 2.0 ** -22 + 2.0 ** -11
    assert ((out.double() - want).abs() <= 2.0 ** -8 * (want.abs() + mag) * 1.01 + 2 * e * mag).all()
    ref = torch.logsumexp(s, -1)
    assert ((lse.double() - ref).abs() <= logit_error(size, D) + 2.0 ** -20 + 2.0 ** -22 * ref.abs()).all()
    add = torch.exp(s - lse.double()[..., None]).sum(1)
    full = torch.ones(S, 8, dtype=torch.float64, device="cuda")
    full[seq] = torch.where(p[None] < c, 1 + add, torch.where(p[None] == c, add, 1.0))
    we = logit_error(size, D) + 2.0 ** -22 * (2 + float(lse.abs().max())) + 2.0 ** -20
    assert ((w[:, 0].double() - full).abs() <= we * full).all()
    # the same rows with every sequence's acceptance: lengths of all of them
    new = torch.empty(S, dtype=torch.int32, device="cuda")
    raw = torch.zeros(T, D, dtype=torch.bfloat16, device="cuda")
    b.tree_accept(raw, raw, cu, par, n - 1, lens, table, 1, None, kc, vc, new, err_flag=err)
    assert torch.equal(new, lens + n) and int(err) == 0


@pytest.mark.parametrize("mx", [False, True])
def test_a_bound_far_above_the_drafts(mx):
    """max_draft is a bound: few tokens under a large one, on the kernels for many rows."""
    sc = Scene([100, 700], [2, 1], 2, 128, 4, 64, mx, "chain", seed=590)
    d = sc.device()
    lse = torch.empty(sc.T, sc.HQ, device="cuda")
    out = sc.attend(d, lse=lse, max_draft=128)
    check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), sc.oracle_attention(), 128)
    assert int(d["err"]) == 0


# -------------------------------------------------------------- huge scores

@pytest.mark.parametrize("power", [4, 26, 30, 36, 100])
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("S, ctx, n", [(1, 700, 1), (1, 700, 20), (1, 700, 50), (160, 90, 20), (160, 140, 50)])
@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("sign", [1, -1])
def test_huge_scores(sign, mx, S, ctx, n, D, power):
    """Scores of any size that floats hold, far apart: the largest wins, wherever it lies, and equal ones share.
    (All products and sums are exact: one dimension counts, with powers of two and small integers.)  Contexts
    that many CTAs share, and ones that a CTA has whole."""
    sc = Scene([ctx] * S, [n] * S, 1, D, 4, 16, mx, "star", seed=600)
    sc.scale = sign * D ** -0.5 * 1.1
    d = sc.device()
    total = ctx + n
    p = np.arange(total)
    at = (torch.from_numpy(sc.table[:, p // 16].astype(np.int64)).cuda(), torch.from_numpy(p % 16).cuda())
    gen = torch.Generator(device="cuda").manual_seed(4)
    c = torch.randint(-100, 100, (S, total), generator=gen, device="cuda").float() if not mx else \
        torch.randint(-12, 13, (S, total), generator=gen, device="cuda").float()
    c[:, [5, ctx - 10]] = 15.0 if mx else 120.0  # the winners, in tiles far apart
    half = 2.0 ** (power // 2)
    d["q"].zero_()
    d["q"][:, :, 0] = half
    rows = torch.zeros(S, total, 1, D, device="cuda")
    rows[..., 0, 0] = sign * c
    if mx:
        d["kv"][0][at] = rows.to(torch.float8_e4m3fn).view(torch.uint8)
        d["kv"][1][at] = 127 + power // 2
    else:
        d["kv"][0][at] = (rows * half).to(torch.bfloat16)
    lse = torch.empty(sc.T, sc.HQ, device="cuda")
    out = sc.attend(d, lse=lse).view(S, n, 4, D)
    assert int(d["err"]) == 0
    s = c.double() * 2.0 ** (2 * (power // 2)) * abs(sc.scale)
    x = s[:, None].expand(S, n, total).clone()
    x[:, :, ctx:].masked_fill_(~torch.eye(n, dtype=torch.bool, device="cuda"), -float("inf"))
    prob = x.softmax(-1)
    v = torch.from_numpy(sc.values(1)).cuda()[at][:, :, 0]
    want, mag = (prob @ v)[:, :, None], (prob @ v.abs())[:, :, None]
    # as in tree_util.check_attention; where more than the winners count (the smallest power) the scores are exact
    # but for the factor scale * log2(e): two roundings each, and those of the difference
    e = 2.0 ** -22 * float(s.abs().max()) if power < 8 else 0.0
    bound = 2.0 ** -8 * (want.abs() + mag) * 1.01 + (2.0 ** -11 + 2 * e) * mag
    assert ((out.double() - want).abs() <= bound).all()
    ref = torch.logsumexp(x, -1)[:, :, None]
    assert ((lse.view(S, n, 4).double() - ref).abs() <= 2.0 ** -21 * ref.abs() + 2.0 ** -20).all()
