"""The drafted-tree operators at the edges of what their documentation allows."""
import numpy as np
import pytest
import torch

from short_conv_kv_b200 import binding as b
from tests.tree_util import Scene, logit_error

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
