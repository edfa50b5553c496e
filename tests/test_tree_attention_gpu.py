"""Attention of drafted trees over the paged cache, against its definition in
64 bits."""
import numpy as np
import pytest
import torch

from tests.tree_util import Scene, check_attention

pytestmark = pytest.mark.gpu

SHAPES = [
    # lens, drafts, H, D, group, page, kind
    ([0], [1], 1, 64, 1, 16, "chain"),
    ([1], [1], 2, 128, 8, 64, "chain"),
    ([15, 16, 17], [1, 1, 1], 2, 64, 4, 16, "chain"),
    ([63, 64, 65, 0], [1, 2, 3, 4], 2, 128, 4, 64, "tree"),
    ([200], [8], 2, 128, 1, 48, "padded"),
    ([129, 5, 700], [5, 16, 2], 1, 128, 5, 100, "padded"),
    ([1000], [3], 3, 256, 2, 64, "tree"),
    ([333, 0], [7, 9], 2, 256, 3, 16, "padded"),
    ([2500], [1], 2, 64, 16, 7, "chain"),
    ([40, 0, 90], [0, 3, 0], 2, 64, 2, 16, "star"),
    ([300], [64], 1, 128, 8, 64, "padded"),
    ([77, 513], [128, 33], 2, 64, 2, 32, "padded"),
    ([260], [40], 1, 256, 4, 64, "tree"),
    ([511, 1100], [17, 30], 2, 128, 3, 128, "padded"),
    ([90], [128], 1, 64, 1, 64, "chain"),
    ([3, 1, 0, 12, 100, 31, 7], [2, 1, 5, 1, 1, 6, 3], 4, 128, 4, 1, "tree"),
]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("case", range(len(SHAPES)))
def test_against_definition(case, mx):
    lens, drafts, H, D, group, page, kind = SHAPES[case]
    sc = Scene(lens, drafts, H, D, group, page, mx, kind, seed=100 + case)
    d = sc.device()
    lse = torch.full((sc.T, sc.HQ), 7.0, device="cuda")
    out = sc.attend(d, lse=lse)
    torch.cuda.synchronize()
    assert int(d["err"]) == 0
    check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), sc.oracle_attention(), D,
                    str(SHAPES[case]))


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("drafts", [[1, 1], [3, 2], [24, 50]])
def test_same_call_same_bits(mx, drafts):
    sc = Scene([3000, 1234], drafts, 2, 128, 8, 64, mx, "padded", seed=3)
    d = sc.device()
    first = sc.attend(d).clone()
    for _ in range(5):
        assert torch.equal(sc.attend(d), first)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("n", [2, 40])
def test_masked_nonfinite_rows_reach_nobody_else(mx, n):
    """NaN and infinities in one drafted row's K and V reach that token and its
    descendants only; the others' results are bit for bit what they were."""
    sc = Scene([50], [n], 2, 128, 4, 16, mx, "star", seed=5)
    d = sc.device()
    clean = sc.attend(d).clone()
    p = 50 + n - 1
    pg, off = int(sc.table[0, p // 16]), p % 16
    for t in d["kv"]:
        t[pg, off] = 0xFF if t.dtype == torch.uint8 else float("nan")
    got = sc.attend(d)
    assert torch.equal(got[:n - 1], clean[:n - 1])
    assert torch.isnan(got[n - 1]).all()
    if not mx:  # an infinite V alone
        d = sc.device()
        d["kv"][1][pg, off, 0, 3] = float("inf")
        got = sc.attend(d)
        assert torch.equal(got[:n - 1], clean[:n - 1])
        last = got[n - 1].float()
        g = sc.group
        assert torch.isinf(last[:g, 3]).all() and (last[:g, 3] > 0).all()
        keep = torch.ones_like(last, dtype=torch.bool)
        keep[:g, 3] = False
        assert torch.equal(got[n - 1][keep], clean[n - 1][keep])


def test_extreme_scores():
    """Scores far apart and large: the running maximum moves many times."""
    sc = Scene([700], [2], 1, 64, 4, 16, False, "chain", seed=8)
    sc.q *= 40
    p = np.arange(700)
    kv = sc._pick(sc.store[0], 0)
    ramp = torch.linspace(0.01, 3, 700)[:, None, None]
    kv[sc.table[0, p // 16], p % 16] = (kv[sc.table[0, p // 16], p % 16].float() * ramp).to(torch.bfloat16)
    d = sc.device()
    lse = torch.empty(sc.T, sc.HQ, device="cuda")
    out = sc.attend(d, lse=lse)
    check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), sc.oracle_attention(), 64)


@pytest.mark.parametrize("split", [True, False])
def test_strided_queries_and_outputs(split):
    sc = Scene([130, 20], [5, 3], 2, 64, 4, 16, False, "padded", seed=11, split=split)
    d = sc.device()
    want = sc.attend(d).clone()
    wide = torch.randn(sc.T, 3, sc.HQ, 64 + 8, device="cuda").to(torch.bfloat16)
    wide[:, 1, :, :64] = d["q"]
    d["q"] = wide[:, 1, :, :64]
    room = torch.full((sc.T, sc.HQ + 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    sc.attend(d, out=room[:, 1:-1])
    assert torch.equal(room[:, 1:-1], want)
    assert (room[:, 0] == 9).all() and (room[:, -1] == 9).all()


def test_rows_behind_the_last_sequence_are_left():
    sc = Scene([30, 40], [2, 3], 2, 64, 2, 16, seed=12)
    d = sc.device()
    want = sc.attend(d).clone()
    d["q"] = torch.cat([d["q"], d["q"][:4]])
    d["parents"] = torch.cat([d["parents"], d["parents"][:4]])
    out = torch.full_like(d["q"], 5.0)
    lse = torch.full((sc.T + 4, sc.HQ), 5.0, device="cuda")
    sc.attend(d, out=out, lse=lse)
    assert torch.equal(out[:sc.T], want) and (out[sc.T:] == 5).all() and (lse[sc.T:] == 5).all()
    assert int(d["err"]) == 0


def test_bad_sequences_are_skipped_and_flagged():
    from short_conv_kv_b200 import binding as b
    sc = Scene([30, 40, 50], [2, 3, 2], 2, 64, 2, 16, kind="chain", seed=13)
    good = sc.attend(sc.device()).clone()

    def run(change, **kw):
        d = sc.device()
        change(d)
        out = torch.full_like(d["q"], 5.0)
        sc.attend(d, out=out, **kw)
        return out, int(d["err"])

    def lens(d):
        d["lens"][1] = -1
    out, flag = run(lens)
    assert flag == b.FLAG_CONTEXT and (out[2:5] == 5).all()
    assert torch.equal(out[:2], good[:2]) and torch.equal(out[5:], good[5:])

    def far(d):
        d["lens"][2] = sc.table.shape[1] * 16 - 1
    out, flag = run(far)
    assert flag == b.FLAG_CONTEXT and (out[5:] == 5).all() and torch.equal(out[:5], good[:5])

    out, flag = run(lambda d: None, max_draft=2)
    assert flag == b.FLAG_TREE and (out[2:5] == 5).all() and torch.equal(out[:2], good[:2])

    def cu(d):
        d["cu"][3] = 99
    out, flag = run(cu)
    assert flag == b.FLAG_CU_SEQLENS and (out[5:] == 5).all() and torch.equal(out[:5], good[:5])

    def parent(d):  # a token that follows itself: unused
        d["parents"][3] = 1
    out, flag = run(parent)
    assert flag == b.FLAG_TREE and torch.equal(out[:3], good[:3]) and (out[3:5] == 0).all()

    def page(d):
        d["table"][1, 0] = sc.pages
    out, flag = run(page)
    assert flag == b.FLAG_SLOT_RANGE
    assert torch.equal(out[:2], good[:2]) and torch.equal(out[5:], good[5:])


def test_other_stream_and_graph():
    sc = Scene([900, 77], [3, 20], 2, 128, 4, 64, False, seed=14)
    d = sc.device()
    from short_conv_kv_b200 import binding as b
    ws = b.tree_attention_workspace(d["q"], d["kv"][0], 2, sc.max_draft)
    ws.random_(0, 255)  # any contents
    want = sc.attend(d).clone()
    out = torch.zeros_like(want)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    sc.attend(d, out=out, workspace=ws, stream=s)
    s.synchronize()
    assert torch.equal(out, want)
    out.zero_()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sc.attend(d, out=out, workspace=ws)
    for k in range(3):  # lengths change between replays
        d["lens"][0] = 900 - 100 * k
        ws.random_(0, 255)
        g.replay()
        torch.cuda.synchronize()
        sc2 = sc.attend(d).clone()
        assert torch.equal(out, sc2)
