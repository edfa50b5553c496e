"""The drafted-tree operators where they are split over the GPU: contexts that many
CTAs share, more query rows than a tensor-core tile, long evictions, and whole
serving steps captured into a graph."""
import numpy as np
import pytest
import torch

from oracle import tree as ot
from short_conv_kv_b200 import binding as b
from tests.test_tree_ops_gpu import _weigh
from tests.tree_util import Scene, check_attention, logit_error

pytestmark = pytest.mark.gpu

LONG = [
    # lens, drafts, H, D, group, page, kind
    ([7000], [3], 2, 128, 8, 64, "padded"),       # 24 rows: one unit cut into many parts
    ([5000, 129, 2600], [16, 9, 2], 1, 64, 4, 16, "padded"),
    ([3000, 1], [50, 5], 2, 128, 4, 64, "tree"),  # 200 rows: a pair of streams; beside 20
    ([1500], [128], 1, 128, 5, 7, "padded"),      # 640 rows: three units, the last of 128
    ([4000, 300], [6, 40], 1, 256, 4, 48, "padded"),
    ([128, 127, 255, 256, 257], [17, 18, 33, 64, 65], 1, 128, 2, 64, "tree"),  # tiles' edges
    ([6000], [1], 1, 128, 1, 64, "chain"),        # few rows, many parts
]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("case", range(len(LONG)))
def test_attention(case, mx):
    lens, drafts, H, D, group, page, kind = LONG[case]
    sc = Scene(lens, drafts, H, D, group, page, mx, kind, seed=300 + case)
    d = sc.device()
    lse = torch.empty(sc.T, sc.HQ, device="cuda")
    out = sc.attend(d, lse=lse)
    assert int(d["err"]) == 0
    check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), sc.oracle_attention(), D,
                    str(LONG[case]))


@pytest.mark.parametrize("scale", [-0.11, 0.0, 3e-5])
@pytest.mark.parametrize("mx", [False, True])
def test_scales_of_any_sign(scale, mx):
    sc = Scene([500, 90], [20, 30], 2, 128, 3, 64, mx, "padded", seed=320)
    sc.scale = scale
    d = sc.device()
    lse = torch.empty(sc.T, sc.HQ, device="cuda")
    out = sc.attend(d, lse=lse)
    check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), sc.oracle_attention(), 128)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_growing_scores(D):
    """Scores that keep growing: every tile's maximum passes the one before by more than
    the outputs are allowed to lag."""
    sc = Scene([1900], [30], 1, D, 5, 16, False, "tree", seed=330)
    sc.q *= 40
    p = np.arange(1930)
    kv = sc._pick(sc.store[0], 0)
    at = (sc.table[0, p // 16], p % 16)
    kv[at] = (kv[at].float() * torch.linspace(0.01, 3, 1930)[:, None, None]).to(torch.bfloat16)
    d = sc.device()
    lse = torch.empty(sc.T, sc.HQ, device="cuda")
    out = sc.attend(d, lse=lse)
    check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), sc.oracle_attention(), D)


@pytest.mark.parametrize("n", [2, 20])
def test_scale_bytes_of_any_size(n):
    """MXFP8 scales from the smallest to beyond those of the fast decoding."""
    sc = Scene([300], [n], 2, 128, 4, 16, True, "chain", seed=340)
    gen = torch.Generator().manual_seed(7)
    scales = sc.store[1]
    for half, values in ((0, [0, 100, 118, 119]), (1, [0, 1, 60, 127, 133, 134, 135, 136, 150])):
        s = sc._pick(scales, half)
        held = s != 0xFF
        pick = torch.tensor(values, dtype=torch.uint8)[torch.randint(0, len(values), s.shape, generator=gen)]
        s[held] = pick[held]
    d = sc.device()
    lse = torch.empty(sc.T, sc.HQ, device="cuda")
    out = sc.attend(d, lse=lse)
    check_attention(out.double().cpu().numpy(), lse.double().cpu().numpy(), sc.oracle_attention(), 128)


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("n", [2, 20])
def test_nonfinite_context(n, mx):
    """A NaN in one cached V element reaches that element of that head's rows, a NaN
    in a K row all of its head's, and nothing else."""
    sc = Scene([400], [n], 2, 128, 4, 16, mx, "chain", seed=350)
    d = sc.device()
    clean = sc.attend(d)
    pg, off = int(sc.table[0, 200 // 16]), 200 % 16
    k, v = d["kv"][0], d["kv"][2 if mx else 1]
    keep = v[pg, off, 0, 5].clone()
    v[pg, off, 0, 5] = 0x7F if mx else float("nan")
    got = sc.attend(d)
    assert torch.isnan(got[:, :4, 5]).all()
    rest = torch.ones_like(got, dtype=torch.bool)
    rest[:, :4, 5] = False
    assert torch.equal(got[rest], clean[rest])
    v[pg, off, 0, 5] = keep
    k[pg, off, 1, 77] = 0xFF if mx else float("nan")
    got = sc.attend(d)
    assert torch.isnan(got[:, 4:]).all() and torch.equal(got[:, :4], clean[:, :4])


WEIGHTS = [
    ([6000, 700], [1, 4], 2, 128, 4, 64, "chain"),    # few rows
    ([5000, 40, 300], [9, 30, 3], 1, 64, 4, 16, "padded"),
    ([900], [100], 1, 128, 6, 64, "padded"),          # 600 rows: three passes
    ([260, 1300], [128, 65], 2, 128, 2, 48, "tree"),  # 256 rows: one full pass
    ([700], [40], 1, 256, 3, 64, "padded"),
]


@pytest.mark.parametrize("mx", [False, True])
@pytest.mark.parametrize("case", range(len(WEIGHTS)))
def test_weights(case, mx):
    lens, drafts, H, D, group, page, kind = WEIGHTS[case]
    sc = Scene(lens, drafts, H, D, group, page, mx, kind, seed=360 + case)
    d = sc.device()
    lse = torch.empty(sc.T, sc.HQ, device="cuda")
    sc.attend(d, lse=lse)
    room = max(c + n for c, n in zip(lens, drafts))
    w0 = torch.rand(sc.S, H, room, device="cuda")
    first = None
    for _ in range(3):  # the same bits each time
        w = w0.clone()
        _weigh(sc, d, lse, w)
        assert first is None or torch.equal(w, first)
        first = w
    assert int(d["err"]) == 0
    with np.errstate(invalid="ignore"):
        want, size = ot.weights(sc.q.double().numpy(), lse.double().cpu().numpy(), sc.cu, sc.parents, lens,
                                sc.table, sc.values(0), sc.scale, w0.cpu().numpy())
    old = w0.double().cpu().numpy()
    # as in test_tree_ops_gpu.test_weights: every term's exponent, then up to 2^10 additions
    fin = lse[lse > -1e30].abs().max().item()
    e = logit_error(size, D) + 2.0 ** -22 * (2 + fin) + 2.0 ** -14
    bound = e * np.abs(want - old) + e * np.abs(want) * (want != old) + 2.0 ** -23 * np.abs(want)
    assert (np.abs(first.double().cpu().numpy() - want) <= bound).all()


@pytest.mark.parametrize("values", ["random", "equal"])
@pytest.mark.parametrize("length, keep, D, mx", [(70000, 20000, 64, True), (9001, 9000, 128, False),
                                                 (420000, 30000, 64, False)])
def test_evict(length, keep, D, mx, values):
    """A single long context: clusters of CTAs; the last one's slices are larger than
    what shared memory holds."""
    page, sinks, recent = 64, 4, 100
    pages = -(-length // page)
    gen = torch.Generator(device="cuda").manual_seed(9)
    table = torch.randperm(pages, generator=gen, device="cuda").to(torch.int32)[None]
    shape = (pages, page, 1, D)
    if mx:
        kv = [torch.randint(0, 255, s, generator=gen, device="cuda", dtype=torch.uint8)
              for s in (shape, (*shape[:3], D // 32)) * 2]
    else:
        kv = [torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2)]
    if values == "random":
        w = (torch.rand(1, 1, length, generator=gen, device="cuda") ** 6 * 4096).floor()
    else:
        w = torch.full((1, 1, length), 0.5, device="cuda")
    order = torch.sort(w[0, 0, sinks:length - recent], descending=True, stable=True)[1] + sinks
    pick = torch.cat([torch.arange(sinks, device="cuda"), order[:keep - sinks - recent],
                      torch.arange(length - recent, length, device="cuda")]).sort()[0]
    want = []
    for t in kv:
        flat = t[table[0].long()].flatten(0, 1)[:length]
        moved = flat.clone()
        moved[:keep] = flat[pick]
        want.append(moved)
    kept = torch.empty(1, 1, keep, dtype=torch.int32, device="cuda")
    new, err = torch.empty(1, dtype=torch.int32, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda")
    out = torch.zeros(1, 1, keep, device="cuda")
    lens = torch.tensor([length], dtype=torch.int32, device="cuda")
    (b.evict_mxfp8 if mx else b.evict)(w, lens, table, *kv, sinks, recent, kept, new, out, err_flag=err)
    assert int(err) == 0 and int(new) == keep
    assert torch.equal(kept[0, 0].long(), pick) and torch.equal(out[0, 0], w[0, 0, pick])
    for t, m in zip(kv, want):
        assert torch.equal(t[table[0].long()].flatten(0, 1)[:length], m)


def test_workspace_serves_smaller_calls():
    big = Scene([300, 50, 20], [100, 3, 1], 2, 128, 4, 16, seed=380)
    ws = b.tree_attention_workspace(big.q.cuda(), big.device()["kv"][0], 3, 128)
    for drafts in ([100, 3, 1], [6, 1, 4], [2, 2, 1], [1, 1, 1]):
        sc = Scene([300, 50, 20], drafts, 2, 128, 4, 16, seed=381)
        d = sc.device()
        assert torch.equal(sc.attend(d, workspace=ws), sc.attend(d))


@pytest.mark.parametrize("mx", [False, True])
def test_captured_serving_step(mx):
    """Step, attention, weights, acceptance and eviction in one graph, replayed, against
    the same calls one by one."""
    H, D, page, g, W = 2, 128, 16, 4, 4
    sc = Scene([400, 77, 210], [7, 7, 7], H, D, g, page, mx, "tree", seed=390)
    gen = torch.Generator(device="cuda").manual_seed(3)
    d = sc.device()
    C = H * D
    rnd = lambda *s: torch.randn(*s, generator=gen, device="cuda").to(torch.bfloat16)  # noqa: E731
    raw, wk, state0 = rnd(2, sc.T, C), rnd(2, W, C), rnd(3, W - 1, 2 * C)
    gk = torch.ones(D, device="cuda")
    pos = np.concatenate([c + np.arange(7) for c in sc.lens])
    seq = np.repeat(np.arange(3), 7)
    slots = torch.from_numpy(sc.table[seq, pos // page].astype(np.int64) * page + pos % page).cuda()
    leaves = torch.tensor([6, 3, -1], dtype=torch.int32, device="cuda")
    room = 420
    store0 = [t.clone() for t in d["kv"]]
    w0 = torch.rand(3, H, room, generator=gen, device="cuda")
    fn = {n: getattr(b, n + ("_mxfp8" if mx else "")) for n in
          ("tree_step", "tree_attention", "attention_weights", "tree_accept", "evict")}
    kv, ws = d["kv"], b.tree_attention_workspace(d["q"], d["kv"][0], 3, 7)
    bufs = dict(state=state0.clone(), w=w0.clone(), wo=torch.zeros_like(w0), out=torch.zeros_like(d["q"]),
                lse=torch.zeros(sc.T, sc.HQ, device="cuda"),
                kept=torch.zeros(3, H, 100, dtype=torch.int32, device="cuda"),
                l1=torch.zeros(3, dtype=torch.int32, device="cuda"),
                l2=torch.zeros(3, dtype=torch.int32, device="cuda"))

    def reset():
        for t, s in zip(kv, store0):
            t.copy_(s)
        bufs["state"].copy_(state0)
        bufs["w"].copy_(w0)
        for n in ("wo", "out", "lse", "kept", "l1", "l2"):
            bufs[n].zero_()

    def steps():
        x = bufs
        fn["tree_step"](raw[0], raw[1], d["cu"], d["parents"], wk[0], wk[1], gk, gk, 1e-6, x["state"], slots, *kv,
                        err_flag=d["err"])
        fn["tree_attention"](d["q"], d["cu"], d["parents"], d["lens"], d["table"], *kv, sc.scale, 7, x["out"],
                             x["lse"], ws, d["err"])
        fn["attention_weights"](d["q"], x["lse"], d["cu"], d["parents"], d["lens"], d["table"],
                                *kv[:2 if mx else 1], sc.scale, 7, x["w"], d["err"])
        fn["tree_accept"](raw[0], raw[1], d["cu"], d["parents"], leaves, d["lens"], d["table"], W, x["state"], *kv,
                          x["l1"], weights=x["w"], err_flag=d["err"])
        fn["evict"](x["w"], x["l1"], d["table"], *kv, 2, 16, x["kept"], x["l2"], x["wo"], d["err"])

    steps()  # kernels loaded before the capture
    reset()
    steps()
    want = {n: t.clone() for n, t in bufs.items()}
    cache = [t.clone() for t in kv]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        steps()
    for _ in range(3):
        reset()
        graph.replay()
        torch.cuda.synchronize()
        for n, t in bufs.items():
            assert torch.equal(t, want[n]), n
        for t, s in zip(kv, cache):
            assert torch.equal(t.view(torch.uint8), s.view(torch.uint8))
    assert int(d["err"]) == 0


@pytest.mark.parametrize("mx", [False, True])
def test_two_calls_at_once(mx):
    """Different calls overlapping on two streams, each with a workspace of its own."""
    scenes = [Scene([3000, 50], [20, 3], 2, 128, 4, 64, mx, "padded", seed=400),
              Scene([900, 1700, 4], [1, 2, 1], 2, 128, 4, 16, mx, "chain", seed=401)]
    devs = [sc.device() for sc in scenes]
    want = [sc.attend(d) for sc, d in zip(scenes, devs)]
    ws = [b.tree_attention_workspace(d["q"], d["kv"][0], sc.S, sc.max_draft) for sc, d in zip(scenes, devs)]
    streams = [torch.cuda.Stream() for _ in scenes]
    outs = [[torch.zeros_like(w) for _ in range(8)] for w in want]
    torch.cuda.synchronize()
    for r in range(8):
        for sc, d, w, s, o in zip(scenes, devs, ws, streams, outs):
            sc.attend(d, out=o[r], workspace=w, stream=s)
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(x, w) for x in o)
