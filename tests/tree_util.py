"""Scenarios of the drafted-tree operators: seeded sequences over a paged
cache, on the host and on the device."""
import numpy as np
import torch

from oracle import tree as ot

SENTINEL = 0x7FC1


def make_tree(rng, n, kind):
    if kind == "chain":
        return [j - 1 for j in range(n)]
    if kind == "star":
        return [-1] * n
    pad = int(rng.integers(0, n // 4 + 1)) if kind == "padded" else 0
    par = [int(rng.integers(max(-1, j - 5), j)) for j in range(n - pad)]
    return par + [int(rng.integers(-9, -1)) for _ in range(pad)]


class Scene:
    """Sequences with their cache.  `lens` cached tokens and `drafts` drafted
    ones each; K and V are the halves of one buffer a page (`split`) or two
    buffers.  Rows that no sequence holds are NaN."""

    def __init__(self, lens, drafts, H=2, D=64, group=4, page=16, mx=False, kind="padded", seed=0,
                 split=True, extra_pages=3, width_extra=1):
        rng = self.rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed + 1)
        self.H, self.D, self.page, self.mx, self.group, self.HQ = H, D, page, mx, group, H * group
        self.lens, self.drafts, self.S = list(lens), list(drafts), len(lens)
        self.cu = np.concatenate([[0], np.cumsum(drafts)]).astype(np.int32)
        self.T = int(self.cu[-1])
        self.parents = np.array([p for n in drafts for p in make_tree(rng, n, kind)], np.int32)
        need = [-(-(c + n) // page) + width_extra for c, n in zip(lens, drafts)]
        self.pages = sum(need) + extra_pages
        perm = rng.permutation(self.pages)
        self.table = np.full((self.S, max(need + [1])), 0, np.int32)
        at = 0
        for i, m in enumerate(need):
            self.table[i, :m] = perm[at:at + m]
            self.table[i, m:] = perm[at]
            at += m
        self.scale = D ** -0.5
        shape = (self.pages, 2, page, H, D) if split else (2, self.pages, page, H, D)
        if mx:
            codes = torch.full(shape, 0xFF, dtype=torch.uint8)
            scales = torch.full(shape[:-1] + (D // 32,), 0xFF, dtype=torch.uint8)
        else:
            kv = torch.full(shape, SENTINEL, dtype=torch.int16)
        for i in range(self.S):
            p = np.arange(self.lens[i] + self.drafts[i])
            used = np.ones(len(p), bool)
            for j, path in enumerate(ot.paths(self.parents[self.cu[i]:self.cu[i + 1]])):
                used[self.lens[i] + j] = bool(path)
            pg, off = self.table[i, p // page], p % page
            for half in range(2):
                z = torch.randn(len(p), H, D, generator=gen)
                idx = (pg, half, off) if split else (half, pg, off)
                if mx:
                    c = torch.randint(0, 127, (len(p), H, D), generator=gen, dtype=torch.uint8)
                    c |= torch.randint(0, 2, c.shape, generator=gen, dtype=torch.uint8) * 128
                    e = torch.randint(116, 120, (len(p), H, D // 32), generator=gen, dtype=torch.uint8)
                    c[~used], e[~used] = 0xFF, 0xFF
                    codes[idx], scales[idx] = c, e
                else:
                    b = z.to(torch.bfloat16).view(torch.int16)
                    b[~used] = SENTINEL
                    kv[idx] = b
        pick = (lambda t, h: t[:, h]) if split else (lambda t, h: t[h])
        self._pick, self.split = pick, split
        self.store = (codes, scales) if mx else (kv.view(torch.bfloat16),)
        self.q = torch.randn(self.T, self.HQ, D, generator=gen).to(torch.bfloat16)

    @property
    def max_draft(self):
        return max(self.drafts + [1])

    def values(self, half):
        """The K (0) or V (1) cache as float64."""
        if self.mx:
            return ot.mx_values(self._pick(self.store[0], half).numpy(),
                                self._pick(self.store[1], half).numpy())
        return self._pick(self.store[0], half).double().numpy()

    def device(self, device="cuda"):
        """Device tensors: cache parts in the binding's order, and the rest."""
        st = [t.to(device) for t in self.store]
        if self.mx:
            kv = (self._pick(st[0], 0), self._pick(st[1], 0), self._pick(st[0], 1), self._pick(st[1], 1))
        else:
            kv = (self._pick(st[0], 0), self._pick(st[0], 1))
        dev = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(device)  # noqa: E731
        return dict(kv=kv, q=self.q.to(device), cu=dev(self.cu), parents=dev(self.parents),
                    lens=dev(np.array(self.lens, np.int32)), table=dev(self.table),
                    err=torch.zeros(1, dtype=torch.int32, device=device))

    def attend(self, d, out=None, lse=None, workspace=None, stream=None, max_draft=None):
        from short_conv_kv_b200 import binding as b
        fn = b.tree_attention_mxfp8 if self.mx else b.tree_attention
        return fn(d["q"], d["cu"], d["parents"], d["lens"], d["table"], *d["kv"], self.scale,
                  max_draft or self.max_draft, out, lse, workspace, d["err"], stream)

    def oracle_attention(self):
        with np.errstate(invalid="ignore"):
            return ot.attention(self.q.double().numpy(), self.cu, self.parents, self.lens, self.table,
                                self.values(0), self.values(1), self.scale)


def logit_error(size, D):
    """Bound of a score's error, in nats: D products exact in fp32, summed in
    some order with at most D + 8 roundings (the tensor cores truncate: a whole
    step, 2^-23, each), then the factor scale * log2(e) (2 roundings)."""
    return (D + 12) * 2.0 ** -23 * size


def check_attention(out, lse, ref, D, what=""):
    """Bound, per element: the output's rounding 2^-8 |o|; every probability's
    rounding to bf16, 2^-8 sum p|v| at most; both scores' errors in numerator and
    denominator (a relative 2 * logit_error each way), ex2's 2^-22, and sums
    of up to 2^13 fp32 additions, 2^-24 each, at 2 sum p|v|."""
    o, l, mag, size = ref
    e = logit_error(size, D)[..., None] + 2.0 ** -22 + 2.0 ** -11
    bound = 2.0 ** -8 * (np.abs(o) + mag) * 1.01 + 2 * e * mag + 1e-30
    err = np.abs(out - o)
    assert np.all(np.isfinite(out)), f"{what}: non-finite output"
    worst = (err / bound).max() if err.size else 0.0
    assert worst <= 1, f"{what}: output error {worst:.3f} of its bound"
    if lse is not None:
        fin = np.isfinite(l)
        assert np.array_equal(lse[~fin], l[~fin]), f"{what}: lse of empty rows"
        lb = logit_error(size, D) + 2.0 ** -22 + 2.0 ** -11 * 2.0 ** -10 + 2.0 ** -22 * np.abs(np.where(fin, l, 0))
        lw = (np.abs(lse[fin] - l[fin]) / lb[fin]).max() if fin.any() else 0.0
        assert lw <= 1, f"{what}: lse error {lw:.3f} of its bound"
    return worst
