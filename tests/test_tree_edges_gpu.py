"""The drafted-tree operators at the edges of what their documentation allows."""
import pytest
import torch

from short_conv_kv_b200 import binding as b
from tests.tree_util import Scene

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
