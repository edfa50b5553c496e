"""The drafted-tree calls at the edges of their arguments (CPU only: none touches a GPU)."""
import os
import random
import subprocess
import sys

import pytest
import torch

from short_conv_kv_b200 import binding as b
from short_conv_kv_b200 import build
from tests import test_tree_abi as abi


def test_accept_without_drafted_tokens_needs_no_token_tensor():
    """Empty tensors may have NULL pointers; with tokens they are still required."""
    none = dict(num_tokens=0, parents=None)
    for mx in (False, True):
        assert abi.accept(seqs=dict(none, context_lens=None), k=None, v=None, mx=mx) == b.ERR_NULL
        assert abi.accept(seqs=dict(none, cu_draft=None), k=None, v=None, mx=mx) == b.ERR_NULL
        # past the pointer checks: the next fault is what is reported
        assert abi.accept(seqs=none, k=None, v=None, W=9, mx=mx) == b.ERR_SHAPE
        assert abi.accept(seqs=dict(none, num_tokens=1), k=None, v=None, W=9, mx=mx) == b.ERR_NULL
        assert abi.accept(seqs=dict(none, num_tokens=1), W=9, mx=mx) == b.ERR_NULL


def test_too_many_tiles_for_the_join_are_refused_before_any_launch():
    """2^31 - 1 sequences with two row tiles each: refused with the other shapes, where nothing has been
    launched yet (without a GPU, a launch or a query of one would be ERR_CUDA)."""
    many = 2 ** 31 - 1
    assert abi.attention(seqs=dict(num_seqs=many, max_draft=128)) == b.ERR_SHAPE
    assert abi.attention(seqs=dict(num_seqs=many, max_draft=128), mx=True) == b.ERR_SHAPE


WITHOUT_MODULE = """
import sys
import torch
from short_conv_kv_b200 import build
build.TREE = build.TREE + ".absent"
from short_conv_kv_b200 import binding as b
assert b.version() > 0 and b.cache_layout(4, 16, 2, 64).head_dim == 64
assert "short_conv_kv_b200._tree" not in sys.modules
for _ in range(2):
    try:
        b.evict(*[torch.zeros(1)] * 5, 0, 0, torch.zeros(1, 1, 1), torch.zeros(1))
    except ImportError as e:
        assert "not built" in str(e)
    else:
        raise AssertionError("no error")
build.TREE = build.TREE[:-len(".absent")]
try:
    b.evict(*[torch.zeros(1)] * 5, 0, 0, torch.zeros(1, 1, 1), torch.zeros(1))
except TypeError:
    print("fine")
"""


def test_the_steps_own_calls_do_without_the_marshalling_module():
    """Where _tree.so is missing, the binding loads; the first call that needs the module says so."""
    got = subprocess.run([sys.executable, "-c", WITHOUT_MODULE], capture_output=True, text=True, cwd=build.ROOT)
    assert got.returncode == 0 and got.stdout.strip() == "fine", got.stderr


def test_a_missing_or_old_marshalling_module_needs_a_build(tmp_path, monkeypatch):
    lib, tree, src = tmp_path / "lib.so", tmp_path / "_tree.so", tmp_path / "tree_bind.cpp"
    for f in (lib, tree, src):
        f.write_text("")
    at = max(os.path.getmtime(d) for d in build.DEPS)
    for f, age in ((src, 0), (lib, 10), (tree, 10)):
        os.utime(f, (at + age, at + age))
    for name, f in (("LIB", lib), ("TREE", tree), ("TREE_SOURCE", src)):
        monkeypatch.setattr(build, name, str(f))
    assert not build.needs_build(str(lib))
    os.utime(src, (at + 20, at + 20))
    assert build.needs_build(str(lib))
    os.utime(src, (at, at))
    tree.unlink()
    assert build.needs_build(str(lib))
    other = tmp_path / "other.so"  # a library elsewhere has no module beside it
    other.write_text("")
    os.utime(other, (at + 10, at + 10))
    assert not build.needs_build(str(other))


def _strided(sizes, strides, dtype):
    """A view of those strides, which may overlap."""
    room = 1 + sum(max(n - 1, 0) * s for n, s in zip(sizes, strides))
    return torch.zeros(room, dtype=dtype).as_strided(sizes, strides)


def _overlaps(n1, s1, n2, s2, length):
    seen = [i * s1 + j * s2 + e for i in range(n1) for j in range(n2) for e in range(length)]
    return len(set(seen)) < len(seen)


def test_overlapping_rows_are_refused_and_others_not():
    """Weights and outputs whose rows share elements in any way would be written by several warps at once.  CPU
    tensors: a layout that is accepted meets the device check instead."""
    rng = random.Random(3)
    i32, bf = torch.int32, torch.bfloat16
    counts = [0, 0]
    for _ in range(3000):
        S, H, n = rng.randint(1, 6), rng.randint(1, 6), rng.randint(0, 9)
        st = (rng.randint(0, 40), rng.randint(0, 40))
        w = _strided((S, H, n), (*st, 1), torch.float32)
        bad = _overlaps(S, st[0], H, st[1], n)
        counts[bad] += 1
        with pytest.raises(ValueError, match="overlap" if bad else "CUDA device"):
            b.attention_weights(torch.zeros(3, H, 64, dtype=bf), torch.zeros(3, H), torch.zeros(S + 1, dtype=i32),
                                torch.zeros(3, dtype=i32), torch.zeros(S, dtype=i32), torch.zeros(S, 4, dtype=i32),
                                torch.zeros(8, 16, H, 64, dtype=bf), 1.0, 2, w)
    assert min(counts) > 500
    q, cu, par = torch.zeros(3, 4, 64, dtype=bf), torch.zeros(3, dtype=i32), torch.zeros(3, dtype=i32)
    kc, lens, table = torch.zeros(8, 16, 2, 64, dtype=bf), torch.zeros(2, dtype=i32), torch.zeros(2, 4, dtype=i32)
    for st, bad in (((256, 64), 0), ((64, 192), 0), ((64, 200), 0), ((128, 64), 1), ((64, 64), 1), ((64, 128), 1),
                    ((72, 8), 1), ((144, 72), 1), ((216, 72), 1), ((72, 216), 0), ((288, 72), 0), ((192, 128), 1),
                    ((320, 128), 0), ((448, 128), 0), ((8, 256), 1)):
        with pytest.raises(ValueError, match="overlap" if bad else "CUDA device"):
            b.tree_attention(q, cu, par, lens, table, kc, kc, 1.0, 2, out=_strided((3, 4, 64), (*st, 1), bf),
                             workspace=torch.zeros(8, dtype=torch.uint8))


def test_accept_refuses_lengths_written_over_the_leaves():
    """A sequence's blocks read its leaf while the first of them writes its length."""
    for mx in (False, True):
        assert abi.accept(leaves=abi.A + 64, mx=mx) == b.ERR_SHAPE  # new_lens' address
