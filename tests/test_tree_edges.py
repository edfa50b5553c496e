"""The drafted-tree calls at the edges of their arguments (CPU only: none touches a GPU)."""
from short_conv_kv_b200 import binding as b
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
