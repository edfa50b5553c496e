"""The drafted-tree entry points reject bad arguments before touching the GPU,
and their 64-bit oracle holds to closed forms (CPU only)."""
import ctypes

import numpy as np
import pytest
import torch

from oracle import tree as ot
from short_conv_kv_b200 import binding as b

A = 0x10000  # an aligned address that is never dereferenced


def _paged(**over):
    f = dict(cu_draft=A, parents=A, num_tokens=10, num_seqs=2, max_draft=8, context_lens=A,
             block_table=A, table_width=4, table_stride=4)
    f.update(over)
    p = b.Paged()
    for k, v in f.items():
        setattr(p, k, v)
    return p


def _layout(**over):
    lay = b.cache_layout(16, 16, 2, 64)
    for k, v in over.items():
        setattr(lay, k, v)
    return lay


def _call(name, base, over):
    """One raw call; seqs and layout fields are given as dicts."""
    args = dict(base)
    mx = over.pop("mx", False)
    args.update(over)
    for k, make in (("seqs", _paged), ("layout", _layout)):
        if k in args and args[k] is not None:
            args[k] = ctypes.byref(make(**args[k]))
    vals = []
    for k, v in args.items():
        if k in ("ks", "vs") and not mx:
            continue
        vals.append(v)
    return getattr(b.lib, name + ("_mxfp8" if mx else ""))(*vals)


def attention(**over):
    return _call("sconv_kv_tree_attention", dict(
        q=A, qt=512, qh=64, HQ=8, H=2, D=64, scale=0.1, seqs={}, k=A, ks=A, v=A, vs=A, layout={}, out=A,
        ot=512, oh=64, lse=None, ws=A, wsb=1 << 40, err=None, stream=None), over)


def weights(**over):
    return _call("sconv_kv_attention_weights", dict(
        q=A, qt=512, qh=64, HQ=8, H=2, D=64, scale=0.1, lse=A, seqs={}, k=A, ks=A, layout={}, w=A,
        pos=64, wseq=128, whead=64, err=None, stream=None), over)


def accept(**over):
    return _call("sconv_kv_tree_accept", dict(
        k=A, v=A, rs=128, seqs={}, leaves=A, W=4, H=2, D=64, state=A, rows=None, pool=2, spos=None, kc=A,
        ks=A, vc=A, vs=A, layout={}, w=A, pos=64, wseq=128, whead=64, new=A + 64, err=None, stream=None), over)


def evict(**over):
    return _call("sconv_kv_evict", dict(
        w=A, pos=64, wseq=128, whead=64, seqs={}, keep=20, sinks=2, recent=3, H=2, D=64, kc=A, ks=A, vc=A,
        vs=A, layout={}, kept=A, new=A + 64, wo=None, opos=0, oseq=0, ohead=0, err=None, stream=None), over)


def step(**over):
    return _call("sconv_kv_tree_step", dict(
        k=A, v=A, rs=128, T=10, cu=A, parents=A, S=2, wk=A, wv=A, gk=A, gv=A, eps=1e-6, W=4, H=2, D=64,
        state=A, rows=None, pool=2, slots=A, kc=A, ks=A, vc=A, vs=A, layout={}, options=None, err=None,
        stream=None), over)


NULLS = {attention: ("q", "out", "ws", "k", "v", "layout", "seqs"), weights: ("q", "lse", "w", "k", "layout", "seqs"),
         accept: ("k", "v", "leaves", "new", "kc", "vc", "layout", "seqs", "state"),
         evict: ("w", "kept", "new", "kc", "vc", "layout", "seqs"),
         step: ("k", "v", "cu", "parents", "slots", "kc", "vc", "layout", "wk", "gk", "state")}


@pytest.mark.parametrize("fn", list(NULLS), ids=lambda f: f.__name__)
@pytest.mark.parametrize("mx", [False, True])
def test_null_pointers(fn, mx):
    for n in NULLS[fn]:
        assert fn(**{n: None, "mx": mx}) == b.ERR_NULL, n
    if mx:
        assert fn(ks=None, mx=True) == b.ERR_NULL


PAGED = [attention, weights, accept, evict]


@pytest.mark.parametrize("fn", PAGED, ids=lambda f: f.__name__)
def test_paged_arguments(fn):
    drafted = fn is not evict
    assert fn(seqs=dict(num_seqs=-1)) == b.ERR_SHAPE
    assert fn(seqs=dict(table_width=0)) == b.ERR_SHAPE
    assert fn(seqs=dict(table_stride=3)) == b.ERR_SHAPE
    assert fn(seqs=dict(table_width=1 << 27, table_stride=1 << 27)) == b.ERR_SHAPE  # 2^31 positions
    assert fn(seqs=dict(context_lens=None)) == b.ERR_NULL
    assert fn(seqs=dict(block_table=None)) == b.ERR_NULL
    if drafted:
        assert fn(seqs=dict(num_tokens=-1)) == b.ERR_SHAPE
        assert fn(seqs=dict(max_draft=0)) == b.ERR_SHAPE
        assert fn(seqs=dict(max_draft=129)) == b.ERR_SHAPE
        assert fn(seqs=dict(cu_draft=None)) == b.ERR_NULL
        assert fn(seqs=dict(parents=None)) == b.ERR_NULL
    assert fn(layout=dict(num_pages=0)) == b.ERR_SHAPE
    assert fn(layout=dict(head_dim=128)) == b.ERR_SHAPE
    assert fn(layout=dict(num_kv_heads=4)) == b.ERR_SHAPE
    assert fn(layout=dict(page_size=0)) == b.ERR_SHAPE
    assert fn(layout=dict(stride_page=1 << 45)) == b.ERR_SHAPE
    assert fn(layout=dict(stride_slot=132)) == b.ERR_ALIGN
    assert fn(layout=dict(stride_slot=136), mx=True) == b.ERR_ALIGN
    assert fn(D=96) == b.ERR_SHAPE
    assert fn(H=0) == b.ERR_SHAPE
    # no sequence: nothing enqueued
    assert fn(seqs=dict(num_seqs=0, context_lens=None, cu_draft=None)) == b.OK


def test_attention_arguments():
    assert attention(HQ=7) == b.ERR_SHAPE
    assert attention(HQ=1) == b.ERR_SHAPE
    assert attention(qh=32) == b.ERR_SHAPE
    assert attention(qt=516) == b.ERR_ALIGN
    assert attention(oh=68) == b.ERR_ALIGN
    assert attention(q=A + 8) == b.ERR_ALIGN
    assert attention(out=A + 2) == b.ERR_ALIGN
    assert attention(ws=A + 8) == b.ERR_ALIGN
    assert attention(k=A + 8) == b.ERR_ALIGN
    assert attention(scale=float("nan")) == b.ERR_SHAPE
    assert attention(scale=float("inf")) == b.ERR_SHAPE
    assert attention(seqs=dict(num_tokens=0), q=None, out=None) == b.OK
    need = ctypes.c_int64()
    ws = b.lib.sconv_kv_tree_attention_workspace
    assert ws(2, 8, 8, 2, 64, None) == b.ERR_NULL
    assert ws(-1, 8, 8, 2, 64, ctypes.byref(need)) == b.ERR_SHAPE
    assert ws(2, 129, 8, 2, 64, ctypes.byref(need)) == b.ERR_SHAPE
    assert ws(2, 8, 7, 2, 64, ctypes.byref(need)) == b.ERR_SHAPE
    assert ws(2, 8, 8, 2, 80, ctypes.byref(need)) == b.ERR_SHAPE


def test_weights_arguments():
    assert weights(pos=-1) == b.ERR_SHAPE
    assert weights(wseq=-1) == b.ERR_SHAPE
    assert weights(w=A + 2) == b.ERR_ALIGN
    assert weights(HQ=3) == b.ERR_SHAPE
    assert weights(qt=516) == b.ERR_ALIGN
    assert weights(scale=float("nan")) == b.ERR_SHAPE


def test_accept_arguments():
    assert accept(W=0) == b.ERR_SHAPE
    assert accept(W=9) == b.ERR_SHAPE
    assert accept(rs=64) == b.ERR_SHAPE
    assert accept(pool=-1) == b.ERR_SHAPE
    assert accept(new=A) == b.ERR_SHAPE  # the context lengths themselves
    assert accept(rs=132) == b.ERR_ALIGN
    assert accept(k=A + 8) == b.ERR_ALIGN
    assert accept(state=A + 8) == b.ERR_ALIGN
    assert accept(pos=-1) == b.ERR_SHAPE


def test_evict_arguments():
    assert evict(keep=0) == b.ERR_SHAPE
    assert evict(sinks=-1) == b.ERR_SHAPE
    assert evict(recent=-1) == b.ERR_SHAPE
    assert evict(sinks=10, recent=11) == b.ERR_SHAPE
    assert evict(new=A) == b.ERR_SHAPE
    assert evict(wo=A, opos=64, oseq=128, ohead=64) == b.ERR_SHAPE  # the weights themselves
    assert evict(wo=A + 64, opos=19, oseq=128, ohead=64) == b.ERR_SHAPE
    assert evict(w=A + 2) == b.ERR_ALIGN


def test_step_arguments():
    assert step(W=9) == b.ERR_SHAPE
    assert step(D=96) == b.ERR_SHAPE
    assert step(T=-1) == b.ERR_SHAPE
    assert step(S=-1) == b.ERR_SHAPE
    assert step(rs=64) == b.ERR_SHAPE
    assert step(rs=132) == b.ERR_ALIGN
    assert step(T=0, k=None) == b.OK
    assert step(S=0, k=None) == b.OK
    o = b.Options()
    o.gamma_head_stride = 32
    assert step(options=ctypes.byref(o)) == b.ERR_SHAPE


def test_binding_checks():
    """The front end's own refusals, on CPU tensors (none reaches the library)."""
    z = torch.zeros
    i32 = torch.int32
    q, lens, table = z(3, 4, 64, dtype=torch.bfloat16), z(2, dtype=i32), z(2, 4, dtype=i32)
    cu, par = z(3, dtype=i32), z(3, dtype=i32)
    kc = z(8, 16, 2, 64, dtype=torch.bfloat16)
    ok = dict(q=q, cu_draft=cu, parents=par, context_lens=lens, block_table=table, k_cache=kc, v_cache=kc,
              scale=1.0, max_draft=2)

    def refused(err, fn=b.tree_attention, base=ok, **over):
        with pytest.raises(err):
            fn(**{**base, **over})

    refused(ValueError, out=torch.empty_like(q), workspace=z(8, dtype=torch.uint8))  # not on a GPU
    refused(TypeError, q=q.float())
    refused(ValueError, q=z(3, 4, 128, dtype=torch.bfloat16))
    refused(TypeError, cu_draft=cu.long())
    refused(ValueError, cu_draft=cu[:2])
    refused(ValueError, parents=par[:2])
    refused(TypeError, block_table=table.long())
    refused(ValueError, context_lens=lens[:1])
    refused(TypeError, k_cache=kc.half(), v_cache=kc.half())
    refused(ValueError, v_cache=kc[:, :8])
    refused(ValueError, lse=z(3, 5))
    refused(TypeError, lse=z(3, 4, dtype=torch.float64))
    refused(ValueError, out=q[:2])
    w = z(2, 2, 64)
    ev = dict(weights=w, context_lens=lens, block_table=table, k_cache=kc, v_cache=kc, sinks=1, recent=1,
              kept=z(2, 2, 9, dtype=i32), new_lens=lens.clone())
    refused(ValueError, b.evict, ev)
    refused(TypeError, b.evict, ev, weights=w.half())
    refused(ValueError, b.evict, ev, weights=w[:1])
    refused(ValueError, b.evict, ev, kept=z(2, 3, 9, dtype=i32))
    refused(TypeError, b.evict, ev, new_lens=z(2))
    raw = z(3, 128, dtype=torch.bfloat16)
    ac = dict(k=raw, v=raw, cu_draft=cu, parents=par, leaves=lens, context_lens=lens, block_table=table, W=4,
              conv_state=z(2, 3, 256, dtype=torch.bfloat16), k_cache=kc, v_cache=kc, new_lens=lens.clone())
    refused(ValueError, b.tree_accept, ac)
    refused(ValueError, b.tree_accept, ac, W=3)
    refused(ValueError, b.tree_accept, ac, leaves=lens[:1])
    refused(TypeError, b.tree_accept, ac, state_indices=lens.long())


# ------------------------------------------------------------------- the oracle

def test_oracle_paths():
    assert ot.paths([-1, 0, 0, 2, -1, 4]) == [[0], [0, 1], [0, 2], [0, 2, 3], [4], [4, 5]]
    assert ot.paths([-1, -2, 1, 3, 9, -5]) == [[0], [], [], [], [], []]


def test_oracle_attention_closed_forms():
    rng = np.random.default_rng(0)
    k, v = rng.standard_normal((3, 4, 1, 8)), rng.standard_normal((3, 4, 1, 8))
    table, cu = np.array([[2, 0, 1]]), [0, 2]
    q = np.zeros((2, 2, 8))
    out, lse, _, _ = ot.attention(q, cu, [-1, -1], [5], table, k, v, 1.0)  # equal scores: means
    rows = ot.rows_of(v, table[0], np.arange(7), 4)[:, 0]
    assert np.allclose(out[0, 0], rows[:6].mean(0)) and np.allclose(lse, np.log(6))
    assert np.allclose(out[1, 1], (rows[:5].sum(0) + rows[6]) / 6)
    q[0, 0] = 1e4 * ot.rows_of(k, table[0], [3], 4)[0, 0]  # a single winner
    out, _, _, _ = ot.attention(q, cu, [-1, -2], [5], table, k, v, 1.0)
    s = ot.rows_of(k, table[0], np.arange(6), 4)[:, 0] @ q[0, 0]
    assert np.allclose(out[0, 0], rows[s.argmax()]) and (out[1] == 0).all()


def test_oracle_weights_sum_to_one():
    rng = np.random.default_rng(1)
    k = rng.standard_normal((4, 4, 2, 8))
    q, table, cu, par = rng.standard_normal((3, 4, 8)), np.array([[3, 1, 0]]), [0, 3], [-1, 0, 0]
    _, lse, _, _ = ot.attention(q, cu, par, [6], table, k, k, 0.3)
    w, _ = ot.weights(q, lse, cu, par, [6], table, k, 0.3, np.zeros((1, 2, 12)))
    assert np.allclose(w.sum(2), 3 * 2)  # tokens times query heads a K/V head


def test_oracle_mx_values():
    codes = torch.arange(256, dtype=torch.uint8)
    assert np.array_equal(ot.e4m3_values(codes.numpy()), codes.view(torch.float8_e4m3fn).double().numpy(),
                          equal_nan=True)
    assert ot.mx_values(np.full((1, 64), 0x38, np.uint8), np.array([[127, 130]], np.uint8)).sum() == 32 * 9


def test_oracle_evict():
    w = np.array([1, 9, 3, 3, 3, 0, np.nan, 5.0])
    assert ot.evict_pick(w, 8, 4, 1, 1) == [0, 1, 6, 7]
    assert ot.evict_pick(w, 8, 5, 0, 1) == [1, 2, 3, 6, 7]  # ties: the lower position
    assert ot.evict_pick(w, 3, 4, 1, 1) == [0, 1, 2]


# ------------------------------------------------- rows that overlap in memory

def test_binding_refuses_overlapping_rows():
    """Broadcast inputs, whose stride the kernels could not follow, are refused (CPU
    tensors: none reaches the library)."""
    z, i32, bf = torch.zeros, torch.int32, torch.bfloat16
    lens, cu, par = z(2, dtype=i32), z(3, dtype=i32), z(3, dtype=i32)
    kc, table = z(8, 16, 2, 64, dtype=bf), z(2, 4, dtype=i32)
    q, w, raw = z(3, 4, 64, dtype=bf), z(2, 2, 64), z(3, 128, dtype=bf)

    def refused(fn, **kw):
        with pytest.raises(ValueError, match="overlap"):
            fn(**kw)
    at = dict(cu_draft=cu, parents=par, context_lens=lens, k_cache=kc, scale=1.0, max_draft=2)
    refused(b.tree_attention, q=q, v_cache=kc, block_table=table[:1].expand(2, 4), **at)
    refused(b.attention_weights, q=q, lse=z(3, 4), block_table=table, weights=w[:1].expand(2, 2, 64), **at)
    refused(b.attention_weights, q=q, lse=z(3, 4), block_table=table, weights=w[:, :1].expand(2, 2, 64), **at)
    refused(b.evict, weights=w[:1].expand(2, 2, 64), context_lens=lens, block_table=table, k_cache=kc,
            v_cache=kc, sinks=1, recent=1, kept=z(2, 2, 9, dtype=i32), new_lens=lens.clone())
    one = raw[:1].expand(3, 128)
    refused(b.tree_accept, k=one, v=one, cu_draft=cu, parents=par, leaves=lens, context_lens=lens,
            block_table=table, W=1, conv_state=None, k_cache=kc, v_cache=kc, new_lens=lens.clone())
    refused(b.tree_step, k=one, v=one, cu_draft=cu, parents=par, conv_w_k=z(1, 128, dtype=bf),
            conv_w_v=z(1, 128, dtype=bf), gamma_k=z(64), gamma_v=z(64), eps=1e-6, conv_state=None,
            slot_mapping=z(3, dtype=torch.int64), k_cache=kc, v_cache=kc)


def test_evict_keep_limit():
    assert evict(keep=2 ** 31 - 65536) == b.ERR_SHAPE
