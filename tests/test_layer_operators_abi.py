"""The delta rule, the block's norms and the embedding without a GPU: their entry points refuse what they cannot take before any
CUDA call (no pointer below is ever dereferenced), and the binding refuses CPU tensors and wrong shapes."""

import ctypes

import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from sparse_slot_memory_gb300 import _abi

A = 0x100000   # an aligned address that nothing reads
L = 1 << 21    # between rows


@pytest.fixture(scope="module")
def lib():
    sdm.build()
    return _abi.load()


def gdr(**kw):
    base = dict(P=2, k_heads=2, v_heads=4, dk=64, dv=32, x_dtype=1, g_dtype=0, scale=1.0, rows=64)
    base.update(kw)
    return ctypes.byref(_abi.GdrShape(**base))


def gdr_forward(lib, s, n=None, **kw):
    """The forward's call with every array at A, but for those named."""
    a = dict(q=A, q_ld=L, k=A, k_ld=L, v=A, v_ld=L, g=A, g_ld=L, beta=A, beta_ld=L, offsets=None, h0=None, y=A, y_ld=L, hT=None,
             states=None, ws=A, ws_bytes=1 << 40, status=None)
    assert set(kw) <= set(a)
    return lib.sdm_gdr_forward(s, *{**a, **kw}.values(), None)


def gdr_backward(lib, s, **kw):
    a = dict(q=A, q_ld=L, k=A, k_ld=L, v=A, v_ld=L, g=A, g_ld=L, beta=A, beta_ld=L, dy=A, dy_ld=L, offsets=None, states=A, dhT=None,
             dq=A, dq_ld=L, dk=A, dk_ld=L, dv=A, dv_ld=L, dg=A, dg_ld=L, dbeta=A, dbeta_ld=L, dh0=None, ws=A, ws_bytes=1 << 40,
             status=None)
    assert set(kw) <= set(a)
    return lib.sdm_gdr_backward(s, *{**a, **kw}.values(), None)


def gdr_step(lib, s, **kw):
    a = dict(q=A, q_ld=L, k=A, k_ld=L, v=A, v_ld=L, g=A, g_ld=L, beta=A, beta_ld=L, slots=A, state=A, state_ld=L, states=100, y=A,
             y_ld=L, status=None)
    assert set(kw) <= set(a)
    return lib.sdm_gdr_step(s, *{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw, code", [
    (dict(P=0), -2), (dict(rows=-1), -2), (dict(rows=63), -2), (dict(k_heads=0), -2), (dict(v_heads=0), -2), (dict(v_heads=3), -2),
    (dict(dk=0), -2), (dict(dk=136), -2), (dict(dv=136), -2), (dict(dv=-8), -2), (dict(dk=60), -4), (dict(dv=20), -4),
    (dict(x_dtype=2), -3), (dict(g_dtype=-1), -3), (dict(scale=float("nan")), -2), (dict(rows=1 << 41), -2),
    (dict(k_heads=1, v_heads=65537), -2), (dict(rows=1 << 36), -2), (dict(P=1 << 28, rows=0), -2)])
def test_gdr_shapes(lib, kw, code):
    s = gdr(**kw)
    assert gdr_forward(lib, s) == code and gdr_backward(lib, s) == code
    if kw != dict(rows=63):   # equal lengths concern sequences only
        assert gdr_step(lib, s) == code
        assert lib.sdm_gdr_states_bytes(s) == 0
        assert lib.sdm_gdr_workspace_bytes(s, 0) == 0 and lib.sdm_gdr_workspace_bytes(s, 1) == 0


@pytest.mark.parametrize("call, name", [(gdr_forward, n) for n in "q k v g beta y".split()]
                         + [(gdr_backward, n) for n in "q k v g beta dy dq dk dv dg dbeta".split()]
                         + [(gdr_step, n) for n in "q k v g beta y state".split()])
def test_gdr_arrays(lib, call, name):
    s, gate, state = gdr(), name in ("g", "beta", "dg", "dbeta"), name == "state"
    out = name[0] == "d" and name != "dy" or name in ("y", "state")
    assert call(lib, s, **{name: None}) == -1
    assert call(lib, s, **{name + "_ld": -8}) == -1
    assert call(lib, s, **{name + "_ld": (1 << 40) + 8}) == -1
    if out:   # rows that overlap
        width = 4 if gate else 4 * 32 * 64 if state else 2 * 64 if name in ("dq", "dk") else 4 * 32
        assert call(lib, s, **{name + "_ld": width - (4 if gate else 8)}) == -1
    assert call(lib, s, **{name: A + (2 if gate else 8)}) == -4
    if not gate:
        assert call(lib, s, **{name + "_ld": L + (2 if state else 4)}) == -4


def test_gdr_small_arrays(lib):
    s = gdr()
    for n in ("h0", "hT", "states"):
        assert gdr_forward(lib, s, **{n: A + 8}) == -4
    for n in ("states", "dhT", "dh0"):
        assert gdr_backward(lib, s, **{n: A + 8}) == -4
    assert gdr_backward(lib, s, states=None) == -1
    for call in (gdr_forward, gdr_backward):
        assert call(lib, s, offsets=A + 4) == -4 and call(lib, s, status=A + 2) == -4
        n = lib.sdm_gdr_workspace_bytes(s, int(call is gdr_backward))
        assert n > 0
        for ws in (dict(ws=None), dict(ws=A + 8), dict(ws_bytes=n - 1)):
            assert call(lib, s, **ws) == -5
        assert call(lib, None) == -1
    assert gdr_step(lib, s, states=63, slots=None) == -2   # fewer states than rows
    assert gdr_step(lib, s, states=-1) == -2 and gdr_step(lib, s, slots=A + 2) == -4
    assert gdr_step(lib, gdr(rows=0), q=None, k=None, v=None, g=None, beta=None, y=None, state=None) == 0   # nothing to do


def test_gdr_sizes(lib):
    """Sizes grow with the rows, the backward's workspace serves the forward, and heads of 8 channels fit too."""
    for kw in (dict(), dict(x_dtype=0), dict(dk=8, dv=8), dict(rows=0), dict(P=1, rows=1), dict(k_heads=4)):
        s, more = gdr(**kw), gdr(**{**kw, "rows": 64 * 40})
        assert 0 < lib.sdm_gdr_workspace_bytes(s, 0) <= lib.sdm_gdr_workspace_bytes(s, 1) < lib.sdm_gdr_workspace_bytes(more, 1)
        assert 0 < lib.sdm_gdr_states_bytes(s) < lib.sdm_gdr_states_bytes(more)


def norm(**kw):
    base = dict(rows=8, D=64, group=32, post=1, gate=1, residual=1, pre=1, dtype=1, eps=1e-6, scale=1.0)
    base.update(kw)
    return ctypes.byref(_abi.NormShape(**base))


def norm_forward(lib, s, **kw):
    a = dict(o=A, o_ld=L, z=A, z_ld=L, x=A, x_ld=L, w_post=A, w_pre=A, channel_scale=A, r=A, r_ld=L, y=A, y_ld=L)
    assert set(kw) <= set(a)
    return lib.sdm_block_norm(s, *{**a, **kw}.values(), None)


def norm_backward(lib, s, **kw):
    a = dict(o=A, o_ld=L, z=A, z_ld=L, r=A, r_ld=L, dr=A, dr_ld=L, dy=A, dy_ld=L, w_post=A, w_pre=A, channel_scale=A, d_o=A,
             d_o_ld=L, dz=A, dz_ld=L, dx=A, dx_ld=L, dw_post=A, dw_pre=A, d_channel_scale=A, ws=A, ws_bytes=1 << 30)
    assert set(kw) <= set(a)
    return lib.sdm_block_norm_backward(s, *{**a, **kw}.values(), None)


@pytest.mark.parametrize("kw, code", [
    (dict(rows=-1), -2), (dict(D=0), -2), (dict(group=0), -2), (dict(group=128), -2), (dict(group=24), -2), (dict(post=2), -2),
    (dict(gate=3), -2), (dict(gate=-1), -2), (dict(residual=2), -2), (dict(pre=-1), -2), (dict(dtype=2), -3), (dict(eps=-1.0), -2),
    (dict(eps=float("nan")), -2), (dict(scale=float("nan")), -2), (dict(D=66, group=66), -4), (dict(D=64, group=2), -4),
    (dict(D=1 << 24, group=1 << 24), -2), (dict(D=8192, group=4), -2)])
def test_norm_shapes(lib, kw, code):
    s = norm(**kw)
    assert norm_forward(lib, s) == code and norm_backward(lib, s) == code and lib.sdm_block_norm_workspace_bytes(s) == 0


@pytest.mark.parametrize("call, name", [(norm_forward, n) for n in "o z x r y".split()]
                         + [(norm_backward, n) for n in "o z r dy d_o dz dr dx".split()])
def test_norm_rows(lib, call, name):
    s, optional = norm(), call is norm_backward and name in ("dr", "dx")
    if not optional:
        assert call(lib, s, **{name: None}) == -1
    if call is norm_forward and name in ("r", "y") or name in ("d_o", "dz", "dx"):
        assert call(lib, s, **{name + "_ld": 60}) == -1   # rows that overlap
    assert call(lib, s, **{name + "_ld": -4}) == -1
    assert call(lib, s, **{name: A + 4}) == -4
    assert call(lib, s, **{name + "_ld": L + 2}) == -4
    assert call(lib, norm(dtype=0), **{name: A + 8}) == -4


def test_norm_small_arrays(lib):
    s = norm()
    for n in ("w_post", "w_pre", "channel_scale"):
        assert norm_forward(lib, s, **{n: A + 4}) == -4 and norm_backward(lib, s, **{n: A + 4}) == -4
    for n in ("dw_post", "dw_pre", "d_channel_scale"):
        assert norm_backward(lib, s, **{n: A + 2}) == -4
    size = lib.sdm_block_norm_workspace_bytes(s)
    assert size > 0
    for ws in (dict(ws=None), dict(ws=A + 4), dict(ws_bytes=size - 1)):
        assert norm_backward(lib, s, **ws) == -5
    assert norm_backward(lib, norm(pre=0), dr=None) == -1     # no gradient at all
    assert norm_forward(lib, None) == -1 and norm_backward(lib, None) == -1
    assert norm_forward(lib, norm(rows=0), o=None, z=None, x=None, r=None, y=None) == 0


def embed(**kw):
    base = dict(tokens=8, V=100, D=64, table_dtype=0, dtype=1, scale=1.0)
    base.update(kw)
    return ctypes.byref(_abi.EmbedShape(**base))


@pytest.mark.parametrize("kw, code", [
    (dict(tokens=-1), -2), (dict(tokens=1 << 31), -2), (dict(V=0), -2), (dict(V=(1 << 28) + 1), -2), (dict(D=0), -2),
    (dict(D=(1 << 20) + 4), -2), (dict(D=66), -4), (dict(table_dtype=2), -3), (dict(dtype=-1), -3), (dict(scale=float("nan")), -2)])
def test_embed_shapes(lib, kw, code):
    s = embed(**kw)
    assert lib.sdm_embed(s, A, A, L, A, L, None, None) == code
    assert lib.sdm_embed_backward(s, A, A, L, A, L, 0, A, 1 << 40, None, None) == code
    assert lib.sdm_embed_workspace_bytes(s) == 0


def test_embed_arrays(lib):
    s, f, b = embed(), lib.sdm_embed, lib.sdm_embed_backward
    size = lib.sdm_embed_workspace_bytes(s)
    assert size > 0
    assert f(None, A, A, L, A, L, None, None) == -1
    assert f(s, None, A, L, A, L, None, None) == -1 and f(s, A, None, L, A, L, None, None) == -1
    assert f(s, A, A, L, None, L, None, None) == -1
    assert f(s, A, A, -4, A, L, None, None) == -1 and f(s, A, A, L, A, 60, None, None) == -1
    assert f(s, A + 2, A, L, A, L, None, None) == -4 and f(s, A, A + 8, L, A, L, None, None) == -4
    assert f(s, A, A, L + 2, A, L, None, None) == -4 and f(s, A, A, L, A + 4, L, None, None) == -4
    assert f(s, A, A, L, A, L, A + 2, None) == -4
    assert f(embed(tokens=0), None, None, 0, None, 0, None, None) == 0
    assert b(s, None, A, L, A, L, 0, A, size, None, None) == -1 and b(s, A, None, L, A, L, 0, A, size, None, None) == -1
    assert b(s, A, A, L, None, L, 0, A, size, None, None) == -1 and b(s, A, A, L, A, 60, 0, A, size, None, None) == -1
    assert b(s, A, A, L, A, L, 2, A, size, None, None) == -1
    assert b(s, A, A + 4, L, A, L, 0, A, size, None, None) == -4 and b(s, A, A, L, A + 8, L, 0, A, size, None, None) == -4
    assert b(s, A, A, L, A, L, 0, A, size, A + 2, None) == -4
    for ws, n in ((None, size), (A + 8, size), (A, size - 1)):
        assert b(s, A, A, L, A, L, 0, ws, n, None, None) == -5


def test_the_binding_refuses_what_is_not_on_a_gpu(lib):
    x, y = torch.zeros(8, 1, 8), torch.zeros(8, 1)
    spec = sdm.GdrSpec(P=1, rows=8, k_heads=1, v_heads=1, dk=8, dv=8, x_dtype="f32")
    with pytest.raises(TypeError, match="q: expected a CUDA tensor"):
        sdm.gdr_forward(spec, x, x, x, y, y, x, None)
    with pytest.raises(ValueError, match="states"):
        sdm.gdr_backward(spec, x, x, x, y, y, x, None, x, x, x, y, y, None)
    with pytest.raises(ValueError, match="state"):
        sdm.gdr_step(spec, x, x, x, y, y, x, x)
    with pytest.raises(TypeError, match="o: expected a CUDA tensor"):
        sdm.block_norm(sdm.BlockNormSpec(rows=8, D=8, dtype="f32"), x[:, 0], x[:, 0])
    with pytest.raises(TypeError, match="ids: expected a CUDA tensor"):
        sdm.embed(sdm.EmbedSpec(tokens=8, V=8, D=8), torch.zeros(8, dtype=torch.int32), x[:, 0], x[:, 0])
    for bad in (sdm.GdrSpec(P=1, rows=8, k_heads=2, v_heads=3, dk=8, dv=8), sdm.GdrSpec(P=0, rows=8, k_heads=1, v_heads=1, dk=8, dv=8)):
        with pytest.raises(ValueError):
            sdm.alloc_gdr_workspace(bad, device="cpu")
        with pytest.raises(ValueError):
            sdm.alloc_gdr_states(bad, device="cpu")
    with pytest.raises(KeyError):
        sdm.alloc_block_norm_workspace(sdm.BlockNormSpec(rows=8, D=8, gate="tanh"), device="cpu")
    with pytest.raises(ValueError):
        sdm.alloc_embed_workspace(sdm.EmbedSpec(tokens=8, V=0, D=8), device="cpu")
