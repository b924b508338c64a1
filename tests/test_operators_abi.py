"""The operators around the memory without a GPU: their entry points refuse what they cannot take before any CUDA call
(no pointer below is ever dereferenced), and the binding refuses CPU tensors."""

import ctypes

import pytest
import torch

import sparse_slot_memory_gb300 as sdm
from sparse_slot_memory_gb300 import _abi

A = 0x100000   # an aligned address that nothing reads


@pytest.fixture(scope="module")
def lib():
    sdm.build()
    return _abi.load()


def glr(**kw):
    base = dict(P=2, D=256, gate_width=1, x_dtype=1, g_dtype=0, rows=64)
    base.update(kw)
    return ctypes.byref(_abi.GlrShape(**base))


GLR_BAD = [
    (dict(P=0), -2), (dict(D=0), -2), (dict(D=6), -4), (dict(D=(1 << 20) + 4), -2), (dict(gate_width=0), -2),
    (dict(gate_width=6), -4), (dict(gate_width=60), -2), (dict(x_dtype=2), -3), (dict(g_dtype=-1), -3),
    (dict(rows=-1), -2), (dict(rows=63), -2),
]


@pytest.mark.parametrize("kw, code", GLR_BAD)
def test_glr_shapes(lib, kw, code):
    s = glr(**kw)
    D = 1 << 21
    assert lib.sdm_glr_forward(s, A, D, A, D, None, None, A, D, None, None, None, None) == code
    assert lib.sdm_glr_backward(s, A, D, A, D, A, D, None, A, None, A, D, A, D, None, A, 1 << 40, None, None) == code
    if kw != dict(rows=63):   # equal lengths concern sequences only
        assert lib.sdm_glr_step(s, A, D, A, D, A, A, D, 100, A, D, None, None) == code
        assert lib.sdm_glr_states_bytes(s) == 0 and lib.sdm_glr_workspace_bytes(s) == 0


def test_glr_arrays(lib):
    s = glr()
    f = lib.sdm_glr_forward
    assert f(None, A, 256, A, 256, None, None, A, 256, None, None, None, None) == -1
    assert f(s, None, 256, A, 256, None, None, A, 256, None, None, None, None) == -1
    assert f(s, A, 256, None, 256, None, None, A, 256, None, None, None, None) == -1
    assert f(s, A, 256, A, 256, None, None, None, 256, None, None, None, None) == -1
    assert f(s, A, 256, A, 256, None, None, A, 252, None, None, None, None) == -1      # output rows overlap
    assert f(s, A, -4, A, 256, None, None, A, 256, None, None, None, None) == -1
    assert f(s, A + 4, 256, A, 256, None, None, A, 256, None, None, None, None) == -4
    assert f(s, A, 258, A, 256, None, None, A, 256, None, None, None, None) == -4
    assert f(s, A, 256, A + 8, 256, None, None, A, 256, None, None, None, None) == -4
    assert f(s, A, 256, A, 256, None, A + 4, A, 256, None, None, None, None) == -4
    b = lib.sdm_glr_backward
    assert b(s, A, 256, A, 256, A, 256, None, None, None, A, 256, A, 256, None, None, 0, None, None) == -1   # states
    wide = glr(gate_width=256)
    n = lib.sdm_glr_workspace_bytes(wide)
    assert n >= 2 * 64 * 4
    for ws, size in ((None, n), (A, n - 1), (A + 4, n)):
        assert b(wide, A, 256, A, 1, A, 256, None, A, None, A, 256, A, 1, None, ws, size, None, None) == -5
    t = lib.sdm_glr_step
    assert t(s, A, 256, A, 256, None, A, 256, 63, A, 256, None, None) == -2             # fewer states than rows
    assert t(s, A, 256, A, 256, A, A, 252, 100, A, 256, None, None) == -1
    assert t(s, A, 256, A, 256, A, A + 4, 256, 100, A, 256, None, None) == -4
    assert t(glr(rows=0), None, 0, None, 0, None, None, 0, 0, None, 0, None, None) == 0  # nothing to do, nothing launched


def test_glr_sizes(lib):
    """A state for every 64 rows and one for every sequence, however the rows are divided."""
    assert lib.sdm_glr_states_bytes(glr(P=3, rows=129)) == (2 + 3) * 256 * 4
    assert lib.sdm_glr_states_bytes(glr(P=1, rows=0)) == 256 * 4


def rope(**kw):
    base = dict(tokens=8, q_heads=4, k_heads=2, hd=64, rot_dim=32, max_pos=100, layout=0, dtype=1, norm=1, eps=1e-6)
    base.update(kw)
    return ctypes.byref(_abi.RopeShape(**base))


@pytest.mark.parametrize("kw, code", [
    (dict(tokens=-1), -2), (dict(q_heads=-1), -2), (dict(q_heads=0, k_heads=0), -2), (dict(hd=0), -2), (dict(hd=1032), -2),
    (dict(hd=68), -4), (dict(rot_dim=36), -4), (dict(rot_dim=-8), -2), (dict(rot_dim=72), -2), (dict(max_pos=0), -2),
    (dict(layout=2), -2), (dict(dtype=5), -3), (dict(norm=2), -2), (dict(eps=-1.0), -2), (dict(eps=float("nan")), -2)])
def test_rope_shapes(lib, kw, code):
    s, L = rope(**kw), 1 << 20
    assert lib.sdm_qk_norm_rope(s, A, L, A, L, A, A, A, A, A, L, A, L, None, None) == code
    assert lib.sdm_qk_norm_rope_backward(s, A, L, A, L, A, L, A, L, A, A, A, A, A, L, A, L, A, A, A, 1 << 30, None, None) == code
    assert lib.sdm_rope_table(s, (ctypes.c_double * 512)(), 1.0, A, None) == code
    assert lib.sdm_rope_workspace_bytes(s) == 0


def test_rope_arrays(lib):
    s, f = rope(), lib.sdm_qk_norm_rope
    assert f(s, None, 256, A, 128, A, A, A, A, A, 256, A, 128, None, None) == -1
    assert f(s, A, 256, A, 128, None, A, A, A, A, 256, A, 128, None, None) == -1
    assert f(s, A, 256, A, 128, A, None, A, A, A, 256, A, 128, None, None) == -1
    assert f(s, A, 256, A, 128, A, A, A, A, A, 252, A, 128, None, None) == -1
    assert f(s, A, 256, A + 4, 128, A, A, A, A, A, 256, A, 128, None, None) == -4
    assert f(s, A, 257, A, 128, A, A, A, A, A, 256, A, 128, None, None) == -4
    assert f(s, A, 256, A, 128, A, A, A + 4, A, A, 256, A, 128, None, None) == -4
    assert f(rope(tokens=0), None, 0, None, 0, None, None, None, None, None, 0, None, 0, None, None) == 0
    b = lib.sdm_qk_norm_rope_backward
    assert b(s, A, 256, A, 128, A, 256, A, 128, A, A, A, A, A, 256, A, 128, A, A, None, 0, None, None) == -5
    assert b(s, A, 256, A, 128, A, 256, A, 128, A, A, A, A, A, 256, A, 128, A, A, A, 16, None, None) == -5
    bad = (ctypes.c_double * 16)(*([float("inf")] * 16))
    assert lib.sdm_rope_table(s, bad, 1.0, A, None) == -1
    assert lib.sdm_rope_table(s, None, 1.0, A, None) == -1


def lp(**kw):
    base = dict(rows=4, V=100, K=3, dtype=0, scale=1.0)
    base.update(kw)
    return ctypes.byref(_abi.LogprobShape(**base))


@pytest.mark.parametrize("kw, code", [
    (dict(rows=-1), -2), (dict(rows=1 << 31), -2), (dict(V=0, K=0), -2), (dict(V=(1 << 28) + 1), -2), (dict(K=-1), -2),
    (dict(K=33), -2), (dict(V=2), -2), (dict(dtype=2), -3), (dict(scale=0.0), -2), (dict(scale=-1.0), -2),
    (dict(scale=float("nan")), -2), (dict(scale=float("inf")), -2)])
def test_logprob_shapes(lib, kw, code):
    s, L = lp(**kw), 1 << 30
    assert lib.sdm_token_logprobs(s, A, L, A, A, A, A, A, A, None, None) == code
    assert lib.sdm_token_logprobs_backward(s, A, L, A, A, A, A, A, A, L, None, None) == code


def test_logprob_arrays(lib):
    s, f, b = lp(), lib.sdm_token_logprobs, lib.sdm_token_logprobs_backward
    assert f(s, None, 100, A, A, None, None, None, None, None, None) == -1
    assert f(s, A, 100, None, A, None, None, None, None, None, None) == -1
    assert f(s, A, 100, A, None, None, None, None, None, None, None) == -1
    assert f(s, A, -1, A, A, None, None, None, None, None, None) == -1
    assert f(s, A + 2, 100, A, A, None, None, None, None, None, None) == -4
    assert f(lp(rows=0), None, 0, None, None, None, None, None, None, None, None) == 0
    assert b(s, A, 100, A, None, A, A, A, A, 100, None, None) == -1
    assert b(s, A, 100, A, A, A, A, None, A, 99, None, None) == -1
    assert b(s, A, 100, A, A, A, A, None, A + 2, 100, None, None) == -4


def test_misaligned_small_arrays(lib):
    """Arrays of ids, offsets, scalars per row and the status word off their elements' alignment."""
    f = lib.sdm_glr_forward
    assert f(glr(), A, 256, A, 256, A + 4, None, A, 256, None, None, None, None) == -4
    assert f(glr(), A, 256, A, 256, None, None, A, 256, None, None, A + 2, None) == -4
    assert lib.sdm_glr_backward(glr(), A, 256, A, 256, A, 256, A + 4, A, None, A, 256, A, 256, None, None, 0, None, None) == -4
    assert lib.sdm_glr_step(glr(), A, 256, A, 256, A + 2, A, 256, 100, A, 256, None, None) == -4
    r = lib.sdm_qk_norm_rope
    assert r(rope(), A, 256, A, 128, A + 2, A, A, A, A, 256, A, 128, None, None) == -4
    assert r(rope(), A, 256, A, 128, A, A, A, A, A, 256, A, 128, A + 1, None) == -4
    b = lib.sdm_qk_norm_rope_backward
    assert b(rope(), A, 256, A, 128, A, 256, A, 128, A, A, A, A, A, 256, A, 128, A + 2, A, A, 1 << 20, None, None) == -4
    p, q = lib.sdm_token_logprobs, lib.sdm_token_logprobs_backward
    good = [A, A, A, A, A, A, None]   # targets, logp, entropy, lse, top_vals, top_idx, status
    for i in range(7):
        bad = list(good)
        bad[i] = A + 2
        assert p(lp(), A, 100, *bad, None) == -4, i
    good = [A, A, A, A, A]   # targets, lse, entropy, d_logp, d_entropy
    for i in range(5):
        bad = list(good)
        bad[i] = A + 2
        assert q(lp(), A, 100, *bad, A, 100, None, None) == -4, i


def test_structs_match_the_header(lib):
    """The binding's structs have the header's fields in its order."""
    import os
    import re

    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "sdm.h")).read()
    src = re.sub(r"/\*.*?\*/", "", src, flags=re.S)
    for name, cls in (("sdm_glr_shape", _abi.GlrShape), ("sdm_rope_shape", _abi.RopeShape),
                      ("sdm_logprob_shape", _abi.LogprobShape)):
        body = re.search(r"typedef struct \{([^}]*)\} " + name + ";", src).group(1)
        fields = re.findall(r"(int32_t|int64_t|float)\s+(\w+);", body)
        kinds = {"int32_t": _abi.c_i32, "int64_t": _abi.c_i64, "float": ctypes.c_float}
        assert [(n, kinds[t]) for t, n in fields] == cls._fields_


def test_no_cpu_path():
    x = torch.zeros(4, 8)
    with pytest.raises(TypeError, match="GPU only"):
        sdm.glr_forward(sdm.GlrSpec(P=1, rows=4, D=8, x_dtype="f32"), x, x, x)
    with pytest.raises(TypeError, match="GPU only"):
        sdm.token_logprobs(sdm.LogprobSpec(rows=4, V=8, dtype="f32"), x, torch.zeros(4, dtype=torch.int32), torch.zeros(4))
    h = torch.zeros(4, 1, 8)
    with pytest.raises(TypeError, match="GPU only"):
        sdm.qk_norm_rope(sdm.RopeSpec(tokens=4, q_heads=1, k_heads=1, hd=8, rot_dim=8, max_pos=4, dtype="f32"), h, h,
                         torch.zeros(4, dtype=torch.int32), torch.zeros(4, 8), None, None, h, h)
