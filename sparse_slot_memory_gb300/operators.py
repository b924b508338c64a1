"""Python face of the operators around the memory layer (include/sdm.h): argument marshalling only.

* ``glr_*``: the gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t, its backward, and one token per request;
* ``gdr_*``: the gated delta rule, a state of dk slots a head that every token decays, corrects and reads, its backward, and one
  token per request;
* ``qk_norm_rope*``: the norm of every query and key head with the position rotation in the same pass;
* ``block_norm*``: the norms behind and before a block with its gate, the residual's scale and sum;
* ``embed*``: the rows of an embedding table for tokens, and the table's gradient by sorted tokens;
* ``token_logprobs*``: log probabilities of given tokens, entropy, top alternatives, and the logits' gradient.

Tensors are CUDA tensors owned by the caller. Row arrays are two-dimensional (heads: three-dimensional) views
whose last dimension is contiguous; the distance between rows is read from the tensor, so a slice of a fused
projection's rows can be passed as it is. Every shape, type and alignment is checked before a launch.
"""

from __future__ import annotations

import ctypes
import dataclasses
import math

import torch

from . import _abi
from .api import _DT, _TORCH_DT, _check, _cur_device, _need, _ptr, _stream

_LAYOUT = {"half": 0, "interleaved": 1}


class _Spec:
    """A frozen description; what is derived from it is built once (the C struct is only read by the library)."""

    def _keep(self, name, value):
        object.__setattr__(self, name, value)
        return value

    def c(self):
        cs = self.__dict__.get("_cref")
        if cs is None:
            global _alone
            _alone = torch.cuda.device_count() <= 1
            cs = self._keep("_cref", ctypes.byref(self._struct()))
        return cs


_Tensor = torch.Tensor

# Whether there is no other GPU for a tensor to lie on, so that its place needs no look (a microsecond of a call of seven).
_alone = False

# the device that the library launches on: the current one, asked for without torch.cuda's wrappers where torch has it
_here = _cur_device if _cur_device is not None else torch.cuda.current_device


def _place(t, name: str):
    """Refuses a CPU tensor, and one of another GPU than the current one, whose stream the call would use."""
    if not isinstance(t, _Tensor) or not t.is_cuda:
        raise TypeError(f"{name}: expected a CUDA tensor (the library runs on the GPU only)")
    if not _alone and t.get_device() != _here():
        raise ValueError(f"{name}: lies on GPU {t.get_device()}, the current one is GPU {_here()}")


def _rows(t, dtype, shape, n, name: str, out: bool = False):
    """The address of a row array [rows, ..] whose rows hold n elements, and the distance between its rows in elements.
    The library reads bare pointers, so type, shape, place and layout are checked here."""
    if (t.__class__ is _Tensor and t.dtype is dtype and t.is_cuda and (_alone or t.get_device() == _here())
            and t.shape == shape and t.is_contiguous()):
        return t.data_ptr(), n
    _place(t, name)
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if t.shape != shape:
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    st = t.stride()
    m = 1
    for i in range(len(shape) - 1, 0, -1):   # every dimension but the rows' is contiguous
        if st[i] != m and shape[i] > 1:
            raise ValueError(f"{name}: rows must be contiguous, got strides {st}")
        m *= shape[i]
    if shape[0] <= 1:
        return t.data_ptr(), n
    if out and st[0] < n:
        raise ValueError(f"{name}: rows of an output must not overlap, got strides {st}")
    return t.data_ptr(), st[0]


def _small(t, dtype, numel: int, name: str):
    """The address of an optional contiguous array of at least ``numel`` elements."""
    if t is None:
        return None
    if (t.__class__ is _Tensor and t.dtype is dtype and t.is_cuda and (_alone or t.get_device() == _here())
            and t.numel() >= numel and t.is_contiguous()):
        return t.data_ptr()
    _need(t, dtype, numel, name)
    _place(t, name)
    return _ptr(t)


def _status(status):
    return None if status is None else _small(status, torch.int32, 1, "status")


_F32, _I32 = torch.float32, torch.int32


# ---- the gated linear recurrence -------------------------------------------------------------------
@dataclasses.dataclass(frozen=True)
class GlrSpec(_Spec):
    """P sequences of together ``rows`` rows of D channels. ``gate_width`` channels share a gate: 1, or a
    multiple of 4 that divides D."""

    P: int
    rows: int
    D: int
    gate_width: int = 1
    x_dtype: str = "bf16"
    g_dtype: str = "f32"

    @property
    def gates(self) -> int:
        return self.D // self.gate_width

    def _struct(self):
        return _abi.GlrShape(self.P, self.D, self.gate_width, _DT[self.x_dtype], _DT[self.g_dtype], self.rows)


def _bytes(spec, fn: str) -> int:
    n = spec.__dict__.get(fn)
    if n is None:
        n = spec._keep(fn, int(getattr(_abi.load(), fn)(spec.c())))
        if n == 0:
            raise ValueError(f"invalid shape {spec}")
    return n


def _glr_kinds(spec: GlrSpec):
    """The tensors' types and shapes: x's, g's, rows of x, rows of g, and P * D."""
    k = spec.__dict__.get("_kinds")
    if k is None:
        k = spec._keep("_kinds", (_TORCH_DT[spec.x_dtype], _TORCH_DT[spec.g_dtype], (spec.rows, spec.D),
                                  (spec.rows, spec.gates), spec.P * spec.D))
    return k


def alloc_glr_states(spec: GlrSpec, device="cuda") -> torch.Tensor:
    """The float32 states [.., D] that the forward saves for the backward (one for every 64 rows)."""
    n = _bytes(spec, "sdm_glr_states_bytes")
    return torch.empty((n // (4 * spec.D), spec.D), dtype=torch.float32, device=device)


def alloc_glr_workspace(spec: GlrSpec, device="cuda") -> torch.Tensor:
    return torch.empty(_bytes(spec, "sdm_glr_workspace_bytes"), dtype=torch.uint8, device=device)


def _glr_states(spec: GlrSpec, states):
    return _small(states, _F32, (spec.rows // _abi.SDM_GLR_CHUNK + spec.P) * spec.D, "states")


def glr_forward(spec: GlrSpec, x, g, y, offsets=None, h0=None, hT=None, states=None, status=None, stream=None):
    """sdm_glr_forward: y_t = h_t = exp(g_t) h_{t-1} + x_t over every sequence's rows.
    ``x``, ``y`` [rows, D]; ``g`` [rows, D / gate_width] log gates, at most 0; ``offsets`` (optional) int64
    [P + 1]: sequence p owns rows offsets[p] .. offsets[p+1] - 1, else all have rows / P rows; ``h0``, ``hT``
    (optional) float32 [P, D]: the states before and after (may be one tensor); ``states`` (optional, from
    ``alloc_glr_states``) receives what ``glr_backward`` needs. ``y`` may be ``x``, which
    costs the division of long sequences of few channels into segments."""
    xt, gt, xs, gs, PD = _glr_kinds(spec)
    D, G = xs[1], gs[1]
    st = _abi.load().sdm_glr_forward(
        spec.c(), *_rows(x, xt, xs, D, "x"), *_rows(g, gt, gs, G, "g"), _small(offsets, torch.int64, spec.P + 1, "offsets"),
        _small(h0, _F32, PD, "h0"), *_rows(y, xt, xs, D, "y", True), _small(hT, _F32, PD, "hT"),
        _glr_states(spec, states), _status(status), _stream(stream))
    _check(st, "sdm_glr_forward")


def glr_backward(spec: GlrSpec, x, g, dy, states, dx, dg, ws=None, offsets=None, dhT=None, dh0=None, status=None,
                 stream=None):
    """sdm_glr_backward: the gradients ``dx`` [rows, D], ``dg`` [rows, D / gate_width] and ``dh0`` (optional,
    float32 [P, D]) from ``dy`` and ``dhT`` (optional: the gradient of the states after). ``x``, ``g``, ``offsets`` and
    ``states`` are those of the forward; ``ws`` (from ``alloc_glr_workspace``) is needed where gate_width > 128.
    ``dx`` may be ``dy`` or ``x``."""
    xt, gt, xs, gs, PD = _glr_kinds(spec)
    D, G = xs[1], gs[1]
    if states is None:
        raise ValueError("states: the backward needs the states that the forward saved")
    st = _abi.load().sdm_glr_backward(
        spec.c(), *_rows(x, xt, xs, D, "x"), *_rows(g, gt, gs, G, "g"), *_rows(dy, xt, xs, D, "dy"),
        _small(offsets, torch.int64, spec.P + 1, "offsets"), _glr_states(spec, states), _small(dhT, _F32, PD, "dhT"),
        *_rows(dx, xt, xs, D, "dx", True), *_rows(dg, gt, gs, G, "dg", True), _small(dh0, _F32, PD, "dh0"),
        _small(ws, torch.uint8, 0, "ws"), 0 if ws is None else ws.numel(), _status(status), _stream(stream))
    _check(st, "sdm_glr_backward")


def glr_step(spec: GlrSpec, x, g, state, y, slots=None, status=None, stream=None):
    """sdm_glr_step: one token of each of ``spec.rows`` requests. ``state`` float32 [states, D] is updated in place:
    row ``slots[i]`` (int32, distinct; below 0: a padding row) for token i, or row i without ``slots``."""
    xt, gt, xs, gs, _ = _glr_kinds(spec)
    D = xs[1]
    if not isinstance(state, _Tensor) or state.dim() != 2:
        raise ValueError("state: expected a float32 tensor [states, D]")
    n = state.shape[0]
    st = _abi.load().sdm_glr_step(
        spec.c(), *_rows(x, xt, xs, D, "x"), *_rows(g, gt, gs, gs[1], "g"), _small(slots, _I32, xs[0], "slots"),
        *_rows(state, _F32, (n, D), D, "state", True), n, *_rows(y, xt, xs, D, "y", True), _status(status), _stream(stream))
    _check(st, "sdm_glr_step")


# ---- the gated delta rule ------------------------------------------------------------------------------
@dataclasses.dataclass(frozen=True)
class GdrSpec(_Spec):
    """P sequences of together ``rows`` rows; ``k_heads`` heads of queries and keys of ``dk`` channels, ``v_heads`` (a multiple) heads
    of values of ``dv`` channels, each with its decay, write strength and state [dk, dv]. dk and dv: multiples of 8, up to 128."""

    P: int
    rows: int
    k_heads: int
    v_heads: int
    dk: int
    dv: int
    x_dtype: str = "bf16"
    g_dtype: str = "f32"
    scale: float = 1.0

    def _struct(self):
        return _abi.GdrShape(self.P, self.k_heads, self.v_heads, self.dk, self.dv, _DT[self.x_dtype], _DT[self.g_dtype],
                             self.scale, self.rows)


def alloc_gdr_states(spec: GdrSpec, device="cuda") -> torch.Tensor:
    """What the forward saves for the backward: the state before every 64th row, the rows' writes and what their blocks give
    without the state, in the kernels' own form (bytes)."""
    return torch.empty(_bytes(spec, "sdm_gdr_states_bytes"), dtype=torch.uint8, device=device)


def _gdr_bytes(spec: GdrSpec, backward: bool) -> int:
    name = "_ws_backward" if backward else "_ws_forward"
    n = spec.__dict__.get(name)
    if n is None:
        n = spec._keep(name, int(_abi.load().sdm_gdr_workspace_bytes(spec.c(), int(backward))))
        if n == 0:
            raise ValueError(f"invalid shape {spec}")
    return n


def alloc_gdr_workspace(spec: GdrSpec, backward: bool = True, device="cuda") -> torch.Tensor:
    """The workspace of ``gdr_forward`` and, with ``backward``, of ``gdr_backward`` (one for both; it holds nothing between calls)."""
    return torch.empty(_gdr_bytes(spec, backward), dtype=torch.uint8, device=device)


def _gdr_kinds(spec: GdrSpec):
    """The tensors' types and shapes: x's, g's, queries and keys, values, gates, numbers in a row of each, of a state, and of
    all states."""
    k = spec.__dict__.get("_kinds")
    if k is None:
        n, Hk, Hv, dk, dv = spec.rows, spec.k_heads, spec.v_heads, spec.dk, spec.dv
        k = spec._keep("_kinds", (_TORCH_DT[spec.x_dtype], _TORCH_DT[spec.g_dtype], (n, Hk, dk), (n, Hv, dv), (n, Hv), Hk * dk,
                                  Hv * dv, Hv, Hv * dk * dv, spec.P * Hv * dk * dv))
    return k


def _gdr_inputs(kinds, q, k, v, g, beta):
    xt, gt, ks, vs, gs, kn, vn, H = kinds[:8]
    return (*_rows(q, xt, ks, kn, "q"), *_rows(k, xt, ks, kn, "k"), *_rows(v, xt, vs, vn, "v"), *_rows(g, gt, gs, H, "g"),
            *_rows(beta, gt, gs, H, "beta"))


def _gdr_states(spec: GdrSpec, states):
    return _small(states, torch.uint8, _bytes(spec, "sdm_gdr_states_bytes") if states is not None else 0, "states")


def _workspace(ws):
    return _small(ws, torch.uint8, 0, "ws"), 0 if ws is None else ws.numel()


def gdr_forward(spec: GdrSpec, q, k, v, g, beta, y, ws, offsets=None, h0=None, hT=None, states=None, status=None, stream=None):
    """sdm_gdr_forward: per sequence and value head S_t = exp(g_t) S_{t-1} + k_t u_t^T with u_t = beta_t (v_t - exp(g_t) S_{t-1}^T k_t),
    and y_t = scale S_t^T q_t. ``q``, ``k`` [rows, k_heads, dk]; ``v``, ``y`` [rows, v_heads, dv]; ``g`` (log decays, at most 0) and
    ``beta`` [rows, v_heads]; ``ws`` from ``alloc_gdr_workspace``; ``offsets`` (optional) int64 [P + 1] as in ``glr_forward``; ``h0``,
    ``hT`` (optional) float32 [P, v_heads, dk, dv]: the states before and after (may be one tensor); ``states`` (optional, from
    ``alloc_gdr_states``) receives what ``gdr_backward`` needs."""
    kinds = _gdr_kinds(spec)
    st = _abi.load().sdm_gdr_forward(
        spec.c(), *_gdr_inputs(kinds, q, k, v, g, beta), _small(offsets, torch.int64, spec.P + 1, "offsets"),
        _small(h0, _F32, kinds[9], "h0"), *_rows(y, kinds[0], kinds[3], kinds[6], "y", True), _small(hT, _F32, kinds[9], "hT"),
        _gdr_states(spec, states), *_workspace(ws), _status(status), _stream(stream))
    _check(st, "sdm_gdr_forward")


def gdr_backward(spec: GdrSpec, q, k, v, g, beta, dy, states, dq, dk, dv, dg, dbeta, ws, offsets=None, dhT=None, dh0=None,
                 status=None, stream=None):
    """sdm_gdr_backward: the gradients ``dq``, ``dk`` [rows, k_heads, dk], ``dv`` [rows, v_heads, dv], ``dg``, ``dbeta`` [rows, v_heads] and
    ``dh0`` (optional, float32 [P, v_heads, dk, dv]) from ``dy`` and ``dhT`` (optional: the gradient of the states after). The other
    arrays are the forward's, with the ``states`` that it saved; ``ws`` from ``alloc_gdr_workspace``."""
    kinds = _gdr_kinds(spec)
    xt, gt, ks, vs, gs, kn, vn, H = kinds[:8]
    if states is None:
        raise ValueError("states: the backward needs the states that the forward saved")
    st = _abi.load().sdm_gdr_backward(
        spec.c(), *_gdr_inputs(kinds, q, k, v, g, beta), *_rows(dy, xt, vs, vn, "dy"),
        _small(offsets, torch.int64, spec.P + 1, "offsets"), _gdr_states(spec, states), _small(dhT, _F32, kinds[9], "dhT"),
        *_rows(dq, xt, ks, kn, "dq", True), *_rows(dk, xt, ks, kn, "dk", True), *_rows(dv, xt, vs, vn, "dv", True),
        *_rows(dg, gt, gs, H, "dg", True), *_rows(dbeta, gt, gs, H, "dbeta", True), _small(dh0, _F32, kinds[9], "dh0"),
        *_workspace(ws), _status(status), _stream(stream))
    _check(st, "sdm_gdr_backward")


def gdr_step(spec: GdrSpec, q, k, v, g, beta, state, y, slots=None, status=None, stream=None):
    """sdm_gdr_step: one token of each of ``spec.rows`` requests. ``state`` float32 [states, v_heads, dk, dv] is updated in place:
    ``state[slots[i]]`` (int32, distinct; below 0: a padding row) for token i, or ``state[i]`` without ``slots``."""
    kinds = _gdr_kinds(spec)
    xt, H = kinds[0], spec.v_heads
    if not isinstance(state, _Tensor) or state.dim() != 4:
        raise ValueError("state: expected a float32 tensor [states, v_heads, dk, dv]")
    n = state.shape[0]
    st = _abi.load().sdm_gdr_step(
        spec.c(), *_gdr_inputs(kinds, q, k, v, g, beta), _small(slots, _I32, spec.rows, "slots"),
        *_rows(state, _F32, (n, H, spec.dk, spec.dv), kinds[8], "state", True), n, *_rows(y, xt, kinds[3], kinds[6], "y", True),
        _status(status), _stream(stream))
    _check(st, "sdm_gdr_step")


# ---- norms of queries and keys with the position rotation ---------------------------------------------
@dataclasses.dataclass(frozen=True)
class RopeSpec(_Spec):
    """``tokens`` tokens of q_heads + k_heads heads of ``hd`` columns, the first ``rot_dim`` of which turn, in pairs
    (i, i + rot_dim / 2) for the layout "half" and (2i, 2i + 1) for "interleaved"."""

    tokens: int
    q_heads: int
    k_heads: int
    hd: int
    rot_dim: int
    max_pos: int
    layout: str = "half"
    dtype: str = "bf16"
    norm: bool = True
    eps: float = 1e-6

    def _struct(self):
        return _abi.RopeShape(self.tokens, self.q_heads, self.k_heads, self.hd, self.rot_dim, self.max_pos,
                              _LAYOUT[self.layout], _DT[self.dtype], int(self.norm), self.eps)


def rope_frequencies(rot_dim: int, base: float = 10000.0, scaling: str = "none", factor: float = 1.0,
                     trained_len: int = 0, low: float = 1.0, high: float = 32.0) -> list:
    """The angles of one position, base^(-2i / rot_dim), scaled for contexts ``factor`` times as long:
    "linear" divides every angle by the factor; "base" raises the base so that the slowest angle is divided by it
    and the fastest kept; "by_parts" divides the angles that turn less than ``low`` times within ``trained_len``
    positions, keeps those that turn more than ``high`` times, and blends linearly between."""
    if rot_dim < 0 or rot_dim % 2 or factor <= 0 or base <= 0:
        raise ValueError("rot_dim must be even, base and factor positive")
    if scaling == "base" and rot_dim > 2:
        base = base * factor ** (rot_dim / (rot_dim - 2))
    f = [base ** (-2.0 * i / rot_dim) for i in range(rot_dim // 2)]
    if scaling in ("none", "base"):
        return f
    if scaling == "linear":
        return [v / factor for v in f]
    if scaling == "by_parts":
        if trained_len < 1 or not low < high:
            raise ValueError("by_parts needs trained_len and low < high")
        keep = [min(1.0, max(0.0, (trained_len * v / (2.0 * math.pi) - low) / (high - low))) for v in f]
        return [v * k + v / factor * (1.0 - k) for v, k in zip(f, keep)]
    raise ValueError(f"scaling: expected none, linear, base or by_parts, got {scaling!r}")


def rope_table(spec: RopeSpec, inv_freq, table, scale: float = 1.0, stream=None):
    """sdm_rope_table: ``table`` float32 [max_pos, rot_dim], scale * cos then scale * sin of position * inv_freq[i]
    (``inv_freq``: rot_dim / 2 angles, e.g. from ``rope_frequencies``)."""
    n = spec.rot_dim // 2
    if len(inv_freq) != n:
        raise ValueError(f"inv_freq: expected {n} angles, got {len(inv_freq)}")
    st = _abi.load().sdm_rope_table(spec.c(), (ctypes.c_double * max(n, 1))(*map(float, inv_freq)), scale,
                                    _small(table, torch.float32, spec.max_pos * spec.rot_dim, "table"), _stream(stream))
    _check(st, "sdm_rope_table")


def alloc_rope_workspace(spec: RopeSpec, device="cuda") -> torch.Tensor:
    return torch.empty(_bytes(spec, "sdm_rope_workspace_bytes"), dtype=torch.uint8, device=device)


def _heads(spec: RopeSpec, q, k, qname, kname, out=False):
    kinds = spec.__dict__.get("_kinds")
    if kinds is None:
        kinds = spec._keep("_kinds", (_TORCH_DT[spec.dtype], (spec.tokens, spec.q_heads, spec.hd),
                                      spec.q_heads * spec.hd, (spec.tokens, spec.k_heads, spec.hd), spec.k_heads * spec.hd))
    dt, qs, qn, ks, kn = kinds
    return (*(_rows(q, dt, qs, qn, qname, out) if qn else (None, 0)), *(_rows(k, dt, ks, kn, kname, out) if kn else (None, 0)))


def _rope_small(spec: RopeSpec, positions, table, wq, wk):
    hd = spec.hd
    return (_small(positions, _I32, spec.tokens, "positions"), _small(table, _F32, spec.max_pos * spec.rot_dim, "table"),
            _small(wq, _F32, hd, "wq"), _small(wk, _F32, hd, "wk"))


def qk_norm_rope(spec: RopeSpec, q, k, positions, table, wq, wk, q_out, k_out, status=None, stream=None):
    """sdm_qk_norm_rope: the RMS norm of every head of ``q`` [tokens, q_heads, hd] and ``k`` [tokens, k_heads, hd]
    with the weights ``wq``, ``wk`` (float32 [hd], or None for ones), turned by the table's row of the token's position
    (int32 [tokens]; below 0: a padding token, whose outputs are 0). The outputs may be the inputs."""
    st = _abi.load().sdm_qk_norm_rope(spec.c(), *_heads(spec, q, k, "q", "k"),
                                      *_rope_small(spec, positions, table, wq, wk),
                                      *_heads(spec, q_out, k_out, "q_out", "k_out", True), _status(status),
                                      _stream(stream))
    _check(st, "sdm_qk_norm_rope")


def qk_norm_rope_backward(spec: RopeSpec, dq_out, dk_out, q, k, positions, table, wq, wk, dq, dk, dwq=None, dwk=None,
                          ws=None, status=None, stream=None):
    """sdm_qk_norm_rope_backward: ``dq``, ``dk`` and the weights' gradients ``dwq``, ``dwk`` (optional, float32 [hd]) from
    the outputs' gradients and the forward's inputs. ``ws`` (from ``alloc_rope_workspace``) is needed for dwq, dwk."""
    st = _abi.load().sdm_qk_norm_rope_backward(
        spec.c(), *_heads(spec, dq_out, dk_out, "dq_out", "dk_out"), *_heads(spec, q, k, "q", "k"),
        *_rope_small(spec, positions, table, wq, wk), *_heads(spec, dq, dk, "dq", "dk", True),
        _small(dwq, _F32, spec.hd, "dwq"), _small(dwk, _F32, spec.hd, "dwk"), _small(ws, torch.uint8, 0, "ws"),
        0 if ws is None else ws.numel(), _status(status), _stream(stream))
    _check(st, "sdm_qk_norm_rope_backward")


# ---- the norms around a block -------------------------------------------------------------------------
_GATE = {"none": 0, "sigmoid": 1, "silu": 2}


@dataclasses.dataclass(frozen=True)
class BlockNormSpec(_Spec):
    """``rows`` rows of D columns. ``post``: the block's output is normed, by groups of ``group`` columns (0: whole rows); ``gate``:
    "none", "sigmoid" or "silu"; ``residual``: a stream is added; ``pre``: the sum is normed for the next block."""

    rows: int
    D: int
    group: int = 0
    post: bool = True
    gate: str = "none"
    residual: bool = True
    pre: bool = True
    scale: float = 1.0
    dtype: str = "bf16"
    eps: float = 1e-6

    def _struct(self):
        return _abi.NormShape(self.rows, self.D, self.group or self.D, int(self.post), _GATE[self.gate], int(self.residual),
                              int(self.pre), _DT[self.dtype], self.eps, self.scale)


def alloc_block_norm_workspace(spec: BlockNormSpec, device="cuda") -> torch.Tensor:
    return torch.empty(_bytes(spec, "sdm_block_norm_workspace_bytes"), dtype=torch.uint8, device=device)


def _norm_rows(spec: BlockNormSpec, t, name: str, out: bool = False, optional: bool = False):
    if t is None and optional:
        return None, 0
    return _rows(t, _TORCH_DT[spec.dtype], (spec.rows, spec.D), spec.D, name, out)


def block_norm(spec: BlockNormSpec, o, r, x=None, z=None, y=None, w_post=None, w_pre=None, channel_scale=None, stream=None):
    """sdm_block_norm: ``r`` = x + scale * channel_scale * act(z) * norm(o) * w_post and ``y`` = norm(r) * w_pre, rows [rows, D].
    ``o``: the block's output; ``z`` (with a gate), ``x`` (with residual) and ``y`` (with pre) where the spec has them; ``w_post`` float32
    [group], ``w_pre``, ``channel_scale`` float32 [D] (None: ones). ``r`` may be ``x``, ``y`` may be ``o``."""
    D = spec.D
    st = _abi.load().sdm_block_norm(
        spec.c(), *_norm_rows(spec, o, "o"), *_norm_rows(spec, z, "z", optional=spec.gate == "none"),
        *_norm_rows(spec, x, "x", optional=not spec.residual), _small(w_post, _F32, spec.group or D, "w_post"),
        _small(w_pre, _F32, D, "w_pre"), _small(channel_scale, _F32, D, "channel_scale"), *_norm_rows(spec, r, "r", True),
        *_norm_rows(spec, y, "y", True, not spec.pre), _stream(stream))
    _check(st, "sdm_block_norm")


def block_norm_backward(spec: BlockNormSpec, o, r, dr, d_o, ws=None, z=None, dy=None, w_post=None, w_pre=None, channel_scale=None,
                        dx=None, dz=None, dw_post=None, dw_pre=None, d_channel_scale=None, stream=None):
    """sdm_block_norm_backward: from ``dr`` (the gradient of r; None for zeros where there is ``dy``) and ``dy`` the gradients ``d_o``, ``dz``
    (with a gate), ``dx`` (optional: of the sum, the stream's) [rows, D] and of the weights, ``dw_post`` [group], ``dw_pre``,
    ``d_channel_scale`` [D] (optional, float32; they need ``ws`` from ``alloc_block_norm_workspace``). ``r`` is the forward's."""
    D = spec.D
    st = _abi.load().sdm_block_norm_backward(
        spec.c(), *_norm_rows(spec, o, "o"), *_norm_rows(spec, z, "z", optional=spec.gate == "none"),
        *_norm_rows(spec, r, "r", optional=not spec.pre), *_norm_rows(spec, dr, "dr", optional=spec.pre),
        *_norm_rows(spec, dy, "dy", optional=not spec.pre), _small(w_post, _F32, spec.group or D, "w_post"),
        _small(w_pre, _F32, D, "w_pre"), _small(channel_scale, _F32, D, "channel_scale"), *_norm_rows(spec, d_o, "d_o", True),
        *_norm_rows(spec, dz, "dz", True, spec.gate == "none"), *_norm_rows(spec, dx, "dx", True, True),
        _small(dw_post, _F32, spec.group or D, "dw_post"), _small(dw_pre, _F32, D, "dw_pre"),
        _small(d_channel_scale, _F32, D, "d_channel_scale"), *_workspace(ws), _stream(stream))
    _check(st, "sdm_block_norm_backward")


# ---- the embedding ------------------------------------------------------------------------------------
@dataclasses.dataclass(frozen=True)
class EmbedSpec(_Spec):
    """``tokens`` tokens and a table of V rows of D columns; ``table_dtype`` of the table and its gradient, ``dtype`` of the tokens'
    rows and theirs."""

    tokens: int
    V: int
    D: int
    table_dtype: str = "f32"
    dtype: str = "bf16"
    scale: float = 1.0

    def _struct(self):
        return _abi.EmbedShape(self.tokens, self.V, self.D, _DT[self.table_dtype], _DT[self.dtype], self.scale)


def alloc_embed_workspace(spec: EmbedSpec, device="cuda") -> torch.Tensor:
    return torch.empty(_bytes(spec, "sdm_embed_workspace_bytes"), dtype=torch.uint8, device=device)


def embed(spec: EmbedSpec, ids, table, y, status=None, stream=None):
    """sdm_embed: ``y[i]`` = scale * ``table[ids[i]]`` (``ids`` int32 [tokens]; below 0: padding, zeros; ``table`` [V, D], ``y`` [tokens, D])."""
    D = spec.D
    st = _abi.load().sdm_embed(
        spec.c(), _small(ids, _I32, spec.tokens, "ids"), *_rows(table, _TORCH_DT[spec.table_dtype], (spec.V, D), D, "table"),
        *_rows(y, _TORCH_DT[spec.dtype], (spec.tokens, D), D, "y", True), _status(status), _stream(stream))
    _check(st, "sdm_embed")


def embed_backward(spec: EmbedSpec, ids, dy, dtable, ws, accumulate=False, status=None, stream=None):
    """sdm_embed_backward: ``dtable`` [V, D], row v scale times the sum of ``dy`` over the tokens with id v, in a fixed order. Without
    ``accumulate`` every row is written; with it the sums are added to the rows that have tokens. ``ws`` from ``alloc_embed_workspace``."""
    D = spec.D
    st = _abi.load().sdm_embed_backward(
        spec.c(), _small(ids, _I32, spec.tokens, "ids"), *_rows(dy, _TORCH_DT[spec.dtype], (spec.tokens, D), D, "dy"),
        *_rows(dtable, _TORCH_DT[spec.table_dtype], (spec.V, D), D, "dtable", True), int(accumulate), *_workspace(ws), _status(status),
        _stream(stream))
    _check(st, "sdm_embed_backward")


# ---- log probabilities of tokens ---------------------------------------------------------------------
@dataclasses.dataclass(frozen=True)
class LogprobSpec(_Spec):
    """``rows`` rows of V logits, multiplied by ``scale`` (1 / temperature); K top alternatives (at most 32)."""

    rows: int
    V: int
    K: int = 0
    dtype: str = "bf16"
    scale: float = 1.0

    def _struct(self):
        return _abi.LogprobShape(self.rows, self.V, self.K, _DT[self.dtype], self.scale)


def token_logprobs(spec: LogprobSpec, logits, targets, logp, entropy=None, lse=None, top_vals=None, top_idx=None,
                   status=None, stream=None):
    """sdm_token_logprobs: of every row of ``logits`` [rows, V] the log probability of ``targets`` (int32; below 0:
    ignored, 0) and, where asked for, the entropy and log-sum-exp [rows] and the log probabilities and ids of the K
    largest logits [rows, K], the lower id first among equals (float32; ids int32)."""
    N, V, K = spec.rows, spec.V, spec.K
    st = _abi.load().sdm_token_logprobs(
        spec.c(), *_rows(logits, _TORCH_DT[spec.dtype], (N, V), V, "logits"), _small(targets, _I32, N, "targets"),
        _small(logp, _F32, N, "logp"), _small(entropy, _F32, N, "entropy"), _small(lse, _F32, N, "lse"),
        _small(top_vals, _F32, N * K, "top_vals"), _small(top_idx, _I32, N * K, "top_idx"), _status(status), _stream(stream))
    _check(st, "sdm_token_logprobs")


def token_logprobs_backward(spec: LogprobSpec, logits, targets, lse, entropy, d_logp, dlogits, d_entropy=None,
                            status=None, stream=None):
    """sdm_token_logprobs_backward: ``dlogits`` [rows, V] from the gradients of logp and (optional) of the entropy,
    with the forward's ``lse`` and ``entropy`` (None where there is no ``d_entropy``). ``dlogits`` may be ``logits``."""
    N, V, dt = spec.rows, spec.V, _TORCH_DT[spec.dtype]
    st = _abi.load().sdm_token_logprobs_backward(
        spec.c(), *_rows(logits, dt, (N, V), V, "logits"), _small(targets, _I32, N, "targets"), _small(lse, _F32, N, "lse"),
        _small(entropy, _F32, N, "entropy"), _small(d_logp, _F32, N, "d_logp"), _small(d_entropy, _F32, N, "d_entropy"),
        *_rows(dlogits, dt, (N, V), V, "dlogits", True), _status(status), _stream(stream))
    _check(st, "sdm_token_logprobs_backward")
