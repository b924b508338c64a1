"""Python face of the operators around the memory layer (include/sdm.h): argument marshalling only.

* ``glr_*``: the gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t, its backward, and one token per request;
* ``qk_norm_rope*``: the norm of every query and key head with the position rotation in the same pass;
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
