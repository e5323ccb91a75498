"""Torch-facing drivers of what surrounds a sublayer: norms, the residual add
with its gate and dropout, dropout alone, rotary positions, and the reversible
layer that joins them to the attention and the feed-forward.

As in ``attention``: a driver is made for one fixed problem, owns its output
buffers and workspaces (each call overwrites them; calls that overlap on the
GPU, and graphs that are replayed at the same time, need drivers of their
own), and every step runs in liblsh.so. Tensors are views [B, H, L, d] whose
strides are those of the driver's layout:

  "head"           [B, H, L, d] contiguous (the attention's layout);
  "token"          [B, L, H, d] contiguous, seen as [B, H, L, d];
  (sb, sh, sl)     any strides in elements, features adjacent; positive where
                   the dimension is longer than 1, elements distinct.

A tensor of another shape, type, device or layout raises ``LshError`` before
anything is launched. Parameters and their gradients are float32, contiguous.
Work is queued on ``stream`` (default: the current stream of the driver's
device). A driver made for another device than a GPU describes its problem, but
refuses its calls.
"""
from __future__ import annotations

import ctypes
import decimal
import math
from typing import Optional, Sequence, Tuple, Union

import torch

from . import _lib

_TORCH_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
_KINDS = {None: _lib.LSH_NORM_NONE, "layer": _lib.LSH_NORM_LAYER, "rms": _lib.LSH_NORM_RMS}
_GATES = {None: _lib.LSH_GATE_NONE, "vector": _lib.LSH_GATE_VECTOR,
          "sigmoid": _lib.LSH_GATE_SIGMOID}
_INT32_MAX = (1 << 31) - 1   # the C structs' sizes
Layout = Union[str, Sequence[int]]
_current_device = getattr(torch._C, "_cuda_getDevice", lambda: -1)
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 0)


def _refuse(where: str, what: str):
    raise _lib.LshError(1, f"{where}: {what}")


class _Driver:
    """Shape, type, device and layout checks shared by the drivers."""

    def __init__(self, B, H, L, d, dtype, device):
        if dtype not in _TORCH_DTYPE:
            _refuse(type(self).__name__, f"dtype {dtype!r}")
        self.B, self.H, self.L, self.d = int(B), int(H), int(L), int(d)
        if min(self.B, self.H, self.L) < 0 or self.d < 1:
            _refuse(type(self).__name__, "sizes must not be negative")
        if max(self.B, self.H, self.L, self.d) > _INT32_MAX:
            _refuse(type(self).__name__, "sizes are below 2^31")
        self.dtype = dtype
        self.tdtype = _TORCH_DTYPE[dtype]
        self.shape = (self.B, self.H, self.L, self.d)
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self._index = dev.index if dev.type == "cuda" else -1
        self._lib = _lib.lib()
        self._empty = self.B * self.H * self.L == 0

    def _strides(self, layout: Layout) -> Tuple[int, int, int, int]:
        B, H, L, d = self.shape
        if layout == "head":
            return (H * L * d, L * d, d, 1)
        if layout == "token":
            return (H * L * d, d, H * d, 1)
        if isinstance(layout, str) or len(layout) != 3:
            _refuse(type(self).__name__, f"layout {layout!r}")
        strides = tuple(int(s) for s in layout)
        # all zero would say "contiguous" to the library
        if not self._empty and any(n > 1 and s < 1 for n, s in zip(self.shape, strides)):
            _refuse(type(self).__name__, f"layout {layout!r}: strides of dimensions longer than "
                                         "1 are positive")
        return strides + (1,)

    def _buffer(self, strides) -> torch.Tensor:
        """An activation buffer of the driver's own in the layout's order."""
        B, H, L, d = self.shape
        if strides == self._strides("token"):
            return torch.empty((B, L, H, d), dtype=self.tdtype, device=self.device).transpose(1, 2)
        if strides == self._strides("head"):
            return torch.empty(self.shape, dtype=self.tdtype, device=self.device)
        if self._empty:
            return torch.empty(self.shape, dtype=self.tdtype, device=self.device)
        strides = [max(0, s) for s in strides]   # below 0: of a single element
        last = sum((n - 1) * s for n, s in zip(self.shape, strides))
        return torch.empty(last + 1, dtype=self.tdtype, device=self.device).as_strided(
            self.shape, strides)

    def _act(self, t, strides, name):
        """Address of an activation that has the driver's shape, type, device
        and the given strides. Decoding calls this for every token, so the
        usual case is one expression."""
        if t.dtype is self.tdtype and t.shape == self.shape and t.stride() == strides and \
                t.get_device() == self._index:
            return t.data_ptr()
        if t.dtype is not self.tdtype or t.shape != self.shape or \
                t.get_device() != self._index:
            _refuse(type(self).__name__, f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, "
                                         f"expected {self.tdtype} {self.shape} on {self.device}")
        if not self._empty:
            # strides of dimensions of one element say nothing
            for n, s, want in zip(self.shape, t.stride(), strides):
                if n > 1 and s != want:
                    _refuse(type(self).__name__, f"{name}: strides {t.stride()}, "
                                                 f"the layout's are {strides}")
        return t.data_ptr()

    def _vec(self, t, shape, name, dtype=torch.float32):
        """Address of a contiguous parameter (None: none)."""
        if t is None:
            return None
        if t.dtype is dtype and t.shape == shape and t.is_contiguous() and \
                t.get_device() == self._index:
            return t.data_ptr()
        _refuse(type(self).__name__, f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, "
                                     f"expected contiguous {dtype} {shape} on {self.device}")

    def _away(self):
        """Whether another device than the driver's is the current one."""
        return self._index >= 0 and _current_device() != self._index

    def _there(self, method, *args, **kw):
        with torch.cuda.device(self.device):
            return method(*args, **kw)

    def _stream(self, stream):
        """Handle of a stream; None is the device's current one. The last thing
        that every call looks up, so a driver of host memory, whose addresses no
        kernel can take, ends here."""
        if self._index < 0:
            _refuse(type(self).__name__, f"made for {self.device}, its calls need a CUDA device")
        if stream is None:
            return _current_stream(self._index)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _ok(self, code):
        if code != 0:
            raise _lib.LshError(code, type(self).__name__)

    def _sized(self, n):
        if n == 0 and not self._empty:
            _refuse(type(self).__name__, "workspace size query (problem rejected)")
        return n

    def _workspace(self, n):
        return torch.empty(max(1, n), dtype=torch.uint8, device=self.device)


def _slice0(v, name):
    if not 0 <= int(v) <= _INT32_MAX:
        _refuse(name, f"slice0 {v}")
    return int(v)


def _seed(v, name):
    if v.__class__ is not int:
        v = int(v)
    if not 0 <= v < 1 << 64:
        _refuse(name, "seed and offset are unsigned 64-bit numbers")
    return v


class Norm(_Driver):
    """h = xhat w + b over each token's H d features (``kind`` "layer" or
    "rms"). Buffers: h, and unless ``forward_only`` dx (their layouts), dw, db
    float32 [H d] and the backward's workspace."""

    def __init__(self, B, H, L, kind="layer", eps=1e-5, dtype="bf16", d=64,
                 x_layout: Layout = "head", h_layout: Layout = "head", device="cuda",
                 forward_only=False):
        super().__init__(B, H, L, d, dtype, device)
        if kind not in ("layer", "rms"):
            _refuse("Norm", f"kind {kind!r}")
        self.sx, self.sh = self._strides(x_layout), self._strides(h_layout)
        self.p = _lib.make_norm_problem(B, H, L, d, dtype, _KINDS[kind], eps, self.sx[:3],
                                        self.sh[:3])
        self.ws_bytes = self._sized(_lib.lsh_norm_bwd_workspace_size(self.p))
        self._p, self._norm_fwd = ctypes.byref(self.p), self._lib.lsh_norm_fwd
        self._D = (self.H * self.d,)
        self.h = self._buffer(self.sh)
        self._h = self.h.data_ptr()   # of the driver's own buffer
        self.dx = self.dw = self.db = self.ws = None
        if not forward_only:
            self.dx = self._buffer(self.sx)
            self.dw = torch.empty(self._D, dtype=torch.float32, device=self.device)
            self.db = torch.empty_like(self.dw)
            self.ws = self._workspace(self.ws_bytes)

    def forward(self, x, w=None, b=None, out=None, stream=None):
        if self._away():
            return self._there(self.forward, x, w, b, out, stream)
        D = self._D
        h = self.h if out is None else out
        self._ok(self._norm_fwd(
            self._p, self._act(x, self.sx, "x"), None if w is None else self._vec(w, D, "w"),
            None if b is None else self._vec(b, D, "b"),
            self._h if out is None else self._act(out, self.sh, "out"), self._stream(stream)))
        return h

    def backward(self, x, dh, w=None, b=None, dres=None, out=None, stream=None):
        """(dx, dw, db): gradients of sum(h * dh), with ``dres`` (the gradient
        that reaches x past the norm) added to dx. dw and db are formed where w
        and b are given, else None."""
        if self.ws is None:
            _refuse("Norm", "made forward_only")
        if self._away():
            return self._there(self.backward, x, dh, w, b, dres, out, stream)
        dx = self.dx if out is None else out
        D = self._D
        self._vec(b, D, "b")
        dw, db = None if w is None else self.dw, None if b is None else self.db
        self._ok(self._lib.lsh_norm_bwd(
            self._p, self._act(x, self.sx, "x"), self._vec(w, D, "w"),
            self._act(dh, self.sh, "dh"),
            None if dres is None else self._act(dres, self.sx, "dres"),
            self._act(dx, self.sx, "out"), _lib._ptr(dw), _lib._ptr(db), self.ws.data_ptr(),
            self.ws_bytes, self._stream(stream)))
        return dx, dw, db


class Dropout(_Driver):
    """y = x / (1 - p) where kept, else 0; p is taken to the nearest 2^-16.
    The mask is a function of (seed, offset + counter, position): the same
    arguments give the same mask in any layout, and ``backward`` applies it to
    dy. ``counter`` is an int64 device tensor of one element read when the
    kernel runs (a captured graph's new masks). ``slice0``: global index of
    the first (b, h) slice when ranks hold shards of one problem. Buffers: y, dx."""

    def __init__(self, B, H, L, p, dtype="bf16", d=64, x_layout: Layout = "head",
                 y_layout: Layout = "head", slice0=0, device="cuda"):
        super().__init__(B, H, L, d, dtype, device)
        slice0 = _slice0(slice0, "Dropout")
        self.sx, self.sy = self._strides(x_layout), self._strides(y_layout)
        self.p = _lib.make_dropout_problem(B, H, L, d, dtype, p, slice0, self.sx[:3], self.sy[:3])
        self.p_bwd = _lib.make_dropout_problem(B, H, L, d, dtype, p, slice0, self.sy[:3],
                                               self.sx[:3])
        if not 0.0 <= p <= 1.0:
            _refuse("Dropout", f"p {p}")
        self.y = self._buffer(self.sy)
        self.dx = self._buffer(self.sx)

    def _run(self, q, src, sx, dst, sy, seed, offset, counter, stream):
        if self._away():
            return self._there(self._run, q, src, sx, dst, sy, seed, offset, counter, stream)
        self._ok(self._lib.lsh_dropout_fwd(
            ctypes.byref(q), self._act(src, sx, "input"), _seed(seed, "Dropout"),
            _seed(offset, "Dropout"), self._vec(counter, (1,), "counter", torch.int64),
            self._act(dst, sy, "out"), self._stream(stream)))
        return dst

    def forward(self, x, seed, offset=0, counter=None, out=None, stream=None):
        return self._run(self.p, x, self.sx, self.y if out is None else out, self.sy, seed, offset,
                         counter, stream)

    def backward(self, dy, seed, offset=0, counter=None, out=None, stream=None):
        return self._run(self.p_bwd, dy, self.sy, self.dx if out is None else out, self.sx, seed,
                         offset, counter, stream)


class Residual(_Driver):
    """y = beta x + alpha drop(gate u), u = post(f); h = norm(y as stored).

    post, norm: None, "layer" or "rms". gate: None; "vector", float32 [H d]
    (with gate_batch [B, H d]); "sigmoid", 1 / (1 + exp(-z)) of an activation
    z. p: dropout (see ``Dropout``). x, y, h and their gradients are in
    ``x_layout``; f, z and theirs in ``f_layout``. Buffers: y, h, x (restore),
    dx, df, dgate, dw_post, db_post, dw, db and the backward's workspace."""

    def __init__(self, B, H, L, post=None, norm=None, gate=None, gate_batch=False, p=0.0,
                 alpha=1.0, beta=1.0, eps=1e-5, dtype="bf16", d=64, x_layout: Layout = "head",
                 f_layout: Layout = "head", slice0=0, device="cuda"):
        super().__init__(B, H, L, d, dtype, device)
        if post not in _KINDS or norm not in _KINDS or gate not in _GATES:
            _refuse("Residual", f"post {post!r}, norm {norm!r}, gate {gate!r}")
        self.post, self.norm, self.gate = post, norm, gate
        slice0 = _slice0(slice0, "Residual")
        self.sx, self.sf = self._strides(x_layout), self._strides(f_layout)

        def problem(norm, alpha, beta):
            return _lib.make_residual_problem(B, H, L, d, dtype, _KINDS[post], _KINDS[norm],
                                              _GATES[gate], gate_batch, eps, eps, alpha, beta, p,
                                              slice0, self.sx[:3], self.sf[:3])

        self.p = problem(norm, alpha, beta)
        # x from y: the same branch taken off, and the scale undone
        self.p_restore = problem(None, -alpha / beta, 1.0 / beta) if beta != 0 else None
        self.ws_bytes = self._sized(_lib.lsh_residual_bwd_workspace_size(self.p))
        self._p, self._residual_fwd = ctypes.byref(self.p), self._lib.lsh_residual_fwd
        self._D = (self.H * self.d,)
        self.gate_shape = (self.B, self._D[0]) if gate_batch else self._D
        f32 = dict(dtype=torch.float32, device=self.device)
        self.y = self._buffer(self.sx)
        self.h = self._buffer(self.sx) if norm else None
        # of the driver's own buffers
        self._y, self._h = self.y.data_ptr(), None if self.h is None else self.h.data_ptr()
        self.x = self._buffer(self.sx)
        self.dx = self._buffer(self.sx)
        self.df = self._buffer(self.sf)
        self.dgate = self._buffer(self.sf) if gate == "sigmoid" else \
            torch.empty(self.gate_shape, **f32) if gate == "vector" else None
        self.dw_post, self.db_post = ((torch.empty(self._D, **f32) for _ in range(2)) if post
                                      else (None, None))
        self.dw, self.db = ((torch.empty(self._D, **f32) for _ in range(2)) if norm
                            else (None, None))
        self.ws = self._workspace(self.ws_bytes)

    def _params(self, gate, w_post, b_post, w, b):
        """Addresses of the gate and the parameters."""
        if gate is None:
            if self.gate is not None:
                _refuse("Residual", f"gate is {self.gate!r}")
        elif self.gate == "vector":
            gate = self._vec(gate, self.gate_shape, "gate")
        elif self.gate == "sigmoid":
            gate = self._act(gate, self.sf, "gate")
        else:
            _refuse("Residual", "made without a gate")
        if not self.post and (w_post is not None or b_post is not None):
            _refuse("Residual", "w_post, b_post without a norm of f")
        if not self.norm and (w is not None or b is not None):
            _refuse("Residual", "w, b without a norm of y")
        D, vec = self._D, self._vec
        return (gate, None if w_post is None else vec(w_post, D, "w_post"),
                None if b_post is None else vec(b_post, D, "b_post"),
                None if w is None else vec(w, D, "w"), None if b is None else vec(b, D, "b"))

    def forward(self, x, f, gate=None, w_post=None, b_post=None, w=None, b=None, seed=0, offset=0,
                counter=None, stream=None):
        """(y, h); h is None without a norm."""
        if self._away():
            return self._there(self.forward, x, f, gate, w_post, b_post, w, b, seed, offset,
                               counter, stream)
        self._ok(self._residual_fwd(
            self._p, self._act(x, self.sx, "x"), self._act(f, self.sf, "f"),
            *self._params(gate, w_post, b_post, w, b), _seed(seed, "Residual"),
            _seed(offset, "Residual"),
            None if counter is None else self._vec(counter, (1,), "counter", torch.int64),
            self._y, self._h, self._stream(stream)))
        return self.y, self.h

    def restore(self, y, f, gate=None, w_post=None, b_post=None, seed=0, offset=0, counter=None,
                stream=None):
        """x = (y - alpha drop(gate u)) / beta: the residual input of ``forward``
        from its output, with the same branch, seed and offset."""
        if self.p_restore is None:
            _refuse("Residual", "beta = 0 cannot be undone")
        if self._away():
            return self._there(self.restore, y, f, gate, w_post, b_post, seed, offset, counter,
                               stream)
        self._ok(self._residual_fwd(
            ctypes.byref(self.p_restore), self._act(y, self.sx, "y"), self._act(f, self.sf, "f"),
            *self._params(gate, w_post, b_post, None, None), _seed(seed, "Residual"),
            _seed(offset, "Residual"), self._vec(counter, (1,), "counter", torch.int64),
            self.x.data_ptr(), None, self._stream(stream)))
        return self.x

    def backward(self, dy, f, y=None, dh=None, gate=None, w_post=None, b_post=None, w=None, b=None,
                 seed=0, offset=0, counter=None, stream=None):
        """(dx, df, dgate, dw_post, db_post, dw, db): gradients of sum(y * dy) +
        sum(h * dh). y (forward's) and dh are needed with a norm, where dy may
        be None (zeros). Parameter gradients are formed for the parameters
        given, else None."""
        if self._away():
            return self._there(self.backward, dy, f, y, dh, gate, w_post, b_post, w, b, seed,
                               offset, counter, stream)
        p_gate, p_wp, p_bp, p_w, _ = self._params(gate, w_post, b_post, w, b)
        p_y = p_dh = None
        if self.norm:
            if y is None or dh is None:
                _refuse("Residual", "the backward of a norm needs y and dh")
            p_y, p_dh = self._act(y, self.sx, "y"), self._act(dh, self.sx, "dh")
        elif dh is not None or dy is None:
            _refuse("Residual", "without a norm of y the gradient is dy alone")
        dw_post = None if w_post is None else self.dw_post
        db_post = None if b_post is None else self.db_post
        dw, db = None if w is None else self.dw, None if b is None else self.db
        ptr = _lib._ptr
        self._ok(self._lib.lsh_residual_bwd(
            self._p, None if dy is None else self._act(dy, self.sx, "dy"), p_dh, p_y,
            self._act(f, self.sf, "f"), p_gate, p_wp, p_bp, p_w, _seed(seed, "Residual"),
            _seed(offset, "Residual"), self._vec(counter, (1,), "counter", torch.int64),
            self.dx.data_ptr(), self.df.data_ptr(), ptr(self.dgate), ptr(dw_post), ptr(db_post),
            ptr(dw), ptr(db), self.ws.data_ptr(), self.ws_bytes, self._stream(stream)))
        return self.dx, self.df, self.dgate, dw_post, db_post, dw, db


# Frequencies and tables are formed with 60 digits: a phase is off by the
# position times the table's error, so a double's 53 bits would show from
# position 2^31 on.
_DIGITS = decimal.Context(prec=60)
_TWO_PI = decimal.Decimal("6.28318530717958647692528676655900576839433879875021164194989")


def _frequencies(rot, base, scaling):
    """``rope_frequencies`` as decimals."""
    rot, base = int(rot), float(base)
    if rot < 2 or rot % 2:
        _refuse("rope_frequencies", f"rot {rot}")
    if not (base > 0 and math.isfinite(base)):
        _refuse("rope_frequencies", f"base {base}")
    kind = None if scaling is None else scaling[0]
    if kind not in (None, "linear", "ntk", "yarn") or \
            (kind and (len(scaling) != (3 if kind == "yarn" else 2) or
                       not all(0 < v < math.inf for v in scaling[1:]))) or \
            (kind == "ntk" and rot == 2):
        _refuse("rope_frequencies", f"scaling {scaling!r}")
    with decimal.localcontext(_DIGITS):
        D = decimal.Decimal
        amp, b = 1.0, D(base)
        s = D(float(scaling[1])) if kind else D(1)
        if kind == "ntk":
            b *= s ** (D(rot) / (rot - 2))
        step, f = b ** (D(-2) / rot), [D(1)]   # one power: each takes 30 us
        while len(f) < rot // 2:
            f.append(f[-1] * step)
        if kind == "linear":
            f = [v / s for v in f]
        elif kind == "yarn":
            turns = D(float(scaling[2])) / _TWO_PI
            for i, v in enumerate(f):
                keep = min(D(1), max(D(0), (turns * v - 1) / 31))
                f[i] = v * keep + v / s * (1 - keep)
            amp = 0.1 * math.log(float(scaling[1])) + 1.0
        return f, amp


def rope_frequencies(rot, base=10000.0, scaling=None):
    """(frequencies, amp): radians a position of the rot / 2 pairs, base^(-2i /
    rot), and the multiplier of the turned features. scaling for contexts
    longer than the trained one by a factor s:

      ("linear", s)       positions divided by s (Chen et al. 2023);
      ("ntk", s)          base s^(rot / (rot - 2)): the slowest pair slows by s,
                          the fastest not at all;
      ("yarn", s, L0)     pairs that turn more than 32 times in the trained
                          length L0 keep their frequency, those that turn less
                          than once are divided by s, a linear ramp between;
                          amp = 0.1 ln s + 1 (Peng et al. 2023)."""
    f, amp = _frequencies(rot, base, scaling)
    return [float(v) for v in f], amp


def rope_turns(frequencies) -> torch.Tensor:
    """Frequencies (radians a position; floats, or decimals) as 64-bit fractions
    of a turn, to the nearest: the bits of an unsigned number in an int64 tensor
    (what ``lsh_rope_fwd`` reads)."""
    out = []
    with decimal.localcontext(_DIGITS):
        for f in frequencies:
            v = f if isinstance(f, decimal.Decimal) else decimal.Decimal(float(f))
            if not v.is_finite():
                _refuse("rope_turns", f"frequency {f}")
            t = v / _TWO_PI
            n = int(((t - t.to_integral_value()) * (1 << 64)).to_integral_value()) % (1 << 64)
            out.append(n - (1 << 64) if n >> 63 else n)
    return torch.tensor(out, dtype=torch.int64)


class Rotary(_Driver):
    """Rotary positions on the first ``rot`` features of every head row:
    pairs (2i, 2i + 1) when ``interleaved``, else (i, i + rot / 2), turned by
    position * frequency; the rest is copied. ``frequencies`` overrides those
    of ``base`` and ``scaling`` (see ``rope_frequencies``). Buffers: y, dx."""

    def __init__(self, B, H, L, rot=None, interleaved=False, base=10000.0, scaling=None,
                 frequencies=None, amp=None, dtype="bf16", d=64, x_layout: Layout = "head",
                 y_layout: Layout = "head", device="cuda"):
        super().__init__(B, H, L, d, dtype, device)
        self.rot = self.d if rot is None else int(rot)
        if self.rot < 2 or self.rot % 2 or self.rot > self.d:
            _refuse("Rotary", f"rot {rot} of {d}")
        if frequencies is None:
            frequencies, a = _frequencies(self.rot, base, scaling)
            amp = a if amp is None else amp
        if len(frequencies) != self.rot // 2:
            _refuse("Rotary", f"{len(frequencies)} frequencies for rot {self.rot}")
        self.amp = 1.0 if amp is None else float(amp)
        self.turns = rope_turns(frequencies).to(self.device)
        self.sx, self.sy = self._strides(x_layout), self._strides(y_layout)
        self.p = [_lib.make_rope_problem(B, H, L, d, dtype, self.rot, interleaved, pb, self.amp,
                                         self.sx[:3], self.sy[:3]) for pb in (0, 1)]
        self._p = [ctypes.byref(q) for q in self.p]
        self._turns = self.turns.data_ptr()   # the driver's own table
        self.y = self._buffer(self.sy)
        self.dx = self._buffer(self.sx)

    def _run(self, fn, src, ss, dst, sd, pos, pos0, stream):
        if self._away():
            return self._there(self._run, fn, src, ss, dst, sd, pos, pos0, stream)
        q = self._p[0]
        if pos is not None:
            if pos.dim() == 2:
                q = self._p[1]
                pos = self._vec(pos, (self.B, self.L), "pos", torch.int32)
            else:
                pos = self._vec(pos, (self.L,), "pos", torch.int32)
        self._ok(fn(q, self._act(src, ss, "input"), self._turns, pos, int(pos0),
                    self._act(dst, sd, "out"), self._stream(stream)))
        return dst

    def forward(self, x, pos=None, pos0=0, out=None, stream=None):
        """Position of token (b, l): pos0 + l, or pos0 + pos[l] / pos[b, l] (int32)."""
        return self._run(self._lib.lsh_rope_fwd, x, self.sx, self.y if out is None else out,
                         self.sy, pos, pos0, stream)

    def backward(self, dy, pos=None, pos0=0, out=None, stream=None):
        return self._run(self._lib.lsh_rope_bwd, dy, self.sy, self.dx if out is None else out,
                         self.sx, pos, pos0, stream)

    def backward_sum(self, dqk, dv, pos=None, pos0=0, out=None, stream=None):
        """dx = (backward of dqk) + dv for an activation that fed the attention
        both turned and as it is; dqk, dv: the attention's float32 gradients,
        contiguous."""
        if self._away():
            return self._there(self.backward_sum, dqk, dv, pos, pos0, out, stream)
        dx = self.dx if out is None else out
        f32 = torch.float32
        q, addr = self._p[0], None
        if pos is not None:
            two = pos.dim() == 2
            q = self._p[1] if two else q
            addr = self._vec(pos, (self.B, self.L) if two else (self.L,), "pos", torch.int32)
        self._ok(self._lib.lsh_rope_bwd_sum(
            q, self._vec(dqk, self.shape, "dqk", f32), self._vec(dv, self.shape, "dv", f32),
            self._turns, addr, int(pos0), self._act(dx, self.sx, "out"), self._stream(stream)))
        return dx


class ReversibleLayer(_Driver):
    """One reversible layer with what a trained one has around its sublayers:

      y1 = x1 + alpha drop(gate1 post1(F(n))),  n = norm1(x2)
      y2 = x2 + alpha drop(gate2 post2(G(m))),  m = norm2(y1)

    F is LSH attention with qk = rope(n), v = n (without rotary positions qk =
    n); G the chunked feed-forward. The backward rebuilds x1 and x2 from y1 and
    y2: the dropout masks are recomputed from (seed, offset, position), so
    nothing of the forward is kept but the sort permutation.

    bf16, contiguous [B, H, L, 64]. norm: "layer" or "rms"; post: None or one
    of them; gate: False or True (a learned float32 vector [64 H] for each
    sublayer); rot: rotated features of a head (0: no positions). Parameters
    are a dict: norm1_w, norm2_w (and norm1_b, norm2_b for "layer"), post1_w,
    post2_w (and post1_b, post2_b), gate1, gate2, as far as the layer has them,
    all float32 [64 H], and the feed-forward's W1 [64 H, d_ff], W2 [d_ff, 64 H]
    (bf16), b1, b2 (float32).

    Both sublayers draw from (seed, offset + counter): the attention's mask at
    that offset, the feed-forward's at offset + 2^63; give every layer and step
    its own seed or offset (below 2^63)."""

    def __init__(self, B, H, L, n_buckets, n_rounds, chunk, causal, d_ff, ff_chunk, norm="layer",
                 post=None, gate=False, p=0.0, alpha=1.0, rot=64, interleaved=False, base=10000.0,
                 scaling=None, eps=1e-5, slice0=0, device="cuda"):
        from .attention import LSHAttention
        super().__init__(B, H, L, 64, "bf16", device)
        if norm not in ("layer", "rms"):
            _refuse("ReversibleLayer", f"norm {norm!r}")
        kw = dict(device=self.device)
        self.norm, self.post, self.gate = norm, post, bool(gate)
        self.attn = LSHAttention(B, H, L, n_buckets, n_rounds, chunk, causal, **kw)
        self.f = _lib.make_ff_problem(B, H, L, d_ff, ff_chunk)
        self.ff_ws_bytes = self._sized(_lib.lsh_ff_workspace_size(self.f))
        self.ff_ws = self._workspace(self.ff_ws_bytes)
        self.norm1 = Norm(B, H, L, norm, eps, **kw)
        self.norm2 = Norm(B, H, L, norm, eps, forward_only=True, **kw)
        join = dict(post=post, gate="vector" if gate else None, p=p, alpha=alpha, eps=eps,
                    slice0=slice0, **kw)
        self.join1 = Residual(B, H, L, norm=norm, **join)
        self.join2 = Residual(B, H, L, **join)
        self.rope = Rotary(B, H, L, rot, interleaved, base, scaling, **kw) if rot else None
        if not rot:
            self._sum = _lib.make_rope_problem(B, H, L, 64, "bf16", 0, False, False, 1.0)
        self.D, self.d_ff = 64 * self.H, int(d_ff)
        f32 = dict(dtype=torch.float32, device=self.device)
        act = lambda: self._buffer(self._strides("head"))
        self.g, self.dm = act(), act()
        self.dn = self.rope.dx if rot else act()
        self.dx2 = self.norm1.dx
        self.dW1 = torch.empty((self.D, self.d_ff), **f32)
        self.db1 = torch.empty((self.d_ff,), **f32)
        self.dW2 = torch.empty((self.d_ff, self.D), **f32)
        self.db2 = torch.empty((self.D,), **f32)

    def _check(self, w, acts, seed, counter):
        """All that the calls of a step would refuse, before the first of them."""
        head = self._strides("head")
        for name, t in acts.items():
            self._act(t, head, name)
        want = {"W1", "b1", "W2", "b2"}
        for i in "12":
            want |= {f"norm{i}_w"} | ({f"norm{i}_b"} if self.norm == "layer" else set())
            if self.post:
                want |= {f"post{i}_w"} | ({f"post{i}_b"} if self.post == "layer" else set())
            if self.gate:
                want.add(f"gate{i}")
        if set(w) != want:
            _refuse("ReversibleLayer", f"parameters {sorted(w)}, expected {sorted(want)}")
        bf16, f32 = torch.bfloat16, torch.float32
        ff = dict(W1=((self.D, self.d_ff), bf16), b1=((self.d_ff,), f32),
                  W2=((self.d_ff, self.D), bf16), b2=((self.D,), f32))
        for name in want:
            shape, dtype = ff.get(name, ((self.D,), f32))
            at = self._vec(w[name], shape, name, dtype)
            if at is None and (name in ff or name[:4] == "gate"):
                _refuse("ReversibleLayer", f"{name} is missing")
            if name in ff and at % 16:
                _refuse("ReversibleLayer", f"{name}: its address is not a multiple of 16")
        _seed(seed, "ReversibleLayer")
        self._vec(counter, (1,), "counter", torch.int64)

    def _offsets(self, offset):
        if not 0 <= int(offset) < 1 << 63:
            _refuse("ReversibleLayer", "offset is below 2^63")
        return int(offset), int(offset) + (1 << 63)

    @staticmethod
    def _branch(w, i):
        """The parameters that sublayer i's join takes."""
        return dict(gate=w.get(f"gate{i}"), w_post=w.get(f"post{i}_w"),
                    b_post=w.get(f"post{i}_b"))

    def _attend(self, x2, w, pos0, stream, R=None):
        """F(norm1(x2)); sorts by R's buckets, or keeps the permutation."""
        n = self.norm1.forward(x2, w["norm1_w"], w.get("norm1_b"), stream=stream)
        q = n if self.rope is None else self.rope.forward(n, pos0=pos0, stream=stream)
        if R is not None:
            self.attn.hash(q, R, stream)
            self.attn.sort(None, stream)
        return n, q, self.attn.attend(q, n, None, stream)[0]

    def _feed(self, m, w, stream):
        _lib.lsh_ff_fwd(self.f, m, w["W1"], w["b1"], w["W2"], w["b2"], None, self.g, self.ff_ws,
                        self.ff_ws_bytes, stream)
        return self.g

    def forward(self, x1, x2, R, w, seed=0, offset=0, counter=None, pos0=0, stream=None):
        """(y1, y2); R [n_rounds, 64, n_buckets / 2] bf16. Token l of every
        sequence has position pos0 + l."""
        if self._away():
            return self._there(self.forward, x1, x2, R, w, seed, offset, counter, pos0, stream)
        self._check(w, dict(x1=x1, x2=x2), seed, counter)
        o1, o2 = self._offsets(offset)
        p = self.attn.p
        if R is None:
            _refuse("ReversibleLayer", "R is missing")
        self._vec(R, (p.n_rounds, 64, p.n_buckets // 2), "R", torch.bfloat16)
        _, _, f = self._attend(x2, w, pos0, stream, R)
        rng = dict(seed=seed, counter=counter, stream=stream)
        y1, m = self.join1.forward(x1, f, **self._branch(w, 1), w=w["norm2_w"], b=w.get("norm2_b"),
                                   offset=o1, **rng)
        y2, _ = self.join2.forward(x2, self._feed(m, w, stream), **self._branch(w, 2), offset=o2,
                                   **rng)
        return y1, y2

    def backward(self, y1, y2, dy1, dy2, w, seed=0, offset=0, counter=None, pos0=0, stream=None):
        """(x1, x2, dx1, dx2, grads): the inputs rebuilt from the outputs and
        the gradients of sum(y1 dy1) + sum(y2 dy2); grads is a dict like w, all
        float32. Uses the permutation of the last forward of this driver."""
        if self._away():
            return self._there(self.backward, y1, y2, dy1, dy2, w, seed, offset, counter, pos0,
                               stream)
        self._check(w, dict(y1=y1, y2=y2, dy1=dy1, dy2=dy2), seed, counter)
        o1, o2 = self._offsets(offset)
        rng = dict(seed=seed, counter=counter, stream=stream)
        b1, b2 = self._branch(w, 1), self._branch(w, 2)
        # feed-forward half: x2 = y2 - branch(G(m)), then G's gradients
        m = self.norm2.forward(y1, w["norm2_w"], w.get("norm2_b"), stream=stream)
        g = self._feed(m, w, stream)
        x2 = self.join2.restore(y2, g, **b2, offset=o2, **rng)
        dx2, dg, *d2 = self.join2.backward(dy2, g, **b2, offset=o2, **rng)
        _lib.lsh_ff_bwd(self.f, m, w["W1"], w["b1"], w["W2"], w["b2"], dg, None, None, None,
                        self.dm, self.dW1, self.db1, self.dW2, self.db2, self.ff_ws,
                        self.ff_ws_bytes, stream)
        # attention half: F(norm1(x2)) again, x1 = y1 - branch(F), F's gradients
        n, q, f = self._attend(x2, w, pos0, stream)
        x1 = self.join1.restore(y1, f, **b1, offset=o1, **rng)
        dx1, df, *d1 = self.join1.backward(dy1, f, y=y1, dh=self.dm, **b1, w=w["norm2_w"],
                                           b=w.get("norm2_b"), offset=o1, **rng)
        dqk, dv = self.attn.backward(q, n, df, None, stream)
        if self.rope is not None:
            dn = self.rope.backward_sum(dqk, dv, pos0=pos0, stream=stream)
        else:
            dn = self.dn
            _lib.lsh_rope_bwd_sum(self._sum, dqk, dv, None, None, 0, dn, stream)
        _, dw, db = self.norm1.backward(x2, dn, w["norm1_w"], w.get("norm1_b"), dres=dx2,
                                        stream=stream)
        grads = dict(W1=self.dW1, b1=self.db1, W2=self.dW2, b2=self.db2, norm1_w=dw, norm1_b=db,
                     gate1=d1[0], post1_w=d1[1], post1_b=d1[2], norm2_w=d1[3], norm2_b=d1[4],
                     gate2=d2[0], post2_w=d2[1], post2_b=d2[2])
        return x1, x2, dx1, self.dx2, {k: v for k, v in grads.items() if v is not None}
