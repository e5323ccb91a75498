"""Torch-facing drivers of what surrounds a sublayer: norms, the residual add
with its gate and dropout, dropout alone, and rotary positions.

As in ``attention``: a driver is made for one fixed problem, owns its output
buffers and workspaces (each call overwrites them; calls that overlap on the
GPU, and graphs that are replayed at the same time, need drivers of their
own), and every step runs in liblsh.so. Tensors are views [B, H, L, d] whose
strides are those of the driver's layout:

  "head"           [B, H, L, d] contiguous (the attention's layout);
  "token"          [B, L, H, d] contiguous, seen as [B, H, L, d];
  (sb, sh, sl)     any strides in elements, features adjacent.

A tensor of another shape, type, device or layout raises ``LshError`` before
anything is launched. Parameters and their gradients are float32, contiguous.
Work is queued on ``stream`` (default: the current stream of the driver's
device).
"""
from __future__ import annotations

import math
from typing import Optional, Sequence, Tuple, Union

import torch

from . import _lib

_TORCH_DTYPE = {"f32": torch.float32, "bf16": torch.bfloat16}
_KINDS = {None: _lib.LSH_NORM_NONE, "layer": _lib.LSH_NORM_LAYER, "rms": _lib.LSH_NORM_RMS}
_GATES = {None: _lib.LSH_GATE_NONE, "vector": _lib.LSH_GATE_VECTOR,
          "sigmoid": _lib.LSH_GATE_SIGMOID}
Layout = Union[str, Sequence[int]]


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
        self.dtype = dtype
        self.tdtype = _TORCH_DTYPE[dtype]
        self.shape = (self.B, self.H, self.L, self.d)
        dev = torch.device(device)
        if dev.type == "cuda" and dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self._empty = self.B * self.H * self.L == 0

    def _strides(self, layout: Layout) -> Tuple[int, int, int, int]:
        B, H, L, d = self.shape
        if layout == "head":
            return (H * L * d, L * d, d, 1)
        if layout == "token":
            return (H * L * d, d, H * d, 1)
        if isinstance(layout, str) or len(layout) != 3:
            _refuse(type(self).__name__, f"layout {layout!r}")
        return tuple(int(s) for s in layout) + (1,)

    def _buffer(self, strides) -> torch.Tensor:
        """An activation buffer of the driver's own in the layout's order."""
        B, H, L, d = self.shape
        if strides == self._strides("token"):
            return torch.empty((B, L, H, d), dtype=self.tdtype, device=self.device).transpose(1, 2)
        if strides == self._strides("head"):
            return torch.empty(self.shape, dtype=self.tdtype, device=self.device)
        if self._empty:
            return torch.empty(self.shape, dtype=self.tdtype, device=self.device)
        last = sum((n - 1) * s for n, s in zip(self.shape, strides))
        return torch.empty(last + 1, dtype=self.tdtype, device=self.device).as_strided(
            self.shape, strides)

    def _act(self, t, strides, name):
        """Checks an activation."""
        if t.dtype is not self.tdtype or t.shape != self.shape or t.device != self.device:
            _refuse(type(self).__name__, f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, "
                                         f"expected {self.tdtype} {self.shape} on {self.device}")
        if t.stride() != strides and not self._empty:
            for n, s, want in zip(self.shape, t.stride(), strides):
                if n > 1 and s != want:
                    _refuse(type(self).__name__, f"{name}: strides {t.stride()}, "
                                                 f"the layout's are {strides}")
        return t

    def _vec(self, t, shape, name, dtype=torch.float32):
        if t is not None and (t.dtype is not dtype or t.shape != shape or
                              t.device != self.device or not t.is_contiguous()):
            _refuse(type(self).__name__, f"{name}: {t.dtype} {tuple(t.shape)} on {t.device}, "
                                         f"expected contiguous {dtype} {shape} on {self.device}")
        return t

    def _stream(self, stream):
        """The stream's handle; the driver's device must be the current one."""
        if stream is None:
            return torch._C._cuda_getCurrentRawStream(self.device.index)
        return stream if isinstance(stream, int) else stream.cuda_stream

    def _call(self, fn, *args):
        if torch.cuda.current_device() != self.device.index:
            with torch.cuda.device(self.device):
                code = fn(*args)
        else:
            code = fn(*args)
        if code != 0:
            raise _lib.LshError(code, type(self).__name__)

    def _sized(self, n):
        if n == 0 and not self._empty:
            _refuse(type(self).__name__, "workspace size query (problem rejected)")
        return n

    def _workspace(self, n):
        return torch.empty(max(1, n), dtype=torch.uint8, device=self.device)


def _seed(v, name):
    v = int(v)
    if not 0 <= v < 1 << 64:
        _refuse(name, "seed and offset are unsigned 64-bit numbers")
    return v


class Norm(_Driver):
    """h = xhat w + b over each token's H d features (``kind`` "layer" or
    "rms"). Buffers: h, dx (their layouts), dw, db float32 [H d], and the
    backward's workspace."""

    def __init__(self, B, H, L, kind="layer", eps=1e-5, dtype="bf16", d=64,
                 x_layout: Layout = "head", h_layout: Layout = "head", device="cuda"):
        super().__init__(B, H, L, d, dtype, device)
        if kind not in ("layer", "rms"):
            _refuse("Norm", f"kind {kind!r}")
        self.sx, self.sh = self._strides(x_layout), self._strides(h_layout)
        self.p = _lib.make_norm_problem(B, H, L, d, dtype, _KINDS[kind], eps, self.sx[:3],
                                        self.sh[:3])
        self.ws_bytes = self._sized(_lib.lsh_norm_bwd_workspace_size(self.p))
        self.D = self.H * self.d
        self.h = self._buffer(self.sh)
        self.dx = self._buffer(self.sx)
        self.dw = torch.empty(self.D, dtype=torch.float32, device=self.device)
        self.db = torch.empty_like(self.dw)
        self.ws = self._workspace(self.ws_bytes)

    def forward(self, x, w=None, b=None, out=None, stream=None):
        h = self.h if out is None else self._act(out, self.sh, "out")
        D = (self.D,)
        self._call(_lib.lib().lsh_norm_fwd, self.p, self._act(x, self.sx, "x").data_ptr(),
                   _lib._ptr(self._vec(w, D, "w")), _lib._ptr(self._vec(b, D, "b")),
                   h.data_ptr(), self._stream(stream))
        return h

    def backward(self, x, dh, w=None, b=None, dres=None, out=None, stream=None):
        """(dx, dw, db): gradients of sum(h * dh), with ``dres`` (the gradient
        that reaches x past the norm) added to dx. dw and db are formed where w
        and b are given, else None."""
        dx = self.dx if out is None else self._act(out, self.sx, "out")
        D = (self.D,)
        dw = None if self._vec(w, D, "w") is None else self.dw
        db = None if self._vec(b, D, "b") is None else self.db
        if dres is not None:
            self._act(dres, self.sx, "dres")
        self._call(_lib.lib().lsh_norm_bwd, self.p, self._act(x, self.sx, "x").data_ptr(),
                   _lib._ptr(w), self._act(dh, self.sh, "dh").data_ptr(), _lib._ptr(dres),
                   dx.data_ptr(), _lib._ptr(dw), _lib._ptr(db), self.ws.data_ptr(), self.ws_bytes,
                   self._stream(stream))
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
        self.sx, self.sy = self._strides(x_layout), self._strides(y_layout)
        self.p = _lib.make_dropout_problem(B, H, L, d, dtype, p, slice0, self.sx[:3], self.sy[:3])
        self.p_bwd = _lib.make_dropout_problem(B, H, L, d, dtype, p, slice0, self.sy[:3],
                                               self.sx[:3])
        if not 0.0 <= p <= 1.0:
            _refuse("Dropout", f"p {p}")
        self.y = self._buffer(self.sy)
        self.dx = self._buffer(self.sx)

    def _run(self, q, src, dst, seed, offset, counter, stream):
        self._call(_lib.lib().lsh_dropout_fwd, q, src.data_ptr(), _seed(seed, "Dropout"),
                   _seed(offset, "Dropout"),
                   _lib._ptr(self._vec(counter, (1,), "counter", torch.int64)), dst.data_ptr(),
                   self._stream(stream))
        return dst

    def forward(self, x, seed, offset=0, counter=None, out=None, stream=None):
        y = self.y if out is None else self._act(out, self.sy, "out")
        return self._run(self.p, self._act(x, self.sx, "x"), y, seed, offset, counter, stream)

    def backward(self, dy, seed, offset=0, counter=None, out=None, stream=None):
        dx = self.dx if out is None else self._act(out, self.sx, "out")
        return self._run(self.p_bwd, self._act(dy, self.sy, "dy"), dx, seed, offset, counter,
                         stream)


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
        self.sx, self.sf = self._strides(x_layout), self._strides(f_layout)

        def problem(norm, alpha, beta):
            return _lib.make_residual_problem(B, H, L, d, dtype, _KINDS[post], _KINDS[norm],
                                              _GATES[gate], gate_batch, eps, eps, alpha, beta, p,
                                              slice0, self.sx[:3], self.sf[:3])

        self.p = problem(norm, alpha, beta)
        # x from y: the same branch taken off, and the scale undone
        self.p_restore = problem(None, -alpha / beta, 1.0 / beta) if beta != 0 else None
        self.ws_bytes = self._sized(_lib.lsh_residual_bwd_workspace_size(self.p))
        self.D = self.H * self.d
        self.gate_shape = (self.B, self.D) if gate_batch else (self.D,)
        f32 = dict(dtype=torch.float32, device=self.device)
        self.y = self._buffer(self.sx)
        self.h = self._buffer(self.sx) if norm else None
        self.x = self._buffer(self.sx)
        self.dx = self._buffer(self.sx)
        self.df = self._buffer(self.sf)
        self.dgate = self._buffer(self.sf) if gate == "sigmoid" else \
            torch.empty(self.gate_shape, **f32) if gate == "vector" else None
        self.dw_post, self.db_post = ((torch.empty(self.D, **f32) for _ in range(2)) if post
                                      else (None, None))
        self.dw, self.db = ((torch.empty(self.D, **f32) for _ in range(2)) if norm
                            else (None, None))
        self.ws = self._workspace(self.ws_bytes)

    def _params(self, gate, w_post, b_post, w, b):
        if (gate is None) != (self.gate is None):
            _refuse("Residual", f"gate is {self.gate!r}")
        if gate is not None:
            if self.gate == "sigmoid":
                self._act(gate, self.sf, "gate")
            else:
                self._vec(gate, self.gate_shape, "gate")
        if not self.post and (w_post is not None or b_post is not None):
            _refuse("Residual", "w_post, b_post without a norm of f")
        if not self.norm and (w is not None or b is not None):
            _refuse("Residual", "w, b without a norm of y")
        D = (self.D,)
        for t, name in ((w_post, "w_post"), (b_post, "b_post"), (w, "w"), (b, "b")):
            if t is not None:
                self._vec(t, D, name)

    def _join(self, q, x, f, gate, w_post, b_post, w, b, seed, offset, counter, y, h, stream):
        ptr = _lib._ptr
        self._call(_lib.lib().lsh_residual_fwd, q, x.data_ptr(), f.data_ptr(), ptr(gate),
                   ptr(w_post), ptr(b_post), ptr(w), ptr(b), _seed(seed, "Residual"),
                   _seed(offset, "Residual"), ptr(self._vec(counter, (1,), "counter", torch.int64)),
                   y.data_ptr(), ptr(h), self._stream(stream))

    def forward(self, x, f, gate=None, w_post=None, b_post=None, w=None, b=None, seed=0, offset=0,
                counter=None, stream=None):
        """(y, h); h is None without a norm."""
        self._params(gate, w_post, b_post, w, b)
        self._join(self.p, self._act(x, self.sx, "x"), self._act(f, self.sf, "f"), gate, w_post,
                   b_post, w, b, seed, offset, counter, self.y, self.h, stream)
        return self.y, self.h

    def restore(self, y, f, gate=None, w_post=None, b_post=None, seed=0, offset=0, counter=None,
                stream=None):
        """x = (y - alpha drop(gate u)) / beta: the residual input of ``forward``
        from its output, with the same branch, seed and offset."""
        if self.p_restore is None:
            _refuse("Residual", "beta = 0 cannot be undone")
        self._params(gate, w_post, b_post, None, None)
        self._join(self.p_restore, self._act(y, self.sx, "y"), self._act(f, self.sf, "f"), gate,
                   w_post, b_post, None, None, seed, offset, counter, self.x, None, stream)
        return self.x

    def backward(self, dy, f, y=None, dh=None, gate=None, w_post=None, b_post=None, w=None, b=None,
                 seed=0, offset=0, counter=None, stream=None):
        """(dx, df, dgate, dw_post, db_post, dw, db): gradients of sum(y * dy) +
        sum(h * dh). y (forward's) and dh are needed with a norm, where dy may
        be None (zeros). Parameter gradients are formed for the parameters
        given, else None."""
        self._params(gate, w_post, b_post, w, b)
        if self.norm:
            self._act(y, self.sx, "y")
            self._act(dh, self.sx, "dh")
        elif dh is not None:
            _refuse("Residual", "dh without a norm of y")
        if dy is not None:
            self._act(dy, self.sx, "dy")
        dw_post = None if w_post is None else self.dw_post
        db_post = None if b_post is None else self.db_post
        dw = None if w is None else self.dw
        db = None if b is None else self.db
        ptr = _lib._ptr
        self._call(_lib.lib().lsh_residual_bwd, self.p, ptr(dy), ptr(dh),
                   ptr(y) if self.norm else None, self._act(f, self.sf, "f").data_ptr(), ptr(gate),
                   ptr(w_post), ptr(b_post), ptr(w), _seed(seed, "Residual"),
                   _seed(offset, "Residual"), ptr(self._vec(counter, (1,), "counter", torch.int64)),
                   self.dx.data_ptr(), self.df.data_ptr(), ptr(self.dgate), ptr(dw_post),
                   ptr(db_post), ptr(dw), ptr(db), self.ws.data_ptr(), self.ws_bytes,
                   self._stream(stream))
        return self.dx, self.df, self.dgate, dw_post, db_post, dw, db


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
    rot = int(rot)
    if rot < 2 or rot % 2:
        _refuse("rope_frequencies", f"rot {rot}")
    base, amp = float(base), 1.0
    kind = None if scaling is None else scaling[0]
    if kind not in (None, "linear", "ntk", "yarn") or \
            (kind and (len(scaling) != (3 if kind == "yarn" else 2) or scaling[1] <= 0)) or \
            (kind == "yarn" and scaling[2] <= 0) or (kind == "ntk" and rot == 2):
        _refuse("rope_frequencies", f"scaling {scaling!r}")
    if kind == "ntk":
        base *= float(scaling[1]) ** (rot / (rot - 2))
    f = [base ** (-2.0 * i / rot) for i in range(rot // 2)]
    if kind == "linear":
        f = [v / scaling[1] for v in f]
    elif kind == "yarn":
        s, L0 = float(scaling[1]), float(scaling[2])
        for i, v in enumerate(f):
            keep = min(1.0, max(0.0, (L0 * v / (2 * math.pi) - 1.0) / 31.0))
            f[i] = v * keep + v / s * (1.0 - keep)
        amp = 0.1 * math.log(s) + 1.0
    return f, amp


def rope_turns(frequencies) -> torch.Tensor:
    """Frequencies (radians a position) as 64-bit fractions of a turn, the bits
    of an unsigned number in an int64 tensor (what ``lsh_rope_fwd`` reads)."""
    out = []
    for f in frequencies:
        t = f / (2.0 * math.pi)
        if not math.isfinite(t):
            _refuse("rope_turns", f"frequency {f}")
        n = int(math.ldexp(t - math.floor(t), 64)) & ((1 << 64) - 1)
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
            frequencies, a = rope_frequencies(self.rot, base, scaling)
            amp = a if amp is None else amp
        if len(frequencies) != self.rot // 2:
            _refuse("Rotary", f"{len(frequencies)} frequencies for rot {self.rot}")
        self.amp = 1.0 if amp is None else float(amp)
        self.turns = rope_turns(frequencies).to(self.device)
        self.sx, self.sy = self._strides(x_layout), self._strides(y_layout)
        self.p = [_lib.make_rope_problem(B, H, L, d, dtype, self.rot, interleaved, pb, self.amp,
                                         self.sx[:3], self.sy[:3]) for pb in (0, 1)]
        self.y = self._buffer(self.sy)
        self.dx = self._buffer(self.sx)

    def _run(self, fn, src, dst, pos, pos0, stream):
        q = self.p[0]
        if pos is not None:
            if pos.dim() == 2:
                q = self.p[1]
                self._vec(pos, (self.B, self.L), "pos", torch.int32)
            else:
                self._vec(pos, (self.L,), "pos", torch.int32)
        self._call(fn, q, src.data_ptr(), self.turns.data_ptr(), _lib._ptr(pos), int(pos0),
                   dst.data_ptr(), self._stream(stream))
        return dst

    def forward(self, x, pos=None, pos0=0, out=None, stream=None):
        """Position of token (b, l): pos0 + l, or pos0 + pos[l] / pos[b, l] (int32)."""
        y = self.y if out is None else self._act(out, self.sy, "out")
        return self._run(_lib.lib().lsh_rope_fwd, self._act(x, self.sx, "x"), y, pos, pos0, stream)

    def backward(self, dy, pos=None, pos0=0, out=None, stream=None):
        dx = self.dx if out is None else self._act(out, self.sx, "out")
        return self._run(_lib.lib().lsh_rope_bwd, self._act(dy, self.sy, "dy"), dx, pos, pos0,
                         stream)
