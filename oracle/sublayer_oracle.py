"""float64 CPU oracle of the operators around a sublayer: norms, the residual
add with gate and dropout, dropout's mask, rotary positions.

Plain numpy, written from the definitions; shares no code with the CUDA path.
Activations are [B, H, L, d]; a norm runs over a token's (h, c).
"""
from __future__ import annotations

import numpy as np

from oracle import lsh_oracle as lsh
from oracle import rev_ff_oracle as ff

M32 = 0xFFFFFFFF


def philox4x32(n, seed, offset):
    """Philox4x32-10 (Salmon et al., SC 2011) of the 64-bit counters n: the
    four words [len(n), 4]. Counter (n, offset), key seed, low words first."""
    u = np.uint64
    n = np.asarray(n, dtype=u)
    x = [n & u(M32), n >> u(32), np.full_like(n, offset & M32), np.full_like(n, offset >> 32)]
    k0, k1 = seed & M32, seed >> 32
    for _ in range(10):
        p, q = x[0] * u(0xD2511F53), x[2] * u(0xCD9E8D57)
        x = [(q >> u(32)) ^ x[1] ^ u(k0), q & u(M32), (p >> u(32)) ^ x[3] ^ u(k1), p & u(M32)]
        k0, k1 = (k0 + 0x9E3779B9) & M32, (k1 + 0xBB67AE85) & M32
    return np.stack(x, -1)


def dropout_factor(shape, p, seed, offset=0, slice0=0):
    """Multiplier of every element: 0 or 1 / (1 - p), p to the nearest 2^-16."""
    B, H, L, d = shape
    g = -(-d // 8)
    rows = np.arange(B * H * L, dtype=np.uint64) + np.uint64(slice0 * L)
    ctr = (rows[:, None] * np.uint64(g) + np.arange(g, dtype=np.uint64)).reshape(-1)
    w = philox4x32(ctr, seed, offset)
    lanes = np.stack([w & np.uint64(0xFFFF), w >> np.uint64(16)], -1).reshape(B * H * L, 8 * g)
    t = int(np.rint(np.float64(np.float32(p)) * 65536))
    keep = lanes[:, :d].astype(np.int64) >= t
    return (keep * (65536.0 / (65536 - t) if t < 65536 else 0.0)).reshape(shape)


def norm_stats(x, kind, eps):
    m = x.mean((1, 3), keepdims=True) if kind == "layer" else 0.0
    r = 1.0 / np.sqrt(((x - m) ** 2).mean((1, 3), keepdims=True) + eps)
    return (x - m) * r, r


def _p(v, shape):
    """A [D] or [B, D] vector against [B, H, L, d]."""
    return v.reshape(-1, shape[1], 1, shape[3])


def norm_forward(x, kind, eps, w=None, b=None):
    h, _ = norm_stats(x, kind, eps)
    if w is not None:
        h = h * _p(w, x.shape)
    return h if b is None else h + _p(b, x.shape)


def norm_backward(x, kind, eps, w, dh, dres=None):
    """(dx, dw, db)"""
    xhat, r = norm_stats(x, kind, eps)
    a = dh if w is None else dh * _p(w, x.shape)
    g = a - xhat * (a * xhat).mean((1, 3), keepdims=True)
    if kind == "layer":
        g = g - a.mean((1, 3), keepdims=True)
    dx = r * g + (0.0 if dres is None else dres)
    D = x.shape[1] * x.shape[3]
    return dx, (dh * xhat).sum((0, 2)).reshape(D), dh.sum((0, 2)).reshape(D)


def _gate(gate, kind, shape):
    if kind == "vector":
        return _p(gate, shape)
    if kind == "sigmoid":
        return 1.0 / (1.0 + np.exp(-gate))
    return 1.0


def residual_forward(x, f, post=None, gate=None, kind=None, alpha=1.0, beta=1.0, eps=1e-5,
                     w_post=None, b_post=None, factor=1.0):
    """y; ``kind`` says what ``gate`` is, ``factor`` is dropout_factor's."""
    u = norm_forward(f, post, eps, w_post, b_post) if post else f
    return beta * x + alpha * factor * _gate(gate, kind, f.shape) * u


def residual_backward(dy, dh, y, f, post=None, norm=None, gate=None, kind=None, alpha=1.0,
                      beta=1.0, eps=1e-5, w_post=None, b_post=None, w=None, factor=1.0,
                      gate_batch=False):
    """dict: dx, df, and dgate, dw_post, db_post, dw, db where they exist."""
    out = {}
    t = np.zeros_like(f) if dy is None else dy
    if norm:
        g, out["dw"], out["db"] = norm_backward(y, norm, eps, w, dh)
        t = t + g
    out["dx"] = beta * t
    q = alpha * factor * t
    u = norm_forward(f, post, eps, w_post, b_post) if post else f
    D = f.shape[1] * f.shape[3]
    if kind == "vector":
        dg = (q * u).sum(2).reshape(-1, D)
        out["dgate"] = dg if gate_batch else dg.sum(0)
    elif kind == "sigmoid":
        s = _gate(gate, kind, f.shape)
        out["dgate"] = q * u * s * (1.0 - s)
    du = q * _gate(gate, kind, f.shape)
    if post:
        out["df"], out["dw_post"], out["db_post"] = norm_backward(f, post, eps, w_post, du)
    else:
        out["df"] = du
    return out


def rope(x, freqs, pos, rot, interleaved=False, amp=1.0, inverse=False):
    """pos: integers [B, L] or [L]."""
    a = np.asarray(pos, dtype=np.float64)[..., None] * np.asarray(freqs, dtype=np.float64)
    if a.ndim == 2:
        a = a[None]
    c, s = amp * np.cos(a)[:, None], amp * np.sin(a)[:, None] * (-1.0 if inverse else 1.0)
    y = np.array(x, dtype=np.float64)
    i = np.arange(rot // 2)
    lo, hi = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    y[..., lo] = x[..., lo] * c - x[..., hi] * s
    y[..., hi] = x[..., hi] * c + x[..., lo] * s
    return y


# --------------------------------------------------------------------------
# The reversible layer: y1 = x1 + a drop(g1 post1(F(n))), n = norm1(x2), F =
# attention with qk = rope(n), v = n; y2 = x2 + a drop(g2 post2(G(m))), m =
# norm2(y1). `c` holds the constants: norm, post, gate, alpha, eps, freqs (None:
# no positions), rot, interleaved, amp, pos, chunk, causal, scale, and the two
# sublayers' dropout factors fac1, fac2. `w` holds the parameters by name.
# --------------------------------------------------------------------------

def _turn(x, c, inverse=False):
    if c["freqs"] is None:
        return x
    return rope(x, c["freqs"], c["pos"], c["rot"], c["interleaved"], c["amp"], inverse)


def _join(w, i, c):
    return dict(post=c["post"], gate=w.get(f"gate{i}"), kind="vector" if c["gate"] else None,
                alpha=c["alpha"], eps=c["eps"], w_post=w.get(f"post{i}_w"),
                factor=c[f"fac{i}"])


def _feed(m, w, B, H, L):
    return ff.tokens_to_heads(ff.ff_forward(ff.heads_to_tokens(m), w["W1"], w["b1"], w["W2"],
                                            w["b2"]), B, H, L)


def _norm(x, w, i, c):
    return norm_forward(x, c["norm"], c["eps"], w[f"norm{i}_w"], w.get(f"norm{i}_b"))


def layer_forward(x1, x2, perm, w, c):
    """(y1, y2)"""
    B, H, L, _ = x1.shape
    n = _norm(x2, w, 1, c)
    f, _ = lsh.forward(_turn(n, c), n, perm, c["chunk"], c["causal"], c["scale"])
    y1 = residual_forward(x1, f, **_join(w, 1, c), b_post=w.get("post1_b"))
    g = _feed(_norm(y1, w, 2, c), w, B, H, L)
    return y1, residual_forward(x2, g, **_join(w, 2, c), b_post=w.get("post2_b"))


def layer_backward(y1, y2, dy1, dy2, perm, w, c):
    """(x1, x2, dx1, dx2, grads) from the outputs."""
    B, H, L, _ = y1.shape
    zero = np.zeros_like(y1)
    m = _norm(y1, w, 2, c)
    g = _feed(m, w, B, H, L)
    j2 = _join(w, 2, c)
    x2 = y2 - residual_forward(zero, g, **j2, b_post=w.get("post2_b"))
    r2 = residual_backward(dy2, None, None, g, **j2, b_post=w.get("post2_b"))
    dm, dW1, db1, dW2, db2 = ff.ff_backward(ff.heads_to_tokens(m), w["W1"], w["b1"], w["W2"],
                                            w["b2"], ff.heads_to_tokens(r2["df"]))
    n = _norm(x2, w, 1, c)
    q = _turn(n, c)
    f, lse = lsh.forward(q, n, perm, c["chunk"], c["causal"], c["scale"])
    j1 = _join(w, 1, c)
    x1 = y1 - residual_forward(zero, f, **j1, b_post=w.get("post1_b"))
    r1 = residual_backward(dy1, ff.tokens_to_heads(dm, B, H, L), y1, f, norm=c["norm"],
                           w=w["norm2_w"], **j1, b_post=w.get("post1_b"))
    dqk, dv = lsh.backward(q, n, perm, c["chunk"], c["causal"], c["scale"], f, lse, r1["df"])
    dx2, dw, db = norm_backward(x2, c["norm"], c["eps"], w["norm1_w"], _turn(dqk, c, True) + dv,
                                r2["dx"])
    out = dict(W1=dW1, b1=db1, W2=dW2, b2=db2, norm1_w=dw, norm1_b=db, norm2_w=r1["dw"],
               norm2_b=r1["db"])
    for i, r in ((1, r1), (2, r2)):
        out.update({f"gate{i}": r.get("dgate"), f"post{i}_w": r.get("dw_post"),
                    f"post{i}_b": r.get("db_post")})
    return x1, x2, r1["dx"], dx2, {k: out[k] for k in w}
