"""The operators around a sublayer on the GPU against the float64 oracle.

Tolerances. An output of type t is off by at most half a step of rounding,
eps_t / 2 of its value (bf16 2^-8, float32 2^-24), plus what float32
arithmetic leaves: n roundings of 2^-24 each on the terms' magnitudes, which
the oracle's inputs give. A row sum of D <= 8192 terms passes at most 16 (a
thread's features) + 5 (shuffles) + 16 (warps) additions; with the products
around it 64 roundings cover any row-wise output, its magnitude being that of
the formula with every term taken absolutely. Sums over T tokens pass at most
T additions of such terms (fewer when threads share them): T + 64 roundings
of the sum of magnitudes."""
import numpy as np
import pytest

from oracle import sublayer_oracle as orc

pytestmark = pytest.mark.gpu
U = 2.0 ** -24
HALF_STEP = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}
K = 64


def _torch():
    import torch
    return torch


def _put(a, dtype, strides=None, lead=0):
    """A device view of `a` with the given strides, `lead` elements into its
    buffer; the float64 array of what it holds."""
    torch = _torch()
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    t = torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(td)
    if strides is not None:
        n = 1 + sum((m - 1) * s for m, s in zip(a.shape, strides))
        buf = torch.zeros(n + lead, dtype=td, device="cuda")
        v = buf[lead:].as_strided(a.shape, strides)
        v.copy_(t)
        t = v
    return t, t.double().cpu().numpy()


def _f32(a):
    torch = _torch()
    t = torch.from_numpy(np.asarray(a)).float().to("cuda")
    return t, t.double().cpu().numpy()


def _close(got, want, dtype, mag, k=K):
    g = got.double().cpu().numpy()
    assert g.shape == want.shape
    tol = HALF_STEP[dtype] * np.abs(want) + k * U * mag
    bad = ~(np.abs(g - want) <= tol)
    assert not bad.any(), (int(bad.sum()), float(np.abs(g - want).max()), float(tol[bad].min()))


def _layouts(name, B, H, L, d):
    """(layout argument, strides)"""
    if name == "head":
        return "head", None
    if name == "token":
        return "token", (H * L * d, d, H * d, 1)
    if name == "slice":      # a third of a fused projection's output
        s = (L * 3 * H * d, d, 3 * H * d, 1)
        return s[:3], s
    s = (H * L * (d + 3) + 5, L * (d + 3), d + 3, 1)      # odd
    return s[:3], s


def _norm_mag(x, kind, eps, w, b):
    """Magnitude of the norm's terms: (|x| + |mean|) r |w| + |b|."""
    m = x.mean((1, 3), keepdims=True) if kind == "layer" else 0 * x
    r = 1 / np.sqrt(((x - m) ** 2).mean((1, 3), keepdims=True) + eps)
    mag = (np.abs(x) + np.abs(x).mean((1, 3), keepdims=True)) * r
    if w is not None:
        mag = mag * np.abs(orc._p(w, x.shape))
    return mag + (0 if b is None else np.abs(orc._p(b, x.shape)))


def _norm_back_mag(x, kind, eps, w, dh):
    xm = _norm_mag(x, kind, eps, None, None)
    _, r = orc.norm_stats(x, kind, eps)
    a = np.abs(dh if w is None else dh * orc._p(w, x.shape))
    return r * (a + a.mean((1, 3), keepdims=True) + xm * (a * xm).mean((1, 3), keepdims=True)), xm


NORM_CASES = [
    # B, H, L, d, dtype, kind, x layout, h layout, lead
    (1, 1, 1, 64, "bf16", "layer", "head", "head", 0),
    (2, 3, 5, 64, "bf16", "rms", "head", "head", 0),
    (1, 8, 131, 64, "bf16", "layer", "head", "token", 0),
    (2, 9, 7, 64, "f32", "layer", "token", "head", 0),          # a CTA a token
    (1, 64, 33, 64, "bf16", "rms", "token", "token", 0),
    (3, 128, 2, 64, "bf16", "layer", "head", "head", 0),        # the widest
    (2, 128, 3, 64, "f32", "rms", "slice", "head", 0),
    (1, 5, 40, 24, "f32", "layer", "slice", "odd", 0),
    (2, 3, 9, 7, "bf16", "layer", "head", "odd", 0),            # odd head size
    (1, 1, 17, 1, "f32", "rms", "head", "head", 0),
    (1, 8, 19, 64, "bf16", "layer", "odd", "head", 0),          # unaligned strides
    (2, 8, 19, 64, "bf16", "rms", "head", "head", 1),           # unaligned pointer
    (1, 127, 2, 63, "bf16", "layer", "head", "token", 0),       # wide and odd
    (1, 8, 10007, 64, "bf16", "layer", "head", "head", 0),      # more tokens than one wave
]


@pytest.mark.parametrize("case", NORM_CASES)
def test_norm(case):
    from efficient_transformer_lsh_b200 import sublayer as sl
    B, H, L, d, dtype, kind, xl, hl, lead = case
    g = np.random.default_rng(H * L + d)
    shape, D, eps = (B, H, L, d), H * d, 1e-5
    (xa, xs), (ha, hs) = _layouts(xl, *shape), _layouts(hl, *shape)
    if lead and xs is None:
        xs = (H * L * d, L * d, d, 1)
    x, x64 = _put(1.5 * g.standard_normal(shape) + 0.3, dtype, xs, lead)
    dh, dh64 = _put(g.standard_normal(shape), dtype, hs)
    dres, dres64 = _put(g.standard_normal(shape), dtype, xs, lead)
    w, w64 = _f32(1 + 0.2 * g.standard_normal(D))
    b, b64 = _f32(0.3 * g.standard_normal(D))
    r = sl.Norm(B, H, L, kind, eps, dtype, d, xa, ha)
    _close(r.forward(x, w, b), orc.norm_forward(x64, kind, eps, w64, b64), dtype,
           _norm_mag(x64, kind, eps, w64, b64))
    _close(r.forward(x), orc.norm_forward(x64, kind, eps), dtype, _norm_mag(x64, kind, eps, None, None))
    dx, dw, db = r.backward(x, dh, w, b, dres)
    ex, ew, eb = orc.norm_backward(x64, kind, eps, w64, dh64, dres64)
    mag, xm = _norm_back_mag(x64, kind, eps, w64, dh64)
    _close(dx, ex, dtype, mag + np.abs(dres64))
    T = B * L + K
    _close(dw, ew, "f32", (np.abs(dh64) * xm).sum((0, 2)).reshape(D), T)
    _close(db, eb, "f32", np.abs(dh64).sum((0, 2)).reshape(D), T)
    first = [t.clone() for t in (dx, dw, db)]
    again = r.backward(x, dh, w, b, dres)
    assert all(_torch().equal(p, q) for p, q in zip(first, again))      # the same every time
    dx, dw, db = r.backward(x, dh)                                       # bare
    assert dw is None and db is None
    mag, _ = _norm_back_mag(x64, kind, eps, None, dh64)
    _close(dx, orc.norm_backward(x64, kind, eps, None, dh64)[0], dtype, mag)
    if hs == xs and not lead:                                            # in place
        y = x.clone() if xs is None else _put(x64, dtype, xs)[0]
        want = r.forward(x, w, b).clone()
        assert _torch().equal(r.forward(y, w, b, out=y), want)


def _residual_inputs(g, shape, dtype, post, norm, gate, gate_batch, xs, fs, lead=0):
    B, H, L, d = shape
    D = H * d
    t = {}
    for name, st in (("x", xs), ("f", fs), ("dy", xs), ("dh", xs), ("y", xs)):
        t[name] = _put(g.standard_normal(shape) * 1.2 + 0.2, dtype, st, lead)
    gt = {None: (None, None), "vector": _f32(0.7 + 0.2 * g.standard_normal((B, D) if gate_batch else D)),
          "sigmoid": _put(2 * g.standard_normal(shape), dtype, fs)}[gate]
    t["gate"] = gt
    for name, on in (("w_post", post), ("b_post", post == "layer"), ("w", norm),
                     ("b", norm == "layer")):
        t[name] = _f32((1.0 if name[0] == "w" else 0.0) + 0.2 * g.standard_normal(D)) if on \
            else (None, None)
    return t


RES_CASES = [
    # B, H, L, d, dtype, post, norm, gate, gate_batch, p, alpha, beta, x layout, f layout, lead
    (1, 1, 1, 64, "bf16", "layer", "layer", "vector", False, 0.1, 0.5, 1.0, "head", "head", 0),
    (2, 8, 65, 64, "bf16", "layer", "rms", "vector", False, 0.1, 0.5, 1.0, "head", "head", 0),
    (3, 8, 33, 64, "bf16", "rms", "layer", "vector", True, 0.25, 1.0, 1.5, "token", "head", 0),
    (2, 5, 101, 64, "f32", None, "rms", "sigmoid", False, 0.05, 1.0, 1.0, "head", "token", 0),
    (2, 3, 7, 64, "f32", "rms", None, "sigmoid", False, 0.5, -0.7, 0.5, "head", "head", 0),
    (1, 8, 50, 64, "bf16", None, None, None, False, 0.1, 1.0, 1.0, "head", "head", 0),
    (1, 8, 50, 64, "bf16", None, "layer", None, False, 0.0, 1.0, 1.0, "slice", "head", 0),
    (2, 4, 9, 64, "bf16", None, None, "vector", True, 0.0, 2.0, 1.0, "head", "slice", 0),
    (1, 40, 11, 64, "bf16", "layer", "layer", "sigmoid", False, 0.1, 1.0, 1.0, "token", "token", 0),
    (2, 128, 3, 64, "f32", "layer", "rms", "vector", True, 0.1, 1.0, 1.0, "head", "token", 0),
    (2, 3, 9, 7, "bf16", "layer", "rms", "vector", False, 0.3, 1.0, 1.0, "head", "odd", 0),
    (1, 100, 3, 33, "f32", "rms", "layer", "sigmoid", False, 0.2, 1.0, 1.0, "odd", "head", 0),
    (1, 8, 21, 64, "bf16", "rms", "layer", "sigmoid", False, 0.2, 1.0, 1.0, "head", "head", 1),
    (1, 8, 9001, 64, "bf16", "layer", "layer", "vector", False, 0.1, 0.5, 1.0, "head", "head", 0),
    (100, 2, 3, 64, "bf16", "layer", "rms", "vector", True, 0.1, 1.0, 1.0, "head", "head", 0),
    (17, 1, 40, 64, "f32", None, "layer", "vector", True, 0.0, 1.0, 1.0, "head", "head", 0),
    (16, 9, 1, 64, "bf16", "rms", None, "vector", True, 0.0, 1.0, 1.0, "token", "token", 0),
    # wide rows: teams of several warps with several rounds, each form of the backward
    (1, 64, 700, 64, "bf16", "layer", "layer", "vector", False, 0.1, 0.5, 1.0, "head", "token", 0),
    (1, 49, 350, 64, "bf16", "rms", None, None, False, 0.0, 1.0, 1.0, "token", "head", 0),
    (1, 128, 320, 64, "bf16", "layer", "rms", None, False, 0.1, 1.0, 0.5, "head", "head", 0),
    (1, 64, 640, 64, "bf16", "layer", "layer", "sigmoid", False, 0.1, 1.0, 1.0, "head", "head", 0),
    (1, 64, 640, 64, "f32", "rms", "layer", "vector", False, 0.1, 1.0, 1.0, "token", "token", 0),
    (2, 32, 450, 64, "bf16", "layer", None, "sigmoid", False, 0.0, 1.0, 1.0, "head", "head", 0),
    # parameter gradients of wide rows whose last block of features is not full
    (1, 33, 333, 72, "bf16", "layer", "layer", "vector", False, 0.1, 1.0, 1.0, "head", "head", 0),
    (17, 33, 3, 72, "f32", "layer", "layer", "vector", True, 0.1, 1.0, 1.0, "head", "head", 0),
]


@pytest.mark.parametrize("case", RES_CASES)
def test_residual(case):
    from efficient_transformer_lsh_b200 import sublayer as sl
    torch = _torch()
    B, H, L, d, dtype, post, norm, gate, gb, p, alpha, beta, xl, fl, lead = case
    g = np.random.default_rng(H * L + d + B)
    shape, D, eps = (B, H, L, d), H * d, 1e-5
    (xa, xs), (fa, fs) = _layouts(xl, *shape), _layouts(fl, *shape)
    if lead:
        xs = fs = (H * L * d, L * d, d, 1)
    t = _residual_inputs(g, shape, dtype, post, norm, gate, gb, xs, fs, lead)
    T = {k: v[0] for k, v in t.items()}
    N = {k: v[1] for k, v in t.items()}
    seed, off = (1 << 63) + 12345, (1 << 33) + 5
    r = sl.Residual(B, H, L, post, norm, gate, gb, p, alpha, beta, eps, dtype, d, xa, fa)
    par = {k: T[k] for k in ("gate", "w_post", "b_post", "w", "b")}
    y, h = r.forward(T["x"], T["f"], **par, seed=seed, offset=off)
    fac = orc.dropout_factor(shape, p, seed, off)
    y64 = orc.residual_forward(N["x"], N["f"], post, N["gate"], gate, alpha, beta, eps, N["w_post"],
                               N["b_post"], fac)
    gm = np.abs(orc._gate(N["gate"], gate, shape)) if gate else 1.0
    um = _norm_mag(N["f"], post, eps, N["w_post"], N["b_post"]) if post else np.abs(N["f"])
    ymag = abs(beta) * np.abs(N["x"]) + abs(alpha) * fac * gm * um
    _close(y, y64, dtype, ymag)
    ys = y.double().cpu().numpy()
    if norm:
        # h is the norm of y as stored, and bit for bit what the norm alone gives
        _close(h, orc.norm_forward(ys, norm, eps, N["w"], N["b"]), dtype,
               _norm_mag(ys, norm, eps, N["w"], N["b"]))
        # (where both run at the same access width: f alone may be unaligned)
        if fl != "odd" or xl == "odd" or d % 8:
            n = sl.Norm(B, H, L, norm, eps, dtype, d, xa, xa)
            assert torch.equal(n.forward(y, T["w"], T["b"]), h)
    else:
        assert h is None
    # the inverse: y's half step and x's, and the sum's rounding
    x2 = r.restore(y, T["f"], T["gate"], T["w_post"], T["b_post"], seed=seed, offset=off)
    want = (ys - alpha * fac * orc._gate(N["gate"], gate, shape) *
            (orc.norm_forward(N["f"], post, eps, N["w_post"], N["b_post"]) if post else N["f"])) / beta
    _close(x2, want, dtype, ymag / abs(beta) + np.abs(want))

    got = r.backward(T["dy"], T["f"], y=T["y"] if norm else None, dh=T["dh"] if norm else None,
                     **par, seed=seed, offset=off)
    got = dict(zip(("dx", "df", "dgate", "dw_post", "db_post", "dw", "db"), got))
    ref = orc.residual_backward(N["dy"], N["dh"], N["y"], N["f"], post, norm, N["gate"], gate, alpha,
                                beta, eps, N["w_post"], N["b_post"], N["w"], fac, gb)
    tm = np.abs(N["dy"])
    if norm:
        m, ym = _norm_back_mag(N["y"], norm, eps, N["w"], N["dh"])
        tm = tm + m
        _close(got["dw"], ref["dw"], "f32", (np.abs(N["dh"]) * ym).sum((0, 2)).reshape(D), B * L + K)
        if got["db"] is not None:
            _close(got["db"], ref["db"], "f32", np.abs(N["dh"]).sum((0, 2)).reshape(D), B * L + K)
    _close(got["dx"], ref["dx"], dtype, abs(beta) * tm)
    qm = abs(alpha) * fac * tm
    dum = qm * gm
    n = 2 * K                      # two row-wise stages, one after the other
    if post:
        m, fm = _norm_back_mag(N["f"], post, eps, N["w_post"], dum)
        _close(got["df"], ref["df"], dtype, m, n)
        _close(got["dw_post"], ref["dw_post"], "f32", (dum * fm).sum((0, 2)).reshape(D), B * L + n)
        if got["db_post"] is not None:
            _close(got["db_post"], ref["db_post"], "f32", dum.sum((0, 2)).reshape(D), B * L + n)
    else:
        _close(got["df"], ref["df"], dtype, dum, n)
        assert got["dw_post"] is None and got["db_post"] is None
    if gate == "vector":
        mag = (qm * um).sum(2).reshape(-1, D)
        _close(got["dgate"], ref["dgate"], "f32", mag if gb else mag.sum(0), B * L + n)
    elif gate == "sigmoid":
        s = orc._gate(N["gate"], gate, shape)
        _close(got["dgate"], ref["dgate"], dtype, qm * um * s * (1 - s), n)
    else:
        assert got["dgate"] is None
    if norm:
        # no gradient of y: the norm's alone
        dx = r.backward(None, T["f"], y=T["y"], dh=T["dh"], **par, seed=seed, offset=off)[0]
        ref = orc.residual_backward(None, N["dh"], N["y"], N["f"], post, norm, N["gate"], gate,
                                    alpha, beta, eps, N["w_post"], N["b_post"], N["w"], fac, gb)
        _close(dx, ref["dx"], dtype, abs(beta) * tm)


@pytest.mark.parametrize("H,d,dtype,post,norm", [
    (5, 64, "bf16", "layer", "layer"), (3, 64, "f32", "rms", "layer"), (9, 64, "bf16", "rms", "layer"),
    (5, 7, "bf16", "layer", "layer"), (11, 64, "f32", "layer", "rms")])
def test_residual_without_parameters(H, d, dtype, post, norm):
    """Norms with no weights on rows that do not fill their threads: the
    features past the row's end stay out of its sums."""
    from efficient_transformer_lsh_b200 import sublayer as sl
    g = np.random.default_rng(H)
    B, L, eps = 2, 21, 1e-5
    shape = (B, H, L, d)
    (f, f_), (y, y_), (dy, dy_), (dh, dh_) = (_put(g.standard_normal(shape) + 0.4, dtype)
                                              for _ in range(4))
    r = sl.Residual(B, H, L, post, norm, None, dtype=dtype, d=d)
    dx, df, *rest = r.backward(dy, f, y=y, dh=dh)
    assert all(t is None for t in rest)
    ref = orc.residual_backward(dy_, dh_, y_, f_, post, norm, eps=eps)
    m, _ = _norm_back_mag(y_, norm, eps, None, dh_)
    tm = np.abs(dy_) + m
    _close(dx, ref["dx"], dtype, tm)
    _close(df, ref["df"], dtype, _norm_back_mag(f_, post, eps, None, tm)[0], 2 * K)
    out, h = r.forward(y, f)
    want = orc.residual_forward(y_, f_, post, eps=eps)
    _close(out, want, dtype, np.abs(y_) + _norm_mag(f_, post, eps, None, None))
    o = out.double().cpu().numpy()
    _close(h, orc.norm_forward(o, norm, eps), dtype, _norm_mag(o, norm, eps, None, None))


DROP_CASES = [(1, 1, 1, 64, "bf16", 0.1, "head", "head"), (7, 3, 401, 64, "f32", 0.25, "head", "head"),
              (2, 5, 33, 64, "bf16", 0.5, "token", "head"), (2, 3, 11, 7, "bf16", 0.3, "head", "odd"),
              (1, 2, 5, 20, "f32", 0.3, "odd", "token"), (1, 8, 4099, 64, "bf16", 0.1, "head", "head"),
              (2, 2, 3, 64, "bf16", 0.0, "head", "head"), (2, 2, 3, 64, "f32", 1.0, "head", "head"),
              (1, 3, 2, 3000, "bf16", 0.1, "head", "head")]


@pytest.mark.parametrize("case", DROP_CASES)
def test_dropout(case):
    from efficient_transformer_lsh_b200 import sublayer as sl
    B, H, L, d, dtype, p, xl, yl = case
    g = np.random.default_rng(L)
    shape = (B, H, L, d)
    (xa, xs), (ya, ys) = _layouts(xl, *shape), _layouts(yl, *shape)
    x, x64 = _put(g.standard_normal(shape), dtype, xs)
    dy, dy64 = _put(g.standard_normal(shape), dtype, ys)
    seed, off = (0xDEADBEEF << 32) + 77, (1 << 40) + 9
    r = sl.Dropout(B, H, L, p, dtype, d, xa, ya)
    fac = orc.dropout_factor(shape, p, seed, off)
    # one product: float32's rounding of the scale and of the product
    _close(r.forward(x, seed, off), x64 * fac, dtype, np.abs(x64 * fac), 2)
    _close(r.backward(dy, seed, off), dy64 * fac, dtype, np.abs(dy64 * fac), 2)
    counter = _torch().tensor([off - 3], dtype=_torch().int64, device="cuda")
    _close(r.forward(x, seed, 3, counter), x64 * fac, dtype, np.abs(x64 * fac), 2)
    sl0 = sl.Dropout(B, H, L, p, dtype, d, xa, ya, slice0=1234)
    fac = orc.dropout_factor(shape, p, seed, off, slice0=1234)
    _close(sl0.forward(x, seed, off), x64 * fac, dtype, np.abs(x64 * fac), 2)


def test_dropped_elements_are_zero_whatever_they_held():
    from efficient_transformer_lsh_b200 import sublayer as sl
    torch = _torch()
    x = torch.full((1, 2, 50, 64), float("nan"), device="cuda")
    x[0, 1] = float("inf")
    y = sl.Dropout(1, 2, 50, 0.5, "f32").forward(x, 3)
    keep = torch.from_numpy(orc.dropout_factor((1, 2, 50, 64), 0.5, 3) > 0).cuda()
    assert (y[~keep] == 0).all() and not torch.isfinite(y[keep]).any()


ROPE_CASES = [
    # B, H, L, d, dtype, rot, interleaved, scaling, positions, x layout, y layout
    (1, 1, 1, 64, "bf16", 64, False, None, None, "head", "head"),
    (2, 8, 65, 64, "bf16", 64, False, None, None, "head", "head"),
    (2, 8, 65, 64, "bf16", 64, True, None, "batch", "token", "head"),
    (64, 8, 1, 64, "bf16", 64, False, None, "batch", "head", "head"),
    (1, 3, 33, 64, "f32", 32, True, ("yarn", 8.0, 4096), "far", "head", "token"),
    (2, 5, 17, 64, "f32", 64, False, ("linear", 4.0), "far", "slice", "head"),
    (1, 2, 301, 64, "bf16", 20, False, ("ntk", 8.0), "shared", "head", "head"),
    (1, 2, 31, 64, "bf16", 20, True, None, "shared", "head", "head"),
    (1, 2, 31, 64, "bf16", 40, False, None, None, "head", "head"),
    (1, 2, 31, 64, "bf16", 48, False, None, None, "slice", "head"),
    (1, 2, 31, 64, "bf16", 62, False, None, None, "head", "head"),
    (3, 1, 9, 6, "bf16", 2, False, None, None, "head", "odd"),
    (2, 3, 9, 64, "f32", 64, False, None, None, "odd", "head"),
    (1, 70, 3, 128, "bf16", 64, False, None, None, "token", "token"),
    (1, 2, 3, 512, "f32", 2, True, None, "shared", "head", "head"),
    (1, 2, 20011, 64, "bf16", 64, False, None, None, "head", "head"),
    # adjacent pairs at no more than their elements' alignment
    (2, 3, 9, 64, "bf16", 64, True, None, "shared", "odd", "head"),
    (2, 3, 9, 64, "f32", 32, True, None, None, "head", "odd"),
    (1, 2, 5, 10, "bf16", 6, True, None, None, "odd", "odd"),
    (2, 1, 7, 6, "f32", 2, True, None, "batch", "odd", "slice"),
]


@pytest.mark.parametrize("case", ROPE_CASES)
def test_rope(case):
    from efficient_transformer_lsh_b200 import sublayer as sl
    torch = _torch()
    B, H, L, d, dtype, rot, inter, scaling, where, xl, yl = case
    g = np.random.default_rng(L + rot)
    shape = (B, H, L, d)
    (xa, xs), (ya, ys) = _layouts(xl, *shape), _layouts(yl, *shape)
    x, x64 = _put(g.standard_normal(shape), dtype, xs)
    dy, dy64 = _put(g.standard_normal(shape), dtype, ys)
    r = sl.Rotary(B, H, L, rot, inter, scaling=scaling, dtype=dtype, d=d, x_layout=xa, y_layout=ya)
    freqs, amp = sl.rope_frequencies(rot, scaling=scaling)
    pos0 = 11
    pos = {None: None, "batch": g.integers(0, 1 << 20, (B, L)), "shared": g.integers(-99, 99, L),
           "far": g.integers(-(1 << 31), 1 << 31, (B, L))}[where]
    p64 = pos0 + (np.arange(L) if pos is None else pos)
    pt = None if pos is None else torch.from_numpy(pos.astype(np.int32)).cuda()
    # the phase's conversion to float32 (pi 2^-25 of angle), sine, cosine, amp
    # and the products: eight roundings on |p| + |q|. bf16 multiplies the half
    # turns by pi in float32 (pi 2^-24 of angle, and pi's own 2^-25 relative:
    # below 5 roundings) and takes the approximate sine and cosine, on [-pi, pi]
    # off by at most 2^-21.41 and 2^-21.19 (the programming guide's bounds),
    # below 2^-21 = 8 roundings: 21 in all, still 2^-11 of a bf16 half step
    k = 21 if dtype == "bf16" else 8
    pair = lambda a: amp * (_pair_sum(np.abs(a), rot, inter))
    # the oracle's own angle in 64 bits: |pos| freq 2^-52
    far = np.abs(p64).max() * 2.0 ** -51
    _close(r.forward(x, pt, pos0), orc.rope(x64, freqs, p64, rot, inter, amp), dtype,
           pair(x64) * (1 + far / (k * U)), k)
    _close(r.backward(dy, pt, pos0), orc.rope(dy64, freqs, p64, rot, inter, amp, True), dtype,
           pair(dy64) * (1 + far / (k * U)), k)
    if xs == ys:
        want = r.forward(x, pt, pos0).clone()
        z = _put(x64, dtype, xs)[0]
        assert torch.equal(r.forward(z, pt, pos0, out=z), want)


def _pair_sum(a, rot, inter):
    out = a.copy()
    i = np.arange(rot // 2)
    lo, hi = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
    s = a[..., lo] + a[..., hi]
    out[..., lo] = s
    out[..., hi] = s
    return out


def test_rows_between_strided_rows_are_left_as_they_were():
    from efficient_transformer_lsh_b200 import sublayer as sl
    torch = _torch()
    B, H, L, d = 2, 3, 5, 64
    buf = torch.full((B, L, 3, H, d), 7.0, device="cuda", dtype=torch.bfloat16)
    x = torch.randn(B, H, L, d, device="cuda").bfloat16()
    lay = (L * 3 * H * d, d, 3 * H * d)
    out = buf[:, :, 1].transpose(1, 2)
    for run in (lambda: sl.Norm(B, H, L, h_layout=lay).forward(x, out=out),
                lambda: sl.Rotary(B, H, L, y_layout=lay).forward(x, out=out),
                lambda: sl.Dropout(B, H, L, 0.5, y_layout=lay).forward(x, 1, out=out)):
        run()
        assert (buf[:, :, 0] == 7).all() and (buf[:, :, 2] == 7).all()
        assert not (buf[:, :, 1] == 7).all()


def test_offsets_past_32_bits():
    from efficient_transformer_lsh_b200 import sublayer as sl
    torch = _torch()
    B, H, L, d = 2, 2, 3, 64
    far = (1 << 32) + 64                      # elements between the two sequences: 8 GB
    buf = torch.empty(far + H * L * d, dtype=torch.bfloat16, device="cuda")
    big = buf.as_strided((B, H, L, d), (far, L * d, d, 1))
    x = torch.randn(B, H, L, d, device="cuda").bfloat16()
    lay = (far, L * d, d)
    for a, b in ((sl.Norm(B, H, L, x_layout=lay, h_layout=lay), sl.Norm(B, H, L)),
                 (sl.Rotary(B, H, L, x_layout=lay, y_layout=lay), sl.Rotary(B, H, L)),
                 (sl.Dropout(B, H, L, 0.5, x_layout=lay, y_layout=lay), sl.Dropout(B, H, L, 0.5))):
        big.copy_(x)
        args = (5,) if isinstance(a, sl.Dropout) else ()
        assert torch.equal(a.forward(big, *args, out=big), b.forward(x, *args))
        if isinstance(a, sl.Norm):
            big.copy_(x)
            assert torch.equal(a.backward(big, big)[0], b.backward(x, x)[0])
        del a
    assert torch.cuda.max_memory_allocated() < 80 << 30


def test_constant_rows_and_special_values():
    from efficient_transformer_lsh_b200 import sublayer as sl
    torch = _torch()
    x = torch.randn(1, 2, 4, 64, device="cuda")
    x[:, :, 0] = 3.0                          # variance 0: xhat is 0, h is b
    x[0, 1, 1, 5] = float("nan")
    x[0, 0, 2, 9] = float("inf")
    b = torch.randn(128, device="cuda")
    h = sl.Norm(1, 2, 4, "layer", dtype="f32").forward(x, None, b)
    assert torch.equal(h[0, :, 0], b.view(2, 64))
    assert torch.isnan(h[:, :, 1]).all() and torch.isnan(h[:, :, 2]).all()
    assert torch.isfinite(h[:, :, 3]).all()   # and no further than its row
    z = torch.tensor([-float("inf"), float("inf"), -200.0, 200.0], device="cuda").repeat(16)
    z = z.expand(1, 1, 1, 64).contiguous()
    r = sl.Residual(1, 1, 1, gate="sigmoid", dtype="f32")
    y, _ = r.forward(torch.zeros_like(z), torch.ones_like(z), z)
    want = torch.tensor([0.0, 1.0, 0.0, 1.0], device="cuda").repeat(16)
    assert (y.view(-1) - want).abs().max() <= 2.0 ** -24
    dz = r.backward(torch.ones_like(z), torch.ones_like(z), gate=z)[2]
    assert torch.isfinite(dz).all() and dz.abs().max() < 1e-30


@pytest.mark.parametrize("shape", [(0, 2, 3), (2, 2, 0)])
def test_empty_batches_give_zero_parameter_gradients(shape):
    from efficient_transformer_lsh_b200 import sublayer as sl
    torch = _torch()
    B, H, L = shape
    x = torch.empty(B, H, L, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(H * 64, device="cuda")
    n = sl.Norm(B, H, L)
    n.dw.fill_(9), n.db.fill_(9)
    assert n.forward(x, w, w).shape == x.shape
    _, dw, db = n.backward(x, x, w, w)
    assert (dw == 0).all() and (db == 0).all()
    for gb in (False, True):
        r = sl.Residual(B, H, L, "layer", "layer", "vector", gb, 0.1)
        g = torch.ones((B, H * 64) if gb else (H * 64,), device="cuda")
        for t in (r.dw, r.db, r.dw_post, r.db_post, r.dgate):
            t.fill_(9)
        r.forward(x, x, g, w, w, w, w)
        out = r.backward(x, x, x, x, g, w, w, w, w)
        assert all((t == 0).all() for t in out[2:])
    sl.Dropout(B, H, L, 0.1).forward(x, 1)
    sl.Rotary(B, H, L).forward(x)


def test_other_stream_and_captured_graph():
    """A captured forward and backward, replayed with new inputs and a new
    counter on another stream, gives what eager calls give."""
    from efficient_transformer_lsh_b200 import sublayer as sl
    torch = _torch()
    B, H, L = 2, 8, 37
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda: torch.randn(B, H, L, 64, device="cuda", generator=g).bfloat16()
    w = 1 + 0.1 * torch.randn(H * 64, device="cuda", generator=g)
    gate = torch.rand(H * 64, device="cuda", generator=g)
    x, f, dy, dh = rnd(), rnd(), rnd(), rnd()
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")

    def make():
        return (sl.Residual(B, H, L, "rms", "layer", "vector", False, 0.2), sl.Rotary(B, H, L))

    def step(r, e):
        y, h = r.forward(x, f, gate, w, None, w, w, seed=7, counter=counter)
        q = e.forward(h, pos0=3)
        back = e.backward(dh, pos0=3)
        return [y, h, q] + [t for t in r.backward(dy, f, y, back, gate, w, None, w, w, seed=7,
                                                  counter=counter) if t is not None]

    captured, eager = make(), make()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*captured)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = step(*captured)
    side.synchronize()
    previous = None
    for n in range(3):
        for t in (x, f, dy, dh):
            t.copy_(rnd())
        counter.fill_(n)
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        side.synchronize()
        want = step(*eager)
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert previous is None or not torch.equal(previous, outs[0])
        previous = outs[0].clone()


def test_two_drivers_at_once_on_two_streams():
    from efficient_transformer_lsh_b200 import sublayer as sl
    torch = _torch()
    B, H, L = 4, 8, 3001
    xs = [torch.randn(B, H, L, 64, device="cuda").bfloat16() for _ in range(2)]
    w = torch.ones(H * 64, device="cuda")
    want = []
    for x in xs:
        n = sl.Norm(B, H, L)
        want.append([t.clone() for t in (n.forward(x, w, w), *n.backward(x, x, w, w))])
    runs = [sl.Norm(B, H, L) for _ in xs]
    streams = [torch.cuda.Stream() for _ in xs]
    torch.cuda.synchronize()
    got = [None, None]
    for _ in range(5):
        for i, (n, s, x) in enumerate(zip(runs, streams, xs)):
            got[i] = (n.forward(x, w, w, stream=s), *n.backward(x, x, w, w, stream=s))
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(a, b))


@pytest.mark.parametrize("H,d,dtype,tokens", [
    (1, 64, "bf16", 20000), (8, 64, "bf16", 20000), (16, 64, "bf16", 20000), (24, 64, "bf16", 9000),
    (32, 64, "f32", 9000), (64, 64, "bf16", 9000), (100, 64, "bf16", 3000), (8, 63, "bf16", 9000),
    (33, 31, "f32", 9000)])
def test_backward_stays_inside_its_workspace(H, d, dtype, tokens):
    """The partial sums of more tokens than the GPU holds at once: nothing
    behind the workspace that the size query asks for is written."""
    from efficient_transformer_lsh_b200 import _lib
    torch = _torch()
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, L, D = 1, tokens, H * d
    x, f, dy, dh, dx, df = (torch.randn(B, H, L, d, device="cuda").to(td) for _ in range(6))
    w = torch.ones(D, device="cuda")
    grads = [torch.empty(D, device="cuda") for _ in range(5)]
    guard = 1 << 20

    def room(n):
        buf = torch.full((n + guard,), 77, dtype=torch.uint8, device="cuda")
        return buf, n

    n = _lib.make_norm_problem(B, H, L, d, dtype, _lib.LSH_NORM_LAYER, 1e-5)
    buf, size = room(_lib.lsh_norm_bwd_workspace_size(n))
    _lib.lsh_norm_bwd(n, x, w, dh, dy, dx, grads[0], grads[1], buf, size)
    assert (buf[size:] == 77).all()
    for norm in (_lib.LSH_NORM_NONE, _lib.LSH_NORM_RMS):
        q = _lib.make_residual_problem(B, H, L, d, dtype, _lib.LSH_NORM_LAYER, norm,
                                       _lib.LSH_GATE_VECTOR, False, 1e-5, 1e-5, 1.0, 1.0, 0.1)
        buf, size = room(_lib.lsh_residual_bwd_workspace_size(q))
        dw = grads[4] if norm else None
        _lib.lsh_residual_bwd(q, dy, dh, x, f, w, w, w, w, 1, 0, None, dx, df, grads[0], grads[1],
                              grads[2], dw, None, buf, size)
        assert (buf[size:] == 77).all()
    q = _lib.make_residual_problem(3, H, L // 3, d, dtype, _lib.LSH_NORM_LAYER, _lib.LSH_NORM_RMS,
                                   _lib.LSH_GATE_VECTOR, True, 1e-5, 1e-5, 1.0, 1.0, 0.1)
    buf, size = room(_lib.lsh_residual_bwd_workspace_size(q))
    gate = torch.ones(3, D, device="cuda")
    _lib.lsh_residual_bwd(q, dy, dh, x, f, gate, w, w, w, 1, 0, None, dx, df,
                          torch.empty_like(gate), grads[1], grads[2], grads[4], None, buf, size)
    assert (buf[size:] == 77).all()


@pytest.mark.parametrize("B,H,L,d,dtype,rot,inter,yl", [
    (2, 3, 33, 64, "bf16", 64, False, "head"), (1, 8, 65, 64, "bf16", 32, True, "token"),
    (2, 1, 9, 64, "f32", 64, True, "head"), (1, 2, 17, 64, "bf16", 0, False, "head"),
    (1, 3, 5, 10, "f32", 6, False, "odd"), (1, 2, 7, 64, "f32", 20, False, "slice"),
    (1, 3, 5, 10, "bf16", 6, True, "odd"), (2, 3, 5, 14, "f32", 6, True, "odd")])
def test_rope_backward_sum(B, H, L, d, dtype, rot, inter, yl):
    from efficient_transformer_lsh_b200 import _lib
    from efficient_transformer_lsh_b200 import sublayer as sl
    torch = _torch()
    g = np.random.default_rng(L + rot)
    shape = (B, H, L, d)
    lay, strides = _layouts(yl, *shape)
    dqk, dqk64 = _f32(g.standard_normal(shape))
    dv, dv64 = _f32(g.standard_normal(shape))
    pos = torch.arange(L, dtype=torch.int32, device="cuda") * 3
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    k = 22 if dtype == "bf16" else 9        # test_rope's, and the sum's rounding
    if rot:
        r = sl.Rotary(B, H, L, rot, inter, dtype=dtype, d=d, x_layout=lay)
        got = r.backward_sum(dqk, dv, pos, 5)
        freqs, amp = sl.rope_frequencies(rot)
        turned = orc.rope(dqk64, freqs, 5 + 3 * np.arange(L), rot, inter, amp, True)
        pair = _pair_sum(np.abs(dqk64), rot, inter)
    else:
        q = _lib.make_rope_problem(B, H, L, d, dtype, 0, False, False, 1.0)
        got = torch.empty(shape, dtype=td, device="cuda")
        _lib.lsh_rope_bwd_sum(q, dqk, dv, None, None, 0, got)
        turned, pair = dqk64, np.abs(dqk64)
    _close(got, turned + dv64, dtype, pair + np.abs(dv64), k)


def _layer(post, gate, norm, rot, p, causal, seed, B=2, H=2, L=256, dff=256):
    from efficient_transformer_lsh_b200 import sublayer as sl
    torch = _torch()
    g = np.random.default_rng(seed)
    nb, nr = 16, 2
    run = sl.ReversibleLayer(B, H, L, nb, nr, 64, causal, dff, 128, norm=norm, post=post, gate=gate,
                             p=p, alpha=0.5, rot=rot)
    D, shape = 64 * H, (B, H, L, 64)
    w, w64 = {}, {}

    def par(name, a, dtype="f32"):
        w[name], w64[name] = _put(a, dtype) if dtype == "bf16" else _f32(a)

    par("W1", g.standard_normal((D, dff)) / np.sqrt(D), "bf16")
    par("W2", g.standard_normal((dff, D)) / np.sqrt(dff), "bf16")
    par("b1", 0.1 * g.standard_normal(dff))
    par("b2", 0.1 * g.standard_normal(D))
    for i in "12":
        par(f"norm{i}_w", 1 + 0.2 * g.standard_normal(D))
        if norm == "layer":
            par(f"norm{i}_b", 0.1 * g.standard_normal(D))
        if post:
            par(f"post{i}_w", 1 + 0.2 * g.standard_normal(D))
        if post == "layer":
            par(f"post{i}_b", 0.1 * g.standard_normal(D))
        if gate:
            par(f"gate{i}", 0.8 + 0.2 * g.standard_normal(D))
    acts = [_put(g.standard_normal(shape), "bf16") for _ in range(4)]
    R = _put(g.standard_normal((nr, 64, nb // 2)), "bf16")[0]
    return run, w, w64, acts, R


@pytest.mark.parametrize("post,gate,norm,rot,p,causal", [
    (None, False, "layer", 64, 0.0, True), ("layer", True, "layer", 32, 0.1, True),
    ("rms", False, "rms", 0, 0.25, False), (None, True, "rms", 64, 0.1, False)])
def test_reversible_layer_stage_by_stage(post, gate, norm, rot, p, causal):
    """Every stage of the layer against the oracle's formula of what the GPU
    gave it (attention: the path's 2e-2; products: the rounding of the hidden
    layer; the rest as above), then the whole against the oracle."""
    from efficient_transformer_lsh_b200 import _lib
    from efficient_transformer_lsh_b200 import sublayer as sl
    from oracle import lsh_oracle as lsh
    from oracle import rev_ff_oracle as ff
    torch = _torch()
    run, w, w64, acts, R = _layer(post, gate, norm, rot, p, causal, 5)
    (x1, x1_), (x2, x2_), (dy1, dy1_), (dy2, dy2_) = acts
    B, H, L, _ = run.shape
    D, seed, off = 64 * H, 99, 7
    num = lambda t: t.double().cpu().numpy()
    tok = ff.heads_to_tokens
    kind = "vector" if gate else None
    eps = 1e-5
    fac = [orc.dropout_factor(run.shape, p, seed, o) for o in (off, off + (1 << 63))]

    y1, y2 = run.forward(x1, x2, R, w, seed=seed, offset=off, pos0=3)
    assert _lib.lsh_device_status() == 0
    n, f, m, g = (num(t) for t in (run.norm1.h, run.attn.out, run.join1.h, run.g))
    y1_, y2_ = num(y1), num(y2)
    perm = run.attn.perm.cpu().numpy().astype(np.int64)
    nm = lambda x, i: orc.norm_forward(x, norm, eps, w64[f"norm{i}_w"], w64.get(f"norm{i}_b"))
    mag = lambda x, i: _norm_mag(x, norm, eps, w64[f"norm{i}_w"], w64.get(f"norm{i}_b"))
    _close(run.norm1.h, nm(x2_, 1), "bf16", mag(x2_, 1))
    freqs, amp = sl.rope_frequencies(rot) if rot else (None, 1.0)
    turn = lambda a, inv=False: a if not rot else orc.rope(a, freqs, 3 + np.arange(L), rot, False,
                                                           amp, inv)
    q = num(run.rope.y) if rot else n
    if rot:
        _close(run.rope.y, turn(n), "bf16", _pair_sum(np.abs(n), rot, False), 22)
    F, LSE = lsh.forward(q, n, perm, 64, causal, 0.125)
    assert np.abs(f - F).max() <= 2e-2

    def join(x, f, i):
        wp, bp = w64.get(f"post{i}_w"), w64.get(f"post{i}_b")
        gt = w64.get(f"gate{i}")
        y = orc.residual_forward(x, f, post, gt, kind, 0.5, 1.0, eps, wp, bp, fac[i - 1])
        um = _norm_mag(f, post, eps, wp, bp) if post else np.abs(f)
        return y, np.abs(x) + fac[i - 1] * (np.abs(orc._p(gt, f.shape)) if gate else 1.0) * um

    _close(y1, *_swap(join(x1_, f, 1)))
    _close(run.join1.h, nm(y1_, 2), "bf16", mag(y1_, 2))
    W = [w64[k] for k in ("W1", "b1", "W2", "b2")]
    hid = np.maximum(tok(m) @ W[0] + W[1], 0)
    want = ff.ff_forward(tok(m), *W)
    assert (np.abs(tok(g) - want) <= 2.0 ** -8 * (np.abs(want) + hid @ np.abs(W[2])) + 1e-3).all()
    _close(y2, *_swap(join(x2_, g, 2)))

    keep_g, keep_m, keep_f = (t.clone() for t in (run.g, run.join1.h, run.attn.out))
    rx1, rx2, dx1, dx2, grads = run.backward(y1, y2, dy1, dy2, w, seed=seed, offset=off, pos0=3)
    assert _lib.lsh_device_status() == 0
    # the recomputation saw the forward's m, mask and G, bit for bit
    assert torch.equal(run.norm2.h, keep_m) and torch.equal(run.g, keep_g)
    half = 2.0 ** -8
    assert (np.abs(num(rx2) - x2_) <= half * (np.abs(y2_) + np.abs(num(rx2))) + 1e-4).all()
    # x1 = y1 - branch(F(rebuilt x2)): F moves by what x2 moved
    f2 = num(run.attn.out)
    back, bm = join(np.zeros_like(y1_), f2, 1)
    _close(rx1, y1_ - back, "bf16", np.abs(y1_) + bm)
    rx2_ = num(rx2)
    n2, q2 = num(run.norm1.h), num(run.rope.y) if rot else num(run.norm1.h)

    def jb(dy, dh, y, f, i, nrm):
        return orc.residual_backward(dy, dh, y, f, post, nrm, w64.get(f"gate{i}"), kind, 0.5, 1.0,
                                     eps, w64.get(f"post{i}_w"), w64.get(f"post{i}_b"),
                                     w64["norm2_w"] if nrm else None, fac[i - 1])

    def near(got, want, rel):
        """2-norm of the difference over that of the result."""
        a = num(got)
        assert np.linalg.norm(a - want) <= rel * np.linalg.norm(want) + 1e-6, \
            np.linalg.norm(a - want) / np.linalg.norm(want)

    # one bf16 rounding a value: 2^-8 of it; sums in float32 nearer
    r2 = jb(dy2_, None, None, g, 2, None)
    near(run.join2.df, r2["df"], half)
    dm, dW1, db1, dW2, db2 = ff.ff_backward(tok(m), *W, tok(num(run.join2.df)))
    # the hidden layer and its gradient are rounded to bf16 (an element at the
    # kink may fall on the other side: its value is within a rounding of zero)
    near(run.dm, ff.tokens_to_heads(dm, B, H, L), 3 * half)
    for k, v in (("W1", dW1), ("b1", db1), ("W2", dW2), ("b2", db2)):
        near(grads[k], v, 2 * half)
    r1 = jb(dy1_, num(run.dm), y1_, f2, 1, norm)
    near(dx1, r1["dx"], half)
    near(run.join1.df, r1["df"], half)
    for key, name in (("dgate", "gate"), ("dw_post", "post{}_w"), ("db_post", "post{}_b")):
        for i, r in ((1, r1), (2, r2)):
            k = name.format(i) if "{" in name else f"{name}{i}"
            if k in grads:
                near(grads[k], r[key], 2e-5)
    near(grads["norm2_w"], r1["dw"], 2e-5)
    F2, LSE2 = lsh.forward(q2, n2, perm, 64, causal, 0.125)
    dqk, dv = lsh.backward(q2, n2, perm, 64, causal, 0.125, F2, LSE2, num(run.join1.df))
    assert np.abs(num(run.attn.dqk) - dqk).max() <= 2e-2
    assert np.abs(num(run.attn.dv) - dv).max() <= 2e-2
    near(run.dn, turn(num(run.attn.dqk), True) + num(run.attn.dv), half)
    ex, ew, eb = orc.norm_backward(rx2_, norm, eps, w64["norm1_w"], num(run.dn), num(run.join2.dx))
    near(dx2, ex, half)
    near(grads["norm1_w"], ew, 2e-5)
    assert set(grads) == set(w)
    # the whole, from the outputs: about thirteen roundings of 2^-8 on the way,
    # none amplified by more than 2 in these well-conditioned layers
    c = dict(norm=norm, post=post, gate=gate, alpha=0.5, eps=eps, freqs=freqs, rot=rot,
             interleaved=False, amp=amp, pos=3 + np.arange(L), chunk=64, causal=causal, scale=0.125,
             fac1=fac[0], fac2=fac[1])
    _, _, wx1, wx2, wg = orc.layer_backward(y1_, y2_, dy1_, dy2_, perm, w64, c)
    near(dx1, wx1, 0.1)
    near(dx2, wx2, 0.1)
    for k in w:
        near(grads[k], wg[k], 0.1)


def _swap(pair):
    """(value, magnitude) as _close's (want, dtype, magnitude)."""
    return pair[0], "bf16", pair[1]


def test_reversible_layer_captured_and_replayed():
    """Forward and backward in one graph; each replay sees the counter's new
    masks, and the rebuilt inputs are those of an eager layer's."""
    from efficient_transformer_lsh_b200 import _lib
    torch = _torch()
    run, w, _, acts, R = _layer("rms", True, "layer", 64, 0.2, True, 11)
    other = _layer("rms", True, "layer", 64, 0.2, True, 11)[0]
    x1, x2, dy1, dy2 = (a[0] for a in acts)
    counter = torch.zeros(1, dtype=torch.int64, device="cuda")

    def step(r):
        y1, y2 = r.forward(x1, x2, R, w, seed=3, counter=counter)
        out = r.backward(y1, y2, dy1, dy2, w, seed=3, counter=counter)
        return [y1, y2, *out[:4], *(out[4][k] for k in sorted(out[4]))]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(run)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = step(run)
    side.synchronize()
    seen = []
    for i in range(3):
        counter.fill_(i)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        want = step(other)
        torch.cuda.synchronize()
        # the weight gradients of the products are checked by norm: their K
        # splits are added in a fixed order, so they are equal too
        for a, b in zip(outs, want):
            assert torch.equal(a, b)
        seen.append(outs[0].clone())
        assert (outs[2].float() - x1.float()).abs().max() < 0.1
    assert not torch.equal(seen[0], seen[1]) and not torch.equal(seen[1], seen[2])
    assert _lib.lsh_device_status() == 0


def test_reversible_layer_refuses():
    from efficient_transformer_lsh_b200 import _lib
    run, w, _, acts, R = _layer(None, False, "layer", 64, 0.1, True, 1)
    x1, x2 = acts[0][0], acts[1][0]
    for bad in ({k: v for k, v in w.items() if k != "norm1_b"}, {**w, "gate1": w["b2"]},
                {**w, "W1": w["W1"].float()}, {**w, "norm1_w": w["b1"][:64]}):
        with pytest.raises(_lib.LshError):
            run.forward(x1, x2, R, bad)
    with pytest.raises(_lib.LshError):
        run.forward(x1, x2, R[:1], w)
    with pytest.raises(_lib.LshError):
        run.forward(x1, x2, R, w, offset=1 << 63)


def test_a_call_reads_what_the_call_before_it_wrote():
    """Launches overlap their set-up: parameters and activations that the
    previous kernel of the stream wrote are those it wrote."""
    from efficient_transformer_lsh_b200 import sublayer as sl
    torch = _torch()
    B, H, L = 1, 8, 6001
    D = 64 * H
    g = torch.Generator(device="cuda").manual_seed(1)
    rnd = lambda: torch.randn(B, H, L, 64, device="cuda", generator=g).bfloat16()
    x, dh, f = rnd(), rnd(), rnd()
    ones = torch.ones(D, device="cuda")
    a, b = sl.Norm(B, H, L), sl.Norm(B, H, L)
    r = sl.Residual(B, H, L, "rms", "layer", "vector", p=0.1)

    def chain(wait):
        out = []
        for i in range(6):
            dh.copy_(f).mul_(0.01 * (i + 1))
            wait()
            _, dw, db = a.backward(x, dh, ones, ones)          # dw, db are the next calls'
            wait()
            h = b.forward(x, dw, db)                           # parameters
            wait()
            y, h2 = r.forward(h, f, dw, db, None, dw, db, seed=i)
            wait()
            got = r.backward(h2, f, y, h, dw, db, None, dw, db, seed=i)
            out += [t.clone() for t in (h, y, h2, *(t for t in got if t is not None))]
        return out

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(chain(lambda: None), want))


def test_first_calls_of_a_process_may_be_captured():
    """No warm-up: the kernels are loaded while the graph is captured."""
    import os
    import subprocess
    import sys
    code = """
import torch
from efficient_transformer_lsh_b200 import sublayer as sl
B, H, L = 2, 5, 33
x, f = (torch.randn(B, H, L, 64, device="cuda").bfloat16() for _ in range(2))
w = torch.ones(64 * H, device="cuda")
make = lambda: (sl.Residual(B, H, L, "rms", "layer", "vector", p=0.2), sl.Rotary(B, H, L),
                sl.Dropout(B, H, L, 0.3))
def step(r, e, d):
    y, h = r.forward(x, f, w, w, None, w, w, seed=4)
    return [y, h, e.forward(h), d.forward(h, 9)] + \\
        [t for t in r.backward(f, f, y, x, w, w, None, w, w, seed=4) if t is not None]
cap, eager = make(), make()
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    outs = step(*cap)
graph.replay()
want = step(*eager)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(outs, want))
print("captured")
"""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", code], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and "captured" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("lead", [1, 2, 3, 4])
def test_pointers_at_their_elements_alignment(dtype, lead):
    """Elementwise operators give the same bits at any alignment."""
    from efficient_transformer_lsh_b200 import sublayer as sl
    torch = _torch()
    B, H, L, d = 2, 3, 7, 64
    g = np.random.default_rng(lead)
    a = g.standard_normal((B, H, L, d))
    dense = (H * L * d, L * d, d, 1)
    x, z = _put(a, dtype)[0], _put(a, dtype, dense, lead)[0]
    out = _put(0 * a, dtype, dense, lead)[0]
    for inter in (False, True):
        for rot in (64, 20):
            r = sl.Rotary(B, H, L, rot, inter, dtype=dtype)
            want = r.forward(x).clone()
            assert torch.equal(r.forward(z), want) and torch.equal(r.forward(x, out=out), want)
            dqk, dv = torch.randn(2, B, H, L, d, device="cuda")
            want = r.backward_sum(dqk, dv).clone()
            assert torch.equal(r.backward_sum(dqk, dv, out=out), want)
    q = sl.Dropout(B, H, L, 0.4, dtype)
    want = q.forward(x, 3).clone()
    assert torch.equal(q.forward(z, 3), want) and torch.equal(q.forward(x, 3, out=out), want)
