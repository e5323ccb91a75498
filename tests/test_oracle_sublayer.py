"""Pins of the sublayer oracle (CPU): published Philox vectors, differences of
the formulas, closed forms of the rotation; and the frequency tables of the
product's host code."""
import math

import numpy as np
import pytest

from oracle import sublayer_oracle as orc


@pytest.mark.parametrize("ctr,seed,want", [
    # the known-answer vectors published with the generator
    ((0, 0), 0, "6627e8d5 e169c58d bc57ac4c 9b00dbd8"),
    ((2**64 - 1, 2**64 - 1), 2**64 - 1, "408f276d 41c83b0e a20bc7c6 6d5451fd"),
    ((0x85a308d3243f6a88, 0x0370734413198a2e), 0x299f31d0a4093822,
     "d16cfe09 94fdcceb 5001e420 24126ea1"),
])
def test_philox_known_answers(ctr, seed, want):
    w = orc.philox4x32(np.array([ctr[0]], dtype=np.uint64), seed, ctr[1])[0]
    assert " ".join("%08x" % int(v) for v in w) == want


def test_dropout_factor_rate_and_extremes():
    f = orc.dropout_factor((2, 3, 500, 64), 0.3, 5, 7)
    t = round(float(np.float32(0.3)) * 65536)
    p, n = t / 65536, f.size
    # a binomial share: five standard deviations
    assert abs((f == 0).mean() - p) < 5 * math.sqrt(p * (1 - p) / n)
    assert np.allclose(f[f != 0], 65536 / (65536 - t))
    assert (orc.dropout_factor((1, 1, 9, 5), 0.0, 1) == 1).all()
    assert (orc.dropout_factor((1, 1, 9, 5), 1.0, 1) == 0).all()
    # a shard sees the whole problem's elements
    whole = orc.dropout_factor((2, 4, 6, 20), 0.5, 11, 3)
    assert np.array_equal(orc.dropout_factor((1, 4, 6, 20), 0.5, 11, 3, slice0=4), whole[1:])


def _differences(fn, x, dy, at, step=1e-5):
    out = []
    for i in at:
        a, b = x.copy(), x.copy()
        a.flat[i] += step
        b.flat[i] -= step
        out.append(((fn(a) - fn(b)) * dy).sum() / (2 * step))
    return np.array(out)


@pytest.mark.parametrize("kind", ["layer", "rms"])
def test_norm_backward_against_differences(kind):
    g = np.random.default_rng(1)
    x, dh = g.standard_normal((2, 2, 3, 6)) + 0.5, g.standard_normal((2, 2, 3, 6))
    w, b = g.standard_normal(12), g.standard_normal(12)
    dx, dw, db = orc.norm_backward(x, kind, 1e-3, w, dh)
    at = range(0, x.size, 5)
    d = _differences(lambda v: orc.norm_forward(v, kind, 1e-3, w, b), x, dh, at)
    assert np.abs(d - dx.flat[list(at)]).max() < 1e-7
    d = _differences(lambda v: orc.norm_forward(x, kind, 1e-3, v, b), w, dh, range(12))
    assert np.abs(d - dw).max() < 1e-7
    d = _differences(lambda v: orc.norm_forward(x, kind, 1e-3, w, v), b, dh, range(12))
    assert np.abs(d - db).max() < 1e-7


@pytest.mark.parametrize("kind", [None, "vector", "sigmoid"])
@pytest.mark.parametrize("post,norm", [(None, None), ("layer", "rms"), ("rms", "layer")])
def test_residual_backward_against_differences(kind, post, norm):
    g = np.random.default_rng(2)
    shape, D = (2, 2, 3, 4), 8
    x, f, dy, dh = (g.standard_normal(shape) for _ in range(4))
    gate = {None: None, "vector": g.standard_normal((2, D)),
            "sigmoid": g.standard_normal(shape)}[kind]
    wp, bp, w = g.standard_normal(D), g.standard_normal(D), g.standard_normal(D)
    fac = orc.dropout_factor(shape, 0.4, 9)
    if not post:
        wp = bp = None

    def both(x, f, gate, wp, bp, w):
        y = orc.residual_forward(x, f, post, gate, kind, 0.7, 1.3, 1e-3, wp, bp, fac)
        return np.stack([y, orc.norm_forward(y, norm, 1e-3, w) if norm else 0 * y])

    y = both(x, f, gate, wp, bp, w)[0]
    got = orc.residual_backward(dy, dh, y, f, post, norm, gate, kind, 0.7, 1.3, 1e-3, wp, bp, w,
                                fac, gate_batch=True)
    args = dict(x=x, f=f, gate=gate, wp=wp, bp=bp, w=w)
    pairs = [("x", "dx"), ("f", "df")] + [("gate", "dgate")] * (kind is not None) + \
        [("wp", "dw_post"), ("bp", "db_post")] * (post is not None) + [("w", "dw")] * (norm is not None)
    for name, grad in pairs:
        v = args[name]
        at = list(range(0, v.size, max(1, v.size // 9)))
        d = _differences(lambda u: both(**{**args, name: u}), v, np.stack([dy, dh]), at)
        assert np.abs(d - got[grad].flat[at]).max() < 1e-7, (name, grad)


@pytest.mark.parametrize("inter", [False, True])
def test_rope_turns_pairs_and_keeps_relative_positions(inter):
    g = np.random.default_rng(3)
    freqs = [1.0, 0.1, 0.01]
    x = g.standard_normal((1, 2, 5, 8))
    pos = np.array([0, 1, 7, -3, 1000])
    y = orc.rope(x, freqs, pos, 6, inter)
    assert np.array_equal(y[:, :, 0], x[:, :, 0])             # position 0: no turn
    assert np.array_equal(y[..., 6:], x[..., 6:])             # part of the head only
    assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
    assert np.allclose(orc.rope(y, freqs, pos, 6, inter, inverse=True), x)
    # products depend on the distance alone
    k = g.standard_normal((1, 1, 1, 8))
    q = g.standard_normal((1, 1, 1, 8))
    dots = [(orc.rope(q, freqs, [m], 6, inter) * orc.rope(k, freqs, [m - 4], 6, inter)).sum()
            for m in (0, 9, 4096)]
    assert np.ptp(dots) < 1e-9
    # one pair by hand: a quarter turn takes (p, q) to (-q, p)
    z = orc.rope(np.array([[[[3.0, 5.0]]]]), [np.pi / 2], [1], 2, inter)
    assert np.allclose(z, [[[[-5.0, 3.0]]]])


def test_frequency_tables():
    from efficient_transformer_lsh_b200.sublayer import rope_frequencies, rope_turns
    f, amp = rope_frequencies(64)
    assert f[0] == 1.0 and amp == 1.0 and abs(f[16] - 0.01) < 1e-15
    lin, _ = rope_frequencies(64, scaling=("linear", 8.0))
    assert np.allclose(np.array(lin) * 8, f)
    ntk, _ = rope_frequencies(64, scaling=("ntk", 8.0))
    assert ntk[0] == 1.0 and abs(ntk[-1] * 8 / f[-1] - 1) < 1e-12
    yarn, amp = rope_frequencies(64, scaling=("yarn", 8.0, 4096))
    assert yarn[0] == 1.0 and abs(yarn[-1] * 8 / f[-1] - 1) < 1e-12
    assert abs(amp - (0.1 * math.log(8) + 1)) < 1e-15
    assert all(a <= b * (1 + 1e-12) and a >= b / 8 * (1 - 1e-12) for a, b in zip(yarn, f))
    # position * turns modulo 2^64 is the phase, at any distance and sign
    turns = [int(v) % (1 << 64) for v in rope_turns(f)]
    for pos in (1, 1 << 20, (1 << 31) - 1, -5):
        for t, v in zip(turns, f):
            got = (pos * t) % (1 << 64) / 2.0 ** 64
            # 53 bits of f and of 2 pi: three roundings of 2^-53 each, and 2^-64 a position
            err = (got - pos * v / (2 * math.pi) + 0.5) % 1.0 - 0.5
            assert abs(err) < abs(pos) * (v * 4 * 2.0 ** -53 + 2.0 ** -63) + 2.0 ** -52


@pytest.mark.parametrize("post,gate,rot", [(None, False, 0), ("rms", True, 8), ("layer", True, 64)])
def test_reversible_layer_inverts_and_differentiates(post, gate, rot):
    """The layer's backward rebuilds its inputs, and its gradients are the
    differences of its forward (the permutation held fixed)."""
    from oracle import lsh_oracle as lsh
    g = np.random.default_rng(7)
    B, H, L, D, dff = 1, 2, 8, 128, 12
    shape = (B, H, L, 64)
    x1, x2, dy1, dy2 = (g.standard_normal(shape) for _ in range(4))
    w = dict(W1=g.standard_normal((D, dff)) / 11, b1=0.1 * g.standard_normal(dff),
             W2=g.standard_normal((dff, D)) / 4, b2=0.1 * g.standard_normal(D))
    for i in (1, 2):
        w[f"norm{i}_w"], w[f"norm{i}_b"] = 1 + 0.2 * g.standard_normal(D), g.standard_normal(D)
        if post:
            w[f"post{i}_w"] = 1 + 0.2 * g.standard_normal(D)
        if post == "layer":
            w[f"post{i}_b"] = g.standard_normal(D)
        if gate:
            w[f"gate{i}"] = 0.7 + 0.2 * g.standard_normal(D)
    c = dict(norm="layer", post=post, gate=gate, alpha=0.7, eps=1e-4, rot=rot, interleaved=True,
             amp=1.1, pos=np.arange(L) + 3, chunk=4, causal=True, scale=0.125,
             freqs=[10.0 ** (-i / 8) for i in range(rot // 2)] if rot else None,
             fac1=orc.dropout_factor(shape, 0.2, 5, 1), fac2=orc.dropout_factor(shape, 0.2, 5, 2))
    perm = np.stack([[g.permutation(L) for _ in range(2)] for _ in range(B * H)]).reshape(B, H, 2, L)
    y1, y2 = orc.layer_forward(x1, x2, perm, w, c)
    rx1, rx2, dx1, dx2, grads = orc.layer_backward(y1, y2, dy1, dy2, perm, w, c)
    assert np.abs(rx1 - x1).max() < 1e-11 and np.abs(rx2 - x2).max() < 1e-11

    def value(x1, x2, w):
        a, b = orc.layer_forward(x1, x2, perm, w, c)
        return (a * dy1).sum() + (b * dy2).sum()

    def diff(fn, a, i, step=1e-5):
        p, q = a.copy(), a.copy()
        p.flat[i] += step
        q.flat[i] -= step
        return (fn(p) - fn(q)) / (2 * step)

    for i in range(3, x1.size, 131):
        assert abs(diff(lambda a: value(a, x2, w), x1, i) - dx1.flat[i]) < 1e-6
        assert abs(diff(lambda a: value(x1, a, w), x2, i) - dx2.flat[i]) < 1e-6
    for k in w:
        for i in range(1, w[k].size, max(2, w[k].size // 3)):
            d = diff(lambda a: value(x1, x2, {**w, k: a}), w[k], i)
            assert abs(d - grads[k].flat[i]) < 1e-6 * max(1.0, abs(d)), k
