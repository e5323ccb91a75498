"""Further calls of the operators around a sublayer: what a refused call leaves
alone, far positions, both ways of a stride's reach, arrays that are input and
output at once. Tolerances as in test_gpu_sublayer, with fewer roundings where
fewer are made."""
import numpy as np
import pytest

import test_gpu_sublayer as base
from oracle import sublayer_oracle as orc

pytestmark = pytest.mark.gpu
U = base.U


def test_a_refused_call_of_the_layer_launches_nothing():
    """A refusal halfway would have replaced the permutation that the backward
    of the forward before it needs."""
    from efficient_transformer_lsh_b200 import _lib
    torch = base._torch()
    run, w, _, acts, R = base._layer("rms", True, "layer", 64, 0.1, True, 1)
    x1, x2, dy1, dy2 = (a[0] for a in acts)
    y1, y2 = (t.clone() for t in run.forward(x1, x2, R, w, seed=3))
    torch.cuda.synchronize()
    perm = run.attn.perm.clone()
    short = torch.ones(64, device="cuda")
    wrong = [{**w, k: short} for k in ("norm1_w", "norm1_b", "norm2_w", "norm2_b", "post1_w",
                                       "post2_w", "gate1", "gate2", "b2")]
    wrong.append({**w, "norm2_w": w["norm2_w"].bfloat16()})
    wrong += [{**w, k: None} for k in ("W1", "b1", "W2", "b2", "gate1", "gate2")]
    for k in ("W1", "b1", "W2", "b2"):     # the products read 16 bytes at once
        room = torch.zeros(w[k].numel() + 1, dtype=w[k].dtype, device="cuda")
        wrong.append({**w, k: room[1:].view(w[k].shape)})
    int32 = torch.zeros(1, dtype=torch.int32, device="cuda")
    calls = [lambda p=p: run.forward(x2, x1, R, p, seed=3) for p in wrong]
    calls += [lambda p=p: run.backward(y1, y2, dy1, dy2, p, seed=3) for p in wrong]
    for kw in (dict(seed=-1), dict(seed=1 << 64), dict(counter=int32), dict(offset=-1),
               dict(counter=torch.zeros(1, dtype=torch.int64))):
        calls.append(lambda kw=kw: run.forward(x2, x1, R, w, **kw))
        calls.append(lambda kw=kw: run.backward(y1, y2, dy1, dy2, w, **kw))
    for i in range(4):
        t = [y1, y2, dy1, dy2]
        t[i] = t[i].float()
        calls.append(lambda t=t: run.backward(*t, w, seed=3))
    calls += [lambda: run.forward(x2.float(), x1, R, w), lambda: run.forward(x2, x1[:1], R, w),
              lambda: run.forward(x2, x1, R.float(), w), lambda: run.forward(x2, x1, None, w)]
    before = _lib.lsh_launch_count()
    for i, call in enumerate(calls):
        with pytest.raises(_lib.LshError):
            call()
        assert _lib.lsh_launch_count() == before, i
    torch.cuda.synchronize()
    assert torch.equal(run.attn.perm, perm)


@pytest.mark.parametrize("dtype,inter,scale", [("f32", False, 1), ("f32", True, 4),
                                               ("bf16", False, 1)])
def test_rope_at_far_positions(dtype, inter, scale):
    """Phases from integers: position * frequency / 2 pi modulo 1, of which the
    table holds 64 bits, so that it adds |position| 2^-65 turns: at 2^40 2 pi
    2^-25 of angle, below 4 roundings, to the 8 and 21 of test_rope."""
    from efficient_transformer_lsh_b200 import sublayer as sl
    from test_sublayer_drivers import exact_turns
    torch = base._torch()
    B, H, L, d = 1, 2, 5, 64
    shape, pos0 = (B, H, L, d), (1 << 40) - 3
    g = np.random.default_rng(scale)
    x, x64 = base._put(g.standard_normal(shape), dtype)
    r = sl.Rotary(B, H, L, interleaved=inter, dtype=dtype,
                  scaling=("linear", scale) if scale > 1 else None)
    y = r.forward(x, pos0=pos0)
    turns = [t / scale for t in exact_turns()]
    k = 25 if dtype == "bf16" else 12
    for l in range(L):
        angle = np.array([float((pos0 + l) * t % 1) * 2 * np.pi for t in turns])
        row = x64[:, :, l:l + 1]
        want = orc.rope(row, angle, [1], d, inter)
        base._close(y[:, :, l:l + 1], want, dtype, base._pair_sum(np.abs(row), d, inter), k)
    back = r.backward(y, pos0=pos0).double().cpu().numpy()
    assert np.abs(back - x64).max() < 2.0 ** -5
    assert torch.isfinite(y).all()


def test_sigmoid_gate_over_its_range_in_float32():
    """Relative to the value at every z. Exponential 2 units (4 roundings of
    2^-24), 1 + e half a unit, the quotient 2 units: gate at most 4 + (1 + 2 +
    4) + 1 = 12 roundings (the exponential's error enters 1 + e by at most
    half), slope 4 + 2 * 7 + 2 = 20; and two or three products."""
    from efficient_transformer_lsh_b200 import sublayer as sl
    B, H, L, d = 1, 2, 80, 64
    shape = (B, H, L, d)
    g = np.random.default_rng(4)
    num = lambda: base._put(g.uniform(0.5, 2.0, shape) * g.choice([-1.0, 1.0], shape), "f32")
    f, f64 = num()
    dy, dy64 = num()
    z, z64 = base._put(np.linspace(-80.0, 80.0, f64.size).reshape(shape), "f32")
    x, _ = base._put(np.zeros(shape), "f32")
    r = sl.Residual(B, H, L, gate="sigmoid", dtype="f32")
    y, _ = r.forward(x, f, z)
    s, t = (1 / (1 + np.exp(-v)) for v in (z64, -z64))
    base._close(y, s * f64, "f32", np.abs(s * f64), 13)
    _, df, dz = r.backward(dy, f, gate=z)[:3]
    base._close(df, s * dy64, "f32", np.abs(s * dy64), 13)
    want = dy64 * f64 * s * t
    base._close(dz, want, "f32", np.abs(want), 23)


def test_head_strides_within_reach_of_the_wide_kernels():
    """Rows whose heads lie 2^31 elements apart, but 2^29 vectors of 16 bytes,
    give bit for bit what near ones give: the same kernel runs."""
    from efficient_transformer_lsh_b200 import _lib
    torch = base._torch()
    B, H, L, d = 1, 2, 300, 64
    far = (1 << 31) + 64                          # 8.6 GB in float32
    buf = torch.empty(far + L * d, dtype=torch.float32, device="cuda")
    big = buf.as_strided((B, H, L, d), (far, far, d, 1))
    x, f = torch.randn(2, B, H, L, d, device="cuda")
    w, b = torch.randn(2, H * d, device="cuda")
    big.copy_(x)
    near, got, h1, h2 = (torch.empty_like(x) for _ in range(4))
    strides = (far, far, d)
    _lib.lsh_norm_fwd(_lib.make_norm_problem(B, H, L, d, "f32", 1, 1e-5), x, w, b, near)
    _lib.lsh_norm_fwd(_lib.make_norm_problem(B, H, L, d, "f32", 1, 1e-5, x=strides), big, w, b, got)
    assert torch.equal(near, got)
    res = [B, H, L, d, "f32", 1, 0, 0, False, 1e-5, 1e-5, 0.5, 1.0, 0.1, 0]
    _lib.lsh_residual_fwd(_lib.make_residual_problem(*res), f, x, None, w, b, None, None, 5, 0,
                          None, h1, None)
    _lib.lsh_residual_fwd(_lib.make_residual_problem(*res, f=strides), f, big, None, w, b, None,
                          None, 5, 0, None, h2, None)
    assert torch.equal(h1, h2)


def test_head_strides_past_reach_of_the_wide_kernels():
    """2^31 vectors of 16 bytes between two heads: the element-wise kernel,
    with 64-bit offsets."""
    from efficient_transformer_lsh_b200 import _lib
    torch = base._torch()
    B, H, L, d = 1, 2, 3, 64
    far = (1 << 33) + 64                          # 34 GB
    buf = torch.empty(far + L * d, dtype=torch.float32, device="cuda")
    big = buf.as_strided((B, H, L, d), (far, far, d, 1))
    x, x64 = base._put(np.random.default_rng(1).standard_normal((B, H, L, d)), "f32")
    h = torch.empty_like(x)
    n = _lib.make_norm_problem(B, H, L, d, "f32", 1, 1e-5, x=(far, far, d), h=(far, far, d))
    big.copy_(x)
    _lib.lsh_norm_fwd(n, big, None, None, big)    # in place
    want = orc.norm_forward(x64, "layer", 1e-5)
    base._close(big, want, "f32", base._norm_mag(x64, "layer", 1e-5, None, None))
    n = _lib.make_norm_problem(B, H, L, d, "f32", 1, 1e-5, x=(far, far, d))
    big.copy_(x)
    _lib.lsh_norm_fwd(n, big, None, None, h)
    base._close(h, want, "f32", base._norm_mag(x64, "layer", 1e-5, None, None))


def test_rows_too_wide_for_the_wide_backward():
    """float32, 8192 features, a sigmoid gate, both norms and b_post: a stage of
    the ring and the parameters leave the wide kernel no room."""
    base.test_residual((1, 128, 40, 64, "f32", "layer", "layer", "sigmoid", False, 0.1, 1.0, 1.0,
                        "head", "head", 0))
    base.test_residual((1, 112, 40, 64, "f32", "layer", "layer", "sigmoid", False, 0.1, 1.0, 1.0,
                        "head", "head", 0))
