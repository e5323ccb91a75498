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


ALIAS_SHAPES = [(8, 64, 12000), (40, 64, 2600), (3, 7, 7000), (5, 64, 9001)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("H,d,L", ALIAS_SHAPES)
def test_norm_outputs_over_inputs(H, d, L, dtype):
    """Every array that an output may share gives the bits of separate ones, over
    several rounds of tokens."""
    from efficient_transformer_lsh_b200 import _lib
    torch = base._torch()
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    D, B = H * d, 1
    src = {k: torch.randn(B, H, L, d, device="cuda").to(td) for k in ("x", "dh", "dres")}
    w, b = torch.randn(2, D, device="cuda")
    n = _lib.make_norm_problem(B, H, L, d, dtype, _lib.LSH_NORM_LAYER, 1e-5)
    size = _lib.lsh_norm_bwd_workspace_size(n)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")

    def run(fwd, back):
        t = {k: v.clone() for k, v in src.items()}
        h = t[fwd] if fwd else torch.empty_like(t["x"])
        _lib.lsh_norm_fwd(n, t["x"], w, b, h)
        h = h.clone()
        t = {k: v.clone() for k, v in src.items()}
        dx = t[back] if back else torch.empty_like(t["x"])
        dw, db = torch.empty(2, D, device="cuda")
        _lib.lsh_norm_bwd(n, t["x"], w, t["dh"], t["dres"], dx, dw, db, ws, size)
        return h, dx, dw, db

    want = run(None, None)
    for fwd, back in (("x", "x"), (None, "dh"), (None, "dres")):
        assert all(torch.equal(p, q) for p, q in zip(run(fwd, back), want)), (fwd, back)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("gate", [None, "vector", "sigmoid"])
@pytest.mark.parametrize("H,d,L", ALIAS_SHAPES)
def test_residual_outputs_over_inputs(H, d, L, gate, dtype):
    from efficient_transformer_lsh_b200 import _lib
    torch = base._torch()
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    D, B, sig = H * d, 1, gate == "sigmoid"
    names = ["x", "f", "y", "dy", "dh"] + (["z"] if sig else [])
    src = {k: torch.randn(B, H, L, d, device="cuda").to(td) for k in names}
    w_post, b_post, w, b, vec = torch.randn(5, D, device="cuda")
    kind = {None: _lib.LSH_GATE_NONE, "vector": _lib.LSH_GATE_VECTOR,
            "sigmoid": _lib.LSH_GATE_SIGMOID}[gate]
    post = _lib.LSH_NORM_LAYER if gate else _lib.LSH_NORM_NONE
    q = _lib.make_residual_problem(B, H, L, d, dtype, post, _lib.LSH_NORM_LAYER, kind, False, 1e-5,
                                   1e-5, 0.5, 1.5, 0.1)
    size = _lib.lsh_residual_bwd_workspace_size(q)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    wp, bp = (w_post, b_post) if gate else (None, None)

    def arrays(shared):
        """Copies of the inputs, and each output's array: an input's or its own."""
        t = {k: v.clone() for k, v in src.items()}
        return t, lambda o: t[shared[o]] if o in shared else torch.empty_like(t["x"])

    def forward(**shared):
        t, out = arrays(shared)
        y, h = out("y"), out("h")
        g = t["z"] if sig else vec if gate else None
        _lib.lsh_residual_fwd(q, t["x"], t["f"], g, wp, bp, w, b, 7, 0, None, y, h)
        return y, h

    def backward(**shared):
        t, out = arrays(shared)
        dx, df, dz = out("dx"), out("df"), out("dz") if sig else None
        g, dg = (t["z"], dz) if sig else (vec, torch.empty_like(vec)) if gate else (None, None)
        grads = [torch.empty_like(w) if k else None for k in (gate, gate, True, True)]
        _lib.lsh_residual_bwd(q, t["dy"], t["dh"], t["y"], t["f"], g, wp, bp, w, 7, 0, None, dx, df,
                              dg, *grads, ws, size)
        return [v for v in (dx, df, dg, *grads) if v is not None]

    branch = ["f"] + (["z"] if sig else [])
    want = [v.clone() for v in forward()]
    for shared in [dict([(o, i)]) for o in ("y", "h") for i in ["x"] + branch] + \
            [dict(y="x", h="f"), dict(y="f", h="x")]:
        assert all(torch.equal(p, r) for p, r in zip(forward(**shared), want)), shared
    want = [v.clone() for v in backward()]
    every = ["y", "dy", "dh"]
    cases = [dict(dx=i) for i in every] + [dict(df=i) for i in every + branch]
    cases += [dict(dx="dy", df="f"), dict(dx="dh", df="dy"), dict(dx="y", df="dh")]
    if sig:
        cases += [dict(dz=i) for i in every + branch]
        cases += [dict(dx="dy", df="f", dz="z"), dict(dx="dh", df="z", dz="f")]
    for shared in cases:
        assert all(torch.equal(p, r) for p, r in zip(backward(**shared), want)), shared


@pytest.mark.parametrize("H,d,dtype", [(3, 64, "bf16"), (40, 64, "bf16"), (3, 64, "f32"),
                                       (3, 10, "f32"), (2, 512, "f32")])
def test_elementwise_outputs_over_inputs(H, d, dtype):
    from efficient_transformer_lsh_b200 import _lib
    torch = base._torch()
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    B, L = 2, 901
    x = torch.randn(B, H, L, d, device="cuda").to(td)
    q = _lib.make_dropout_problem(B, H, L, d, dtype, 0.3)
    want, same = torch.empty_like(x), x.clone()
    _lib.lsh_dropout_fwd(q, x, 3, 0, None, want)
    _lib.lsh_dropout_fwd(q, same, 3, 0, None, same)
    assert torch.equal(same, want)
    turns = torch.randint(-(1 << 62), 1 << 62, (d // 2,), device="cuda")
    for inter in (False, True):
        p = _lib.make_rope_problem(B, H, L, d, dtype, d - d // 4 * 2, inter, False, 1.0)
        for fn in (_lib.lsh_rope_fwd, _lib.lsh_rope_bwd):
            same = x.clone()
            fn(p, x, turns, None, 9, want)
            fn(p, same, turns, None, 9, same)
            assert torch.equal(same, want)
        if dtype == "f32":
            dv = torch.randn_like(x)
            _lib.lsh_rope_bwd_sum(p, x, dv, turns, None, 9, want)
            for over in (0, 1):
                t = [x.clone(), dv.clone()]
                _lib.lsh_rope_bwd_sum(p, *t, turns, None, 9, t[over])
                assert torch.equal(t[over], want)


@pytest.mark.parametrize("H,d,dtype", [(3, 64, "bf16"), (2, 64, "f32"), (3, 7, "bf16")])
def test_residual_of_a_later_slice(H, d, dtype):
    """slice0: the mask of the rows that the shard holds of the whole problem."""
    from efficient_transformer_lsh_b200 import sublayer as sl
    torch = base._torch()
    B, L, slice0, seed = 2, 33, 1001, 17
    shape = (B, H, L, d)
    g = np.random.default_rng(d)
    (x, x_), (f, f_), (dy, dy_) = (base._put(g.standard_normal(shape), dtype) for _ in range(3))
    r = sl.Residual(B, H, L, p=0.3, dtype=dtype, d=d, slice0=slice0)
    fac = orc.dropout_factor(shape, 0.3, seed, 5, slice0=slice0)
    y, _ = r.forward(x, f, seed=seed, offset=5)
    mag = np.abs(x_) + fac * np.abs(f_)
    base._close(y, x_ + fac * f_, dtype, mag, 4)       # scale, product, sum
    base._close(r.backward(dy, f, seed=seed, offset=5)[1], fac * dy_, dtype, fac * np.abs(dy_), 4)
    # the mask is that of the dropout alone, and of the whole problem's rows
    keep = sl.Dropout(B, H, L, 0.3, dtype, d, slice0=slice0).forward(torch.ones_like(x), seed, 5) != 0
    assert torch.equal(keep, torch.from_numpy(fac > 0).cuda())
    n = -(-(slice0 + B * H) // H)
    whole = orc.dropout_factor((n, H, L, d), 0.3, seed, 5).reshape(n * H, L, d)
    assert np.array_equal(whole[slice0:slice0 + B * H].reshape(shape), fac)


@pytest.mark.parametrize("H,d,dtype", [(8, 64, "bf16"), (40, 64, "f32"), (3, 7, "f32")])
def test_two_epsilons_and_no_dx(H, d, dtype):
    """eps_post is f's, eps is y's; dx may be NULL, and changes nothing else."""
    from efficient_transformer_lsh_b200 import _lib
    torch = base._torch()
    B, L, D = 2, 19, H * d
    shape, ep, en = (B, H, L, d), 0.5, 2.0
    g = np.random.default_rng(H)
    (x, x_), (f, f_), (y, y_), (dy, dy_), (dh, dh_) = (base._put(g.standard_normal(shape), dtype)
                                                       for _ in range(5))
    q = _lib.make_residual_problem(B, H, L, d, dtype, _lib.LSH_NORM_LAYER, _lib.LSH_NORM_RMS,
                                   _lib.LSH_GATE_NONE, False, ep, en, 1.0, 1.0, 0.0)
    out, h = torch.empty_like(x), torch.empty_like(x)
    _lib.lsh_residual_fwd(q, x, f, None, None, None, None, None, 0, 0, None, out, h)
    fm = base._norm_mag(f_, "layer", ep, None, None)
    base._close(out, x_ + orc.norm_forward(f_, "layer", ep), dtype, np.abs(x_) + fm)
    o = out.double().cpu().numpy()
    base._close(h, orc.norm_forward(o, "rms", en), dtype, base._norm_mag(o, "rms", en, None, None))
    size = _lib.lsh_residual_bwd_workspace_size(q)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    got = []
    for dx in (torch.empty_like(x), None):
        df = torch.empty_like(x)
        grads = [torch.empty(D, device="cuda") for _ in range(4)]
        _lib.lsh_residual_bwd(q, dy, dh, y, f, None, None, None, None, 0, 0, None, dx, df, None,
                              *grads, ws, size)
        got.append([df, *grads])
        if dx is not None:
            t, dw, db = orc.norm_backward(y_, "rms", en, None, dh_, dy_)
            m, ym = base._norm_back_mag(y_, "rms", en, None, dh_)
            tm = m + np.abs(dy_)
            base._close(dx, t, dtype, tm)
            want, wp, bp = orc.norm_backward(f_, "layer", ep, None, t)
            m, fm = base._norm_back_mag(f_, "layer", ep, None, tm)
            n = 2 * base.K
            base._close(df, want, dtype, m, n)
            flat = lambda a: a.sum((0, 2)).reshape(D)
            for a, b, c in zip(grads, (wp, bp, dw, db), (flat(tm * fm), flat(tm),
                                                         flat(np.abs(dh_) * ym), flat(np.abs(dh_)))):
                base._close(a, b, "f32", c, B * L + n)
    assert all(torch.equal(a, b) for a, b in zip(*got))


def test_rotary_with_given_frequencies_and_multiplier():
    from efficient_transformer_lsh_b200 import sublayer as sl
    B, H, L, d, rot = 2, 3, 40, 64, 24
    g = np.random.default_rng(8)
    shape = (B, H, L, d)
    (x, x_), (dy, dy_) = (base._put(g.standard_normal(shape), "f32") for _ in range(2))
    freqs = list(g.uniform(-3.0, 3.0, rot // 2))
    r = sl.Rotary(B, H, L, rot, True, frequencies=freqs, amp=1.75, dtype="f32")
    pos = 5 + np.arange(L)
    mag = lambda a: 1.75 * base._pair_sum(np.abs(a), rot, True)
    base._close(r.forward(x, pos0=5), orc.rope(x_, freqs, pos, rot, True, 1.75), "f32", mag(x_), 9)
    base._close(r.backward(dy, pos0=5), orc.rope(dy_, freqs, pos, rot, True, 1.75, True), "f32",
                mag(dy_), 9)
    # without a multiplier it is 1, whatever a scaling's would be
    one = sl.Rotary(B, H, L, rot, True, frequencies=freqs, dtype="f32")
    assert one.amp == 1.0
    base._close(one.forward(x), orc.rope(x_, freqs, np.arange(L), rot, True), "f32", mag(x_), 9)


def test_reversible_layer_of_more_heads_with_scaled_adjacent_pairs():
    """The whole layer against the oracle at 4 heads, 1024 tokens, half of each
    head turned in adjacent pairs with a scaled table; tolerances as in the
    stage by stage test (its last lines)."""
    from efficient_transformer_lsh_b200 import _lib
    from efficient_transformer_lsh_b200 import sublayer as sl
    B, H, L, dff, rot, scaling = 1, 4, 1024, 512, 32, ("yarn", 4.0, 256)
    post, gate, norm, p, seed = "rms", True, "layer", 0.1, 21
    _, w, w64, acts, R = base._layer(post, gate, norm, rot, p, True, 9, B, H, L, dff)
    run = sl.ReversibleLayer(B, H, L, 16, 2, 64, True, dff, 256, norm=norm, post=post, gate=gate,
                             p=p, alpha=0.5, rot=rot, interleaved=True, scaling=scaling)
    (x1, x1_), (x2, x2_), (dy1, dy1_), (dy2, dy2_) = acts
    y1, y2 = run.forward(x1, x2, R, w, seed=seed, pos0=100)
    num = lambda t: t.double().cpu().numpy()
    y1_, y2_ = num(y1), num(y2)
    rx1, rx2, dx1, dx2, grads = run.backward(y1, y2, dy1, dy2, w, seed=seed, pos0=100)
    assert _lib.lsh_device_status() == 0
    freqs, amp = sl.rope_frequencies(rot, scaling=scaling)
    fac = [orc.dropout_factor(run.shape, p, seed, o) for o in (0, 1 << 63)]
    c = dict(norm=norm, post=post, gate=gate, alpha=0.5, eps=1e-5, freqs=freqs, rot=rot,
             interleaved=True, amp=amp, pos=100 + np.arange(L), chunk=64, causal=True, scale=0.125,
             fac1=fac[0], fac2=fac[1])
    perm = run.attn.perm.cpu().numpy().astype(np.int64)
    wx1, wx2, wdx1, wdx2, wg = orc.layer_backward(y1_, y2_, dy1_, dy2_, perm, w64, c)
    for got, want in ((rx1, x1_), (rx2, x2_), (rx1, wx1), (rx2, wx2), (dx1, wdx1), (dx2, wdx2),
                      *((grads[k], wg[k]) for k in w)):
        a = num(got)
        assert np.linalg.norm(a - want) <= 0.1 * np.linalg.norm(want)
