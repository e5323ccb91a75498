"""Refusals of the sublayer operators that need no GPU: arguments are checked
on the host before any launch."""
import ctypes

import pytest

from efficient_transformer_lsh_b200 import _lib

FAKE = 1 << 20   # non-null, aligned; never dereferenced on the host
BIG = 1 << 40


@pytest.fixture(scope="module")
def L():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from efficient_transformer_lsh_b200 import build
        build.build()
    return _lib.lib()


def _norm(**kw):
    a = dict(B=1, H=2, L=5, d=64, dtype="bf16", kind=1, eps=1e-5, x=(0, 0, 0), h=(0, 0, 0))
    a.update(kw)
    return _lib.make_norm_problem(**a)


def _res(**kw):
    a = dict(B=1, H=2, L=5, d=64, dtype="bf16", post=1, norm=2, gate=1, gate_batch=0, eps_post=1e-5,
             eps=1e-5, alpha=1.0, beta=1.0, p=0.1, slice0=0, x=(0, 0, 0), f=(0, 0, 0))
    a.update(kw)
    q = _lib.make_residual_problem(**{**a, "gate_batch": 0})
    q.gate_batch = a["gate_batch"]
    return q


def _drop(**kw):
    a = dict(B=1, H=2, L=5, d=64, dtype="bf16", p=0.1, slice0=0, x=(0, 0, 0), y=(0, 0, 0))
    a.update(kw)
    return _lib.make_dropout_problem(**a)


def _rope(**kw):
    a = dict(B=1, H=2, L=5, d=64, dtype="bf16", rot=64, interleaved=0, pos_batch=0, amp=1.0,
             x=(0, 0, 0), y=(0, 0, 0))
    a.update(kw)
    return _lib.make_rope_problem(**a)


SIZES = [(dict(B=-1), 1), (dict(H=-1), 1), (dict(L=-2), 1), (dict(d=0), 1), (dict(dtype=7), 1),
         (dict(B=1 << 16, L=1 << 15), 2), (dict(d=(1 << 16) + 2), 2)]
STRIDES = [((0, 0, 63), 1), ((640, 320, 0), 1), ((640, 64, 64), 1), ((640, 320, -64), 1),
           ((1, 2, 3), 1), ((0, 1 << 50, 64), 1)]


@pytest.mark.parametrize("kw,code", SIZES + [(dict(kind=0), 1), (dict(kind=3), 1), (dict(eps=0.0), 1),
                                             (dict(eps=float("nan")), 1), (dict(eps=-1.0), 1),
                                             (dict(H=129), 2)])
def test_norm_refuses(L, kw, code):
    n = _norm(**kw)
    assert L.lsh_norm_fwd(n, FAKE, FAKE, FAKE, FAKE, None) == code
    assert L.lsh_norm_bwd_workspace_size(n) == 0
    assert L.lsh_norm_bwd(n, FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE, FAKE, BIG, None) == code


@pytest.mark.parametrize("s,code", STRIDES)
def test_overlapping_strides_are_refused(L, s, code):
    assert L.lsh_norm_fwd(_norm(x=s), FAKE, None, None, FAKE, None) == code
    assert L.lsh_norm_fwd(_norm(h=s), FAKE, None, None, FAKE, None) == code
    assert L.lsh_dropout_fwd(_drop(y=s), FAKE, 1, 0, None, FAKE, None) == code
    assert L.lsh_rope_fwd(_rope(x=s), FAKE, FAKE, None, 0, FAKE, None) == code
    assert L.lsh_residual_fwd(_res(f=s), *[FAKE] * 7, 1, 0, None, FAKE, FAKE, None) == code


def test_norm_pointers_and_workspace(L):
    n = _norm()
    need = L.lsh_norm_bwd_workspace_size(n)
    assert need > 0 and need % 256 == 0
    assert L.lsh_norm_fwd(None, FAKE, None, None, FAKE, None) == 1
    assert L.lsh_norm_fwd(n, None, None, None, FAKE, None) == 1
    assert L.lsh_norm_fwd(n, FAKE, None, None, None, None) == 1
    assert L.lsh_norm_fwd(n, FAKE + 1, None, None, FAKE, None) == 1       # half an element
    assert L.lsh_norm_fwd(n, FAKE, FAKE + 2, None, FAKE, None) == 1       # parameters are float32
    bwd = [FAKE, FAKE, FAKE, None, FAKE, FAKE, FAKE]
    assert L.lsh_norm_bwd(n, *bwd, FAKE, need - 1, None) == 3
    assert L.lsh_norm_bwd(n, *bwd, None, need, None) == 3
    assert L.lsh_norm_bwd(n, *bwd, FAKE + 16, need, None) == 3
    for i in (0, 2, 4):                                                   # x, dh, dx
        bad = list(bwd)
        bad[i] = None
        assert L.lsh_norm_bwd(n, *bad, FAKE, need, None) == 1


@pytest.mark.parametrize("kw,code", SIZES + [
    (dict(post=3), 1), (dict(norm=-1), 1), (dict(gate=3), 1), (dict(gate_batch=2), 1),
    (dict(gate=2, gate_batch=1), 1), (dict(gate=0, gate_batch=1), 1), (dict(eps=0.0), 1),
    (dict(eps_post=float("inf")), 1), (dict(alpha=float("nan")), 1), (dict(beta=float("inf")), 1),
    (dict(p=-0.1), 1), (dict(p=1.5), 1), (dict(p=float("nan")), 1), (dict(slice0=-1), 1),
    (dict(H=256), 2)])
def test_residual_refuses(L, kw, code):
    q = _res(**kw)
    assert L.lsh_residual_fwd(q, *[FAKE] * 7, 1, 0, None, FAKE, FAKE, None) == code
    assert L.lsh_residual_bwd_workspace_size(q) == 0
    assert L.lsh_residual_bwd(q, *[FAKE] * 8, 1, 0, None, *[FAKE] * 8, BIG, None) == code


def test_residual_pointers_and_workspace(L):
    q = _res()
    need = L.lsh_residual_bwd_workspace_size(q)
    assert need > 0 and need % 256 == 0
    fwd = [FAKE] * 7 + [1, 0, None, FAKE, FAKE]
    for i in (0, 1, 2, 10, 11):                    # x, f, gate, y, h
        bad = list(fwd)
        bad[i] = None
        assert L.lsh_residual_fwd(q, *bad, None) == 1
    bad = list(fwd)
    bad[9] = FAKE + 4                              # the counter is 8 bytes
    assert L.lsh_residual_fwd(q, *bad, None) == 1
    bwd = [FAKE] * 8 + [1, 0, None] + [FAKE] * 7
    assert L.lsh_residual_bwd(q, *bwd, FAKE, need - 1, None) == 3
    assert L.lsh_residual_bwd(q, *bwd, None, need, None) == 3
    for i in (1, 2, 3, 4, 12):                     # dh, y, f, gate, df
        bad = list(bwd)
        bad[i] = None
        assert L.lsh_residual_bwd(q, *bad, FAKE, need, None) == 1
    # gradients of what the problem does not have
    for kw in (dict(norm=0), dict(post=0), dict(gate=0)):
        assert L.lsh_residual_bwd(_res(**kw), *bwd, FAKE, BIG, None) == 1
    bad = [None] + bwd[1:]                         # no dy is fine with a norm, not without
    bad[1] = bad[2] = bad[16] = bad[17] = None
    assert L.lsh_residual_bwd(_res(norm=0), *bad, FAKE, BIG, None) == 1


@pytest.mark.parametrize("kw,code", SIZES + [(dict(p=-1e-9), 1), (dict(p=1.001), 1),
                                             (dict(p=float("nan")), 1), (dict(slice0=-1), 1),
                                             (dict(slice0=1 << 40), 1)])
def test_dropout_refuses(L, kw, code):
    assert L.lsh_dropout_fwd(_drop(**kw), FAKE, 1, 0, None, FAKE, None) == code


def test_dropout_pointers(L):
    q = _drop()
    assert L.lsh_dropout_fwd(q, None, 1, 0, None, FAKE, None) == 1
    assert L.lsh_dropout_fwd(q, FAKE, 1, 0, None, FAKE + 1, None) == 1
    assert L.lsh_dropout_fwd(q, FAKE, 1, 0, FAKE + 4, FAKE, None) == 1


@pytest.mark.parametrize("kw,code", SIZES[:-1] + [
    (dict(rot=0), 1), (dict(rot=7), 1), (dict(rot=66), 1), (dict(rot=-2), 1), (dict(d=63, rot=2), 1),
    (dict(amp=float("inf")), 1), (dict(d=514, rot=2), 2)])
def test_rope_refuses(L, kw, code):
    q = _rope(**kw)
    assert L.lsh_rope_fwd(q, FAKE, FAKE, None, 0, FAKE, None) == code
    assert L.lsh_rope_bwd(q, FAKE, FAKE, None, 0, FAKE, None) == code


def test_rope_flags_and_pointers(L):
    q = _rope()
    q.interleaved = 2
    assert L.lsh_rope_fwd(q, FAKE, FAKE, None, 0, FAKE, None) == 1
    q = _rope()
    q.pos_batch = -1
    assert L.lsh_rope_fwd(q, FAKE, FAKE, None, 0, FAKE, None) == 1
    q = _rope()
    assert L.lsh_rope_fwd(q, None, FAKE, None, 0, FAKE, None) == 1
    assert L.lsh_rope_fwd(q, FAKE, None, None, 0, FAKE, None) == 1
    assert L.lsh_rope_fwd(q, FAKE, FAKE + 4, None, 0, FAKE, None) == 1
    assert L.lsh_rope_fwd(q, FAKE, FAKE, FAKE + 2, 0, FAKE, None) == 1


@pytest.mark.parametrize("kw", [dict(B=0), dict(L=0), dict(H=0)])
def test_empty_problems_launch_nothing(L, kw):
    assert L.lsh_norm_fwd(_norm(**kw), None, None, None, None, None) == 0
    assert L.lsh_norm_bwd(_norm(**kw), *[None] * 8, 0, None) == 0
    assert L.lsh_dropout_fwd(_drop(**kw), None, 1, 0, None, None, None) == 0
    assert L.lsh_rope_fwd(_rope(**kw), None, None, None, 0, None, None) == 0
    assert L.lsh_residual_fwd(_res(**kw), *[None] * 7, 1, 0, None, None, None, None) == 0
    assert L.lsh_residual_bwd(_res(**kw), *[None] * 8, 1, 0, None, *[None] * 8, 0, None) == 0


def test_drivers_refuse_before_anything_is_launched():
    import torch
    from efficient_transformer_lsh_b200 import sublayer as sl
    kw = dict(device="cpu")
    with pytest.raises(_lib.LshError):
        sl.Norm(1, 2, 3, kind="batch", **kw)
    with pytest.raises(_lib.LshError):
        sl.Norm(1, 200, 3, **kw)                                   # too wide
    with pytest.raises(_lib.LshError):
        sl.Norm(1, 2, 3, dtype="f16", **kw)
    with pytest.raises(_lib.LshError):
        sl.Norm(1, 2, 3, x_layout="channels", **kw)
    with pytest.raises(_lib.LshError):
        sl.Residual(1, 2, 3, gate="tanh", **kw)
    with pytest.raises(_lib.LshError):
        sl.Dropout(1, 2, 3, 1.2, **kw)
    with pytest.raises(_lib.LshError):
        sl.Rotary(1, 2, 3, rot=66, **kw)
    with pytest.raises(_lib.LshError):
        sl.Rotary(1, 2, 3, scaling=("cubic", 2.0), **kw)
    with pytest.raises(_lib.LshError):
        sl.Rotary(1, 2, 3, frequencies=[1.0], **kw)
    n = sl.Norm(1, 2, 3, **kw)
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    for bad in (x.float(), x[:, :1], x.transpose(1, 2).contiguous().transpose(1, 2)):
        with pytest.raises(_lib.LshError):
            n.forward(bad)
    with pytest.raises(_lib.LshError):
        n.forward(x, torch.ones(64))
    with pytest.raises(_lib.LshError):
        n.forward(x, torch.ones(128, dtype=torch.bfloat16))
    r = sl.Residual(1, 2, 3, gate="vector", p=0.1, **kw)
    with pytest.raises(_lib.LshError):
        r.forward(x, x)                                            # the gate is missing
    with pytest.raises(_lib.LshError):
        r.forward(x, x, torch.ones(128), w=torch.ones(128))        # no norm of y
    with pytest.raises(_lib.LshError):
        r.forward(x, x, torch.ones(128), seed=-1)
    with pytest.raises(_lib.LshError):
        r.backward(x, x, dh=x, gate=torch.ones(128))
    with pytest.raises(_lib.LshError):
        sl.Residual(1, 2, 3, beta=0.0, **kw).restore(x, x)
    e = sl.Rotary(1, 2, 3, **kw)
    with pytest.raises(_lib.LshError):
        e.forward(x, pos=torch.zeros(3, dtype=torch.int64))
    with pytest.raises(_lib.LshError):
        e.forward(x, pos=torch.zeros(2, 3, dtype=torch.int32))


def test_problem_structs_match_the_header():
    """Sizes that the C compiler gives the same field lists."""
    for s, n in ((_lib.lsh_strides, 24), (_lib.lsh_norm_problem, 80),
                 (_lib.lsh_dropout_problem, 80), (_lib.lsh_residual_problem, 112),
                 (_lib.lsh_rope_problem, 88)):
        assert ctypes.sizeof(s) == n, s


def test_rope_backward_sum_refuses(L):
    ok = [FAKE, FAKE, FAKE, None, 0, FAKE, None]
    for kw, code in ((dict(rot=3), 1), (dict(rot=-2), 1), (dict(rot=66), 1), (dict(B=-1), 1),
                     (dict(x=(1, 2, 3)), 1), (dict(d=514), 2)):
        assert L.lsh_rope_bwd_sum(_rope(**kw), *ok) == code
    for i in (0, 1, 2, 5):                 # dqk, dv, turns, dx
        bad = list(ok)
        bad[i] = None
        assert L.lsh_rope_bwd_sum(_rope(), *bad) == 1
    bad = list(ok)
    bad[0] = FAKE + 2
    assert L.lsh_rope_bwd_sum(_rope(), *bad) == 1
    assert L.lsh_rope_bwd_sum(_rope(B=0), None, None, None, None, 0, None, None) == 0
