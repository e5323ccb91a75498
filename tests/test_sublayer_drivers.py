"""What the sublayer drivers refuse or build on the host, without a GPU."""
import pytest

from efficient_transformer_lsh_b200 import _lib

CPU = dict(device="cpu")


@pytest.fixture(scope="module")
def sl():
    import os
    if not os.path.exists(_lib.LIB_PATH):
        from efficient_transformer_lsh_b200 import build
        build.build()
    from efficient_transformer_lsh_b200 import sublayer
    return sublayer


@pytest.mark.parametrize("s", [(0, 0, 0), (384, 192, 0), (0, 192, 64), (384, -192, 64)])
def test_layouts_of_shared_or_backward_rows_are_refused(sl, s):
    """All strides zero say "contiguous" to the C ABI: an expanded tensor and
    the driver's own buffer of those strides hold one row."""
    for make in (lambda: sl.Norm(2, 3, 3, x_layout=s, **CPU),
                 lambda: sl.Norm(2, 3, 3, h_layout=s, **CPU),
                 lambda: sl.Residual(2, 3, 3, x_layout=s, **CPU),
                 lambda: sl.Residual(2, 3, 3, f_layout=s, **CPU),
                 lambda: sl.Dropout(2, 3, 3, 0.1, x_layout=s, **CPU),
                 lambda: sl.Dropout(2, 3, 3, 0.1, y_layout=s, **CPU),
                 lambda: sl.Rotary(2, 3, 3, x_layout=s, **CPU),
                 lambda: sl.Rotary(2, 3, 3, y_layout=s, **CPU)):
        with pytest.raises(_lib.LshError):
            make()


def test_strides_of_single_elements_say_nothing(sl):
    assert sl.Norm(1, 1, 1, x_layout=(0, 0, 0), **CPU).dx.shape == (1, 1, 1, 64)
    assert sl.Norm(1, 2, 1, x_layout=(0, 64, -5), **CPU).dx.shape == (1, 2, 1, 64)
    assert sl.Dropout(2, 0, 3, 0.1, x_layout=(0, 0, 0), **CPU).y.numel() == 0


def test_host_memory_is_refused_by_every_call(sl):
    """A driver of a device that no kernel runs on is refused with the argument
    error, not by whatever a launch on host addresses does."""
    import torch
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    w, pos = torch.ones(128), torch.zeros(3, dtype=torch.int32)
    f32 = x.float()
    n, d, e = sl.Norm(1, 2, 3, **CPU), sl.Dropout(1, 2, 3, 0.1, **CPU), sl.Rotary(1, 2, 3, **CPU)
    r, q = sl.Residual(1, 2, 3, norm="rms", **CPU), sl.Residual(1, 2, 3, **CPU)
    lay = sl.ReversibleLayer(1, 2, 128, 2, 1, 64, True, 256, 128, norm="rms", rot=0, **CPU)
    z = torch.zeros(1, 2, 128, 64, dtype=torch.bfloat16)
    R = torch.zeros(1, 64, 1, dtype=torch.bfloat16)
    p = dict(W1=torch.zeros(128, 256).bfloat16(), W2=torch.zeros(256, 128).bfloat16(),
             b1=torch.zeros(256), b2=torch.zeros(128), norm1_w=w, norm2_w=w)
    for call in (lambda: n.forward(x, w, w), lambda: n.backward(x, x, w, w, x),
                 lambda: n.forward(x, stream=0), lambda: d.forward(x, 1),
                 lambda: d.backward(x, 1), lambda: e.forward(x, pos), lambda: e.backward(x),
                 lambda: e.backward_sum(f32, f32), lambda: r.forward(x, x, w=w),
                 lambda: r.restore(x, x), lambda: r.backward(None, x, x, x),
                 lambda: q.forward(x, x), lambda: q.backward(x, x),
                 lambda: lay.forward(z, z, R, p), lambda: lay.backward(z, z, z, z, p)):
        with pytest.raises(_lib.LshError) as err:
            call()
        assert err.value.code == 1


@pytest.mark.parametrize("dims", [((1 << 32) + 1, 1, 0), (1, (1 << 32) + 1, 0),
                                  (0, 1, (1 << 32) + 1), (1 << 31, 1, 0)])
def test_sizes_past_32_bits_are_refused(sl, dims):
    """The C structs hold 32-bit sizes: a larger one would be cut to another
    problem. (Empty problems, so that no buffer of that size is made.)"""
    for make in (lambda: sl.Norm(*dims, d=1, **CPU), lambda: sl.Residual(*dims, d=1, **CPU),
                 lambda: sl.Dropout(*dims, 0.1, d=1, **CPU),
                 lambda: sl.Rotary(*dims, d=2, **CPU)):
        with pytest.raises(_lib.LshError):
            make()
    with pytest.raises(_lib.LshError):
        sl.Dropout(1, 1, 0, 0.1, d=(1 << 32) + 8, **CPU)


@pytest.mark.parametrize("slice0", [-1, 1 << 31, 1 << 64, (1 << 64) + 3])
def test_slices_past_32_bits_are_refused(sl, slice0):
    """2^64 + 3 would be cut to slice 3, and draw its mask."""
    with pytest.raises(_lib.LshError):
        sl.Dropout(1, 2, 3, 0.1, slice0=slice0, **CPU)
    with pytest.raises(_lib.LshError):
        sl.Residual(1, 2, 3, p=0.1, slice0=slice0, **CPU)


def _pi(bits):
    """floor(pi 2^bits) by Machin's formula, 16 atan(1/5) - 4 atan(1/239)."""
    def atan_inv(n):
        one = 1 << (bits + 32)
        total, term, k, sign = 0, one // n, 1, 1
        while term:
            total += sign * (term // k)
            term //= n * n
            k, sign = k + 2, -sign
        return total
    return (16 * atan_inv(5) - 4 * atan_inv(239)) >> 32


def exact_turns():
    """10000^(-2i/64) / 2 pi as fractions right to 100 bits: 10^(-i/8) is three
    integer square roots."""
    from fractions import Fraction
    from math import isqrt
    pi, out = Fraction(_pi(250), 1 << 250), []
    for i in range(32):
        root = isqrt(isqrt(isqrt(10 ** (8 * 60 - i))))
        out.append(Fraction(root, 10 ** 60) / (2 * pi))
    return out


def test_rope_tables_hold_64_bits(sl):
    """Within half a unit of 2^-64, which is |position| 2^-65 turns of phase."""
    from fractions import Fraction
    half = Fraction(1, 2) + Fraction(1, 1000)
    off = lambda n, t: abs((int(n) % (1 << 64) - t % 1 * (1 << 64) + (1 << 63)) % (1 << 64)
                           - (1 << 63))
    for scale in (1, 8):
        e = sl.Rotary(1, 1, 1, scaling=("linear", scale) if scale > 1 else None, **CPU)
        for n, t in zip(e.turns, exact_turns()):
            assert off(n, t / scale) <= half
    # given frequencies are what their doubles say
    pi = Fraction(_pi(250), 1 << 250)
    fs = [1.0, 0.1, 3.0e-5, 6.5, -0.25, 1e9 + 0.5, 0.0]
    for n, f in zip(sl.rope_turns(fs), fs):
        assert off(n, Fraction(f) / (2 * pi)) <= half
    for bad in (float("nan"), float("inf")):
        with pytest.raises(_lib.LshError):
            sl.rope_turns([bad])
    for base in (0.0, -2.0, float("inf")):
        with pytest.raises(_lib.LshError):
            sl.rope_frequencies(64, base)


@pytest.mark.parametrize("rot", [0, 64])
def test_the_layer_holds_no_buffer_that_nothing_writes(sl, rot):
    """Its second norm runs forward only; the gradients of the first norm and of
    the rotary positions are the drivers' own buffers."""
    import torch
    lay = sl.ReversibleLayer(1, 2, 128, 2, 1, 64, True, 256, 128, rot=rot, **CPU)
    assert lay.dx2 is lay.norm1.dx
    if rot:
        assert lay.dn is lay.rope.dx
    assert [getattr(lay.norm2, k) for k in ("dx", "dw", "db", "ws")] == [None] * 4
    size = lay.dx2.numel()
    held = {}
    for o in (lay, lay.norm1, lay.norm2, lay.join1, lay.join2, *([lay.rope] if rot else [])):
        for k, v in vars(o).items():
            if isinstance(v, torch.Tensor) and v.numel() == size and v.dtype == torch.bfloat16:
                held[v.data_ptr()] = k
    # n, m twice, q and its gradient; y, x, dx and df of each join; g, dm, and dn
    # without rotary positions, dx2
    assert len(held) == 3 + (2 if rot else 1) + 8 + 2 + 1
    n = sl.Norm(1, 2, 3, forward_only=True, **CPU)
    x = torch.zeros(1, 2, 3, 64, dtype=torch.bfloat16)
    with pytest.raises(_lib.LshError):
        n.backward(x, x)
