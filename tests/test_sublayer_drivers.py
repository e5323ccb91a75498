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
