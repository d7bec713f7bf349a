"""How the linear layer's products are cut (CPU: host arithmetic only)."""
import ctypes as C

import pytest

import blockwise_fp8_zero_amd as bfz

F32, BF16, F16 = 0, 1, 2


def shape(product, n, rows, cols, dtype):
    out = (C.c_int64 * 6)()
    assert bfz.lib().bfz_linear_shape(product, n, rows, cols, dtype, out) == 0
    return tuple(out)


def test_refusals():
    f, out = bfz.lib().bfz_linear_shape, (C.c_int64 * 6)()
    for args in ((0, 5, 6, 7, 0, None), (3, 5, 6, 7, 0, out), (-1, 5, 6, 7, 0, out), (0, 0, 6, 7, 0, out), (0, 5, 0, 7, 0, out), (0, 5, 6, 0, 0, out),
                 (0, 5, 6, 7, 3, out), (0, (1 << 24) + 1, 6, 7, 0, out), (0, 5, (1 << 20) + 1, 7, 0, out), (0, 5, 6, (1 << 20) + 1, 0, out)):
        assert f(*args) == bfz.BFZ_EINVAL


@pytest.mark.parametrize("dtype", [F32, BF16, F16])
@pytest.mark.parametrize("product", [0, 1, 2])
def test_bounds(product, dtype):
    """What the workspace and the grids count on."""
    for n in (1, 16, 17, 33, 64, 65, 100, 300, 777, 1013, 2048, 5000, 8192, 100000):
        for rows in (1, 100, 1544, 4096, 11008, 28672):
            for cols in (1, 200, 1001, 4096, 16384):
                tm, tn, waves, splits, whole, exact = shape(product, n, rows, cols, dtype)
                few = product == 0 and n <= 64
                assert exact == (dtype != BF16 or (few and n <= 16))
                m, across, k = {0: (rows, n, cols), 1: (cols, n, rows), 2: (cols, rows, n)}[product]
                if few:
                    assert tm in (16, 32, 48) and tn == (16 if n <= 16 else 32 if n <= 32 else 64) and (splits, waves, whole) == (1, 8, n)
                    continue
                assert (tm, tn, waves) in {(256, 256, 8), (256, 128, 8), (128, 128, 8), (128, 128, 4), (128, 64, 8)} and not (exact and tn == 256)
                assert 0 <= whole <= across and (whole == across or (tm == 256 and whole % tn == 0))
                assert 1 <= splits <= -(-k // 128)
                tiles = -(-m // tm) * -(-across // tn)
                assert splits == 1 or (splits * tiles <= 256 and tm == 128)


@pytest.mark.parametrize("product,n,rows,cols,dtype", [(0, 1300, 4096, 4096, BF16), (0, 3000, 1700, 3600, F32), (1, 512, 4096, 11008, F32)])
def test_pairs_of_workgroups(product, n, rows, cols, dtype):
    """More tiles of 128 x 128 than CUs, too few of 256 x 128: two at a time on a CU
    take less than two rounds of them, or three of tiles half as wide (36.6 us
    instead of 48.5, 56.6 instead of 76, 63 instead of 87)."""
    assert shape(product, n, rows, cols, dtype)[:4] == (128, 128, 4, 1)
