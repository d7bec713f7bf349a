"""What is too large for one launch is refused by its size, before any launch, and
what is not is judged by its other arguments (CPU: pointers here are never
followed)."""
import pytest

from tests.test_layer_refusals_cpu import EINVAL, _linear, _quantize, bfz

TOKENS = 1 << 24


def said():
    return bfz.lib().bfz_last_error().decode()


@pytest.mark.parametrize("n,d,tiles,fits", [
    (TOKENS, 4096, 0, False), (TOKENS - 8, 4096, 0, True), (TOKENS, 3584, 0, True), (TOKENS, 3585, 0, False), (1 << 20, 1 << 16, 0, False),
    ((1 << 20) - 8, 1 << 16, 0, True), (TOKENS, 8192, 1, False), (TOKENS, 8064, 1, True), (TOKENS - 128, 8192, 1, True), (TOKENS, 1 << 20, 1, False),
])
def test_quantize(n, d, tiles, fits):
    """A scale array that is not there is looked at after the sizes."""
    assert _quantize(n=n, d=d, xld=d, cld=d + (-d % 16), sld=1 << 24, tiles=tiles, scales=None) == EINVAL
    assert ("too many" not in said()) == fits, said()
    assert ("scales" in said()) == fits, said()


@pytest.mark.parametrize("n,cols,fits", [(TOKENS, 4096, False), (TOKENS - 8, 4096, True)])
def test_values_of_a_product(n, cols, fits):
    """Few rows, so that the result itself is small enough."""
    rc = _linear(x=None if fits else bfz.C.c_void_p(0x10000), xt=1, xld=cols, s=None, sld=0, n=n, wld=cols, rows=64, cols=cols, old=64)
    assert rc == EINVAL and ("too many" not in said()) == fits, said()
