"""Refusals of the paged-cache operators that need no GPU, beside those of test_paged_args."""
import math

import pytest

from masked_discrete_diffusion_b200 import binding, build
from test_paged_args import attention


@pytest.fixture(scope="module")
def lib():
    build.build()
    return binding.lib()


@pytest.mark.parametrize("window", [-(1 << 32), 1 << 31, 1 << 32, (1 << 32) + 5, (1 << 63) - 1])
def test_windows_that_32_bits_do_not_hold_are_refused(window):
    """Not cut to their low 32 bits (2^32 would be no limit, 2^32 + 5 five positions)."""
    with pytest.raises(ValueError, match="window"):
        binding.dg_paged_attention(None, None, None, window=window)


def test_scales_whose_exponents_overflow_are_refused(lib):
    """The kernel works in powers of two: scale log2(e) has to be finite as well."""
    top = 3.4028234663852886e38  # fp32's largest
    for scale in (top, 2.5e38, math.inf):
        assert attention(lib, scale=scale) == 1 and b"scale" in lib.dg_last_error(), scale
    # refused for its workspace instead, which is checked later
    assert attention(lib, scale=top / 1.4427, ws=None) == 1
    assert b"workspace" in lib.dg_last_error()
