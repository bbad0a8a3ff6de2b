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


def test_the_stall_hook_refuses_limits_that_are_no_test(lib):
    for bad in (0, -1, 99_999, 1_000_000_001):
        assert lib.dg_debug_stall_paged(bad) == 1 and lib.dg_last_error()


class Word:
    """Stands in for a device error word."""

    def __init__(self, bits):
        self.bits = bits

    def item(self):
        return self.bits


@pytest.mark.parametrize("bits,status,text", [
    (binding.PAGED_TIMEOUT, 5, "wait"), (7, 5, "wait"), (binding.PAGED_BAD_BATCH, 1, "kv_len"),
    (binding.PAGED_BAD_PAGE, 1, "page number"), (3, 1, "page number")])
def test_every_error_bit_is_reported(monkeypatch, bits, status, text):
    monkeypatch.setattr(binding, "_arg", lambda *a: None)
    binding.dg_paged_check(Word(0))
    with pytest.raises(binding.DGError, match=text) as e:
        binding.dg_paged_check(Word(bits))
    assert e.value.status == status
