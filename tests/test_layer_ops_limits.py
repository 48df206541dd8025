"""Host-side checks of the C ABI of the norm, the short convolution and the
selective scan at the ends of its argument ranges (no GPU): every call is
refused before anything is launched; the addresses are never dereferenced."""
import ctypes

import pytest

import gated_delta_rule_104_b200._binding as b

BIG = 2 ** 31 - 1


def addr(i):
    return (1 << 46) + i * (1 << 40)


@pytest.fixture(scope="module")
def lib():
    return b.load()


@pytest.mark.parametrize("T", [1, 8, 1 << 20, BIG])
def test_conv_prompt_refuses_tiles_that_pass_31_bits(lib, T):
    """T / 8 + n_seq tiles, and one, are numbered in 32 bits."""
    c = b.dl_conv(addr(0), None, 1, 2, b.DL_BF16, 1)
    n = BIG - T // 8
    args = (addr(1), 1, T, addr(2), n, addr(3), BIG, None, None, addr(4), None)
    assert lib.dl_conv_prompt(ctypes.byref(c), *args) == b.DL_ERR_UNSUPPORTED
    assert b"n_seq" in lib.dl_last_error()
