"""Host-side checks of the norm, the short convolution and the selective scan at
the ends of their argument ranges (no GPU): every call of the C ABI is refused
before anything is launched; the addresses are never dereferenced."""
import ctypes

import pytest
import torch

import gated_delta_rule_104_b200._binding as b
from tests import layer_ref as R

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


# ------------------------------------------------------------------ what a bound tells apart

@pytest.mark.parametrize("dv", [64, 128])
def test_two_parts_of_an_addend_do_not_reach_a_float32_state(dv):
    """The bound of test_ssm_prompt_keeps_a_float32_state_to_its_last_bits tells three bfloat16 parts of an addend from two, on the inputs that it takes."""
    f = R.one_addend(dv, 100 + dv)[3]
    part = f.float().to(torch.bfloat16)
    second = (f.float() - part.float()).to(torch.bfloat16)
    off = ((part.double() + second.double()) - f).abs()
    assert float((off > 4 * R.U32 * f.abs()).double().mean()) > 0.5
    third = (f.float() - part.float() - second.float()).to(torch.bfloat16)
    assert bool(((part.double() + second.double() + third.double() - f).abs() <= 2 * R.U32 * f.abs()).all())


# ------------------------------------------------------------------ the workspace

def test_a_workspace_that_does_not_fit_is_refused(lib):
    """One long sequence on few heads needs a workspace: given too small, missing, misaligned or inside another operand, it is refused."""
    T, H, dk, dv = 1 << 16, 6, 64, 128
    need = lib.dl_ssm_work_bytes(T, 1, H, dk, dv)
    assert need > 0
    m = b.dl_ssm(addr(3), H * dv, addr(4), H, addr(5), dk, addr(6), dk, None, 0, addr(7), None, None, b.DL_BF16)

    def call(work, size):
        status = lib.dl_ssm_prompt(addr(0), b.DL_F32, 1, None, None, ctypes.byref(m), addr(1), 1, T, addr(2), H, 1, dk, dv, work, size, None)
        return status, lib.dl_last_error().decode()

    for work, size, text in ((addr(8), need - 1, "work holds"), (None, need, "work is a null"), (addr(8) + 8, need, "aligned"),
                             (addr(2) + 4096, need, "overlaps")):
        status, error = call(work, size)
        assert status == b.DL_ERR_INVALID_ARG and text in error
