"""Sizes that the 8-bit projections refuse have no workspace and no launches, as the header says
of every operation; segment counts whose tiles no 32-bit number holds are refused."""
import ctypes

import pytest

import adapter_gemv_sgmv_b200 as L
from adapter_gemv_sgmv_b200 import build as B

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 32
FAKE = 0x10000
ROWS = 1 << 30


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


def _status(lib, op, N, d_in, d_out, max_rank=16, n_seg=2):
    """The entry point's answer with no workspace (32: nothing else is wrong)."""
    up = lambda d: (max(d, 1) + 15) // 16 * 16
    if op == L.OP_LINEAR_I8:
        return lib.lora_linear_i8(FAKE, up(d_in), FAKE, FAKE, up(d_in), FAKE, FAKE, 0, up(d_out), N, d_in, d_out, None, 0,
                                  None)
    pool = L.LoraPoolStruct(FAKE, FAKE, FAKE, FAKE, FAKE, 1 << 20, 1 << 20, 4, d_in, d_out, max_rank)
    return lib.lora_linear_i8_sgmv(FAKE, up(d_in), FAKE, FAKE, up(d_in), FAKE, up(d_in), FAKE, FAKE, up(d_out),
                                   ctypes.byref(pool), FAKE, FAKE, n_seg, N, 1.0, None, 0, None)


@pytest.mark.parametrize("op", [L.OP_LINEAR_I8, L.OP_LINEAR_I8_SGMV])
@pytest.mark.parametrize("N,d_in,d_out,ok", [
    (4, 64, 32, True), (0, 64, 32, True), (ROWS, 8, 8, True), (4, 65536, 8, True), (1, 8, ROWS, True),
    (-1, 64, 32, False), (ROWS + 1, 64, 32, False), (4, 60, 32, False), (4, 0, 32, False), (4, 65544, 32, False),
    (4, 64, 28, False), (4, 64, 0, False), (4, 64, ROWS + 8, False),
])
def test_refused_sizes_have_no_workspace(lib, op, N, d_in, d_out, ok):
    assert (_status(lib, op, N, d_in, d_out) == WORKSPACE) == ok
    assert (L.lora_workspace_size(op, N, 4, d_in, d_out, 16, 2) > 0) == ok
    if d_out == 32:                                # (the count of launches does not ask for d_out)
        assert (L.lora_kernel_launches(op, N, 4, d_in, 2) > 0) == (ok and N > 0)


@pytest.mark.parametrize("max_rank,ok", [(8, True), (128, True), (12, False), (0, False), (136, False)])
def test_refused_ranks_have_no_workspace(lib, max_rank, ok):
    assert (_status(lib, L.OP_LINEAR_I8_SGMV, 4, 64, 32, max_rank) == WORKSPACE) == ok
    assert (L.lora_workspace_size(L.OP_LINEAR_I8_SGMV, 4, 4, 64, 32, max_rank, 2) > 0) == ok


@pytest.mark.parametrize("op", [L.OP_SGMV_SHRINK, L.OP_SGMV_EXPAND, L.OP_LINEAR, L.OP_LINEAR_I8_SGMV])
def test_more_segments_than_tiles_can_be_counted(lib, op):
    """The largest counts: 2^31 - 1 tiles at N / 8 + n + 1."""
    most = 2 ** 31 - 1 - 1000 // 8 - 1
    assert L.lora_workspace_size(op, 1000, 4, 64, 32, 16, most) > 16 * most
    assert L.lora_workspace_size(op, 1000, 4, 64, 32, 16, most + 1) == 0
    assert L.lora_workspace_size(op, 1000, 4, 64, 32, 16, 2 ** 31 - 1) == 0
    if op == L.OP_LINEAR_I8_SGMV:
        assert _status(lib, op, 1000, 64, 32, n_seg=most) == WORKSPACE
        assert _status(lib, op, 1000, 64, 32, n_seg=most + 1) == INVALID
