"""The cross entropy's descriptor flags (no GPU needed: the addresses are never read)."""
import ctypes

import pytest

import selective_state_space_17_amd as M

BASE, MB = 0x7F0000000000, 1 << 20
AT = [BASE + i * 100 * MB for i in range(9)]


def fwd(flags, io=M.MSSM_BF16):
    d = M.CrossEntropyDesc(8, 32, 64, -100, io, 8, flags)
    return M.lib.mssm_linear_cross_entropy_fwd(ctypes.byref(d), *AT[:6], 0, None)


def bwd(flags, io=M.MSSM_BF16):
    d = M.CrossEntropyDesc(8, 32, 64, -100, io, 8, flags)
    return M.lib.mssm_linear_cross_entropy_bwd(ctypes.byref(d), *AT[:8], M.MSSM_F32, 0, AT[8], 0, None)


@pytest.mark.parametrize("io", [M.MSSM_BF16, M.MSSM_F32])
def test_flags(io):
    """The one flag passes the checks (a workspace of no bytes is then what is refused); others do not."""
    assert M.MSSM_CROSS_ENTROPY_FINE_G == 2
    for call in (fwd, bwd):
        assert call(0, io) == M.MSSM_ERR_WORKSPACE and call(M.MSSM_CROSS_ENTROPY_FINE_G, io) == M.MSSM_ERR_WORKSPACE
        for flags in (1, 3, 4, 1 << 31):
            assert call(flags, io) == M.MSSM_ERR_INVALID_ARG


def test_workspace():
    """Sixteen bits of the logits' gradient take room where eight would do, and only there."""
    size = M.linear_cross_entropy_bwd_workspace_size
    assert size(300, 2049, 64, fine=True) - size(300, 2049, 64) >= 512 * 2049 * 2
    assert size(256, 2049, 64, fine=True) == size(256, 2049, 64)
    assert size(300, 2049, 64, M.MSSM_F32, fine=True) == size(300, 2049, 64, M.MSSM_F32)
    assert M.linear_cross_entropy_bwd_workspace_size(300, 0, 64, fine=True) == 0
