"""How the 4-bit layer's calls are cut into tiles (host only, no GPU), through
dbf_debug_mx4_cut, and that what the cuts address lies in the workspace."""
import ctypes

import pytest

SMS = 148
FORWARD, GATED, GATED_ADD, GATED_SAVE, BACKWARD, GATED_BACKWARD = range(6)
FEW, MANY, GRADIENT = range(3)
HEADER = 256


@pytest.fixture(scope="module")
def dbf():
    import double_binary_rank_b200 as m
    return m


def cut(dbf, call, M, N, T, dy=None, sms=SMS):
    """The cut as a list, or the status that refused it."""
    out = (ctypes.c_int64 * 8)()
    st = dbf._lib.dbf_debug_mx4_cut(call, M, N, T, dbf.F32 if dy is None else dy, sms, out)
    return list(out) if st == dbf.OK else st


def test_refusals(dbf):
    assert cut(dbf, 6, 64, 64, 4) == cut(dbf, -1, 64, 64, 4) == cut(dbf, FORWARD, 0, 64, 4) == cut(dbf, FORWARD, 64, 64, 0) == dbf.ERR_INVALID_ARG
    assert cut(dbf, FORWARD, 64, 64, 4, sms=0) == cut(dbf, BACKWARD, 64, 64, 4, dy=dbf.F16) == dbf.ERR_INVALID_ARG
    assert cut(dbf, FORWARD, 64, 64, 1 << 40) == cut(dbf, BACKWARD, 64, 64, 1 << 30) == dbf.ERR_UNSUPPORTED
    assert dbf._lib.dbf_debug_mx4_cut(FORWARD, 64, 64, 4, 0, SMS, None) == dbf.ERR_INVALID_ARG


@pytest.mark.parametrize("call", [FORWARD, GATED, GATED_ADD, GATED_SAVE])
@pytest.mark.parametrize("M,N", [(1, 1), (32, 8192), (520, 1352), (4096, 11008)])
def test_the_last_tokens_scales_lie_in_the_workspace(dbf, call, M, N):
    """Token counts up to the largest that are taken: the scale rows of a tile's tokens are padded to 128 or 256, so that
    a scale row passes 2^31 where the token's number does not."""
    L = dbf.DbfMx4LayerC(M, N, 0x1000, 0x1000)
    taken = 0
    for T in (1, 16, 17, 100, 4095, 270_001, 1 << 28, (1 << 28) + 5, 1_878_000_000, 1_900_000_001, 2_000_000_000, (1 << 31) - 4097):
        got = cut(dbf, call, M, N, T)
        if got == dbf.ERR_UNSUPPORTED:
            continue
        taken += 1
        w, row = got[1], got[7]
        assert T - 1 <= row < (T + 15) // 16 * 128, (T, got)
        pad = 256 if got[0] == MANY and w > 128 else 128
        assert row == (T - 1) // w * pad + (T - 1) % w
        # x's codes, then its scales: tiles of 128 rows x 4 blocks, 512 bytes each
        tiles = -(-M // 128)
        codes = -(-(HEADER + T * -(-M // 32) * 16) // 256) * 256
        need = codes + (row // 128 + 1) * tiles * 512
        assert need <= dbf._lib.dbf_mx4_workspace_bytes(ctypes.byref(L), T)
    assert taken >= 8
    if (M, N) == (1, 1):
        assert taken == 12   # the largest count is taken, not refused
