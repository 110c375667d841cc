"""Outputs of the 4-bit layer's calls that share memory with an input or with one
another are refused before anything is launched; no GPU."""
import ctypes

import pytest

T, M, N = 4, 64, 64
SIZE = 1 << 16   # every buffer is smaller


@pytest.fixture(scope="module")
def dbf():
    import double_binary_rank_b200 as m
    return m


def places(n):
    return [0x100000 + i * SIZE for i in range(n)]


def test_forward(dbf):
    L = dbf.DbfMx4LayerC(M, N, *places(2))
    x, ws = 0x900000, 0xA00000
    need = dbf._lib.dbf_mx4_workspace_bytes(ctypes.byref(L), T)
    for y, yd in ((x, dbf.F32), (x, dbf.BF16), (x + 16, dbf.BF16), (x + T * M * 4 - 16, dbf.F32), (x - T * N * 4 + 16, dbf.F32)):
        assert dbf._lib.dbf_mx4_forward(ctypes.byref(L), x, dbf.F32, y, yd, T, 0, ws, need, None) == dbf.ERR_INVALID_ARG
    need = dbf._lib.dbf_mx4_backward_workspace_bytes(ctypes.byref(L), T, dbf.F32)
    for dx in (x, x + 32, x - 32):
        assert dbf._lib.dbf_mx4_backward(ctypes.byref(L), x, dbf.F32, dx, dbf.F32, T, 0, ws, need, None) == dbf.ERR_INVALID_ARG


def test_gated_forward(dbf):
    by = ctypes.byref
    L = dbf.DbfMx4LayerC(M, N, *places(2))
    x, h, gc, gs, uc, us, ws = (0x900000 + i * SIZE for i in range(7))
    need = dbf._lib.dbf_mx4_gated_workspace_bytes(by(L), by(L), T)

    def call(h=h, g=(gc, gs), u=(uc, us)):
        return dbf._lib.dbf_mx4_gated_forward(by(L), by(L), 0, x, dbf.F32, None, None, dbf.F32, h, dbf.F32, by(dbf.DbfAct8C(*g)),
                                              by(dbf.DbfAct8C(*u)), T, 0, ws, need, None)

    assert call(h=x) == call(h=gc) == call(h=us) == call(u=(gc, us)) == call(u=(uc, gs)) == dbf.ERR_INVALID_ARG
    assert call(g=(x, gs)) == call(u=(uc, x)) == call(g=(gc, gc)) == dbf.ERR_INVALID_ARG


def test_gated_backward(dbf):
    by = ctypes.byref
    L = dbf.DbfMx4LayerC(M, N, *places(2))
    dh, dg, du, dx, c, s, ws = (0x900000 + i * SIZE for i in range(7))
    need = dbf._lib.dbf_mx4_gated_backward_workspace_bytes(by(L), by(L), T, dbf.F32)

    def call(dg=dg, du=du, dx=dx):
        a = by(dbf.DbfAct8C(c, s))   # one of both is read twice, which is fine
        return dbf._lib.dbf_mx4_gated_backward(by(L), by(L), 0, a, a, dh, dbf.F32, dg, du, dx, dbf.F32, T, 0, ws, need, None)

    assert call(dg=du) == call(dg=dh) == call(du=dh) == call(dx=dg) == call(dx=du) == dbf.ERR_INVALID_ARG
    assert call(dg=dh + 16) == call(dg=dh, dx=None) == dbf.ERR_INVALID_ARG
