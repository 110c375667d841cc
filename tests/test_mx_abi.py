"""Host-side argument checks and size queries of the 4-bit layer's entry points
(they return before any CUDA call) and of their Python wrappers; no GPU."""
import ctypes

import pytest
import torch

P = 0x1000


@pytest.fixture(scope="module")
def dbf():
    import double_binary_rank_b200 as m
    return m


@pytest.fixture(scope="module")
def lib(dbf):
    return dbf._lib


def test_sizes(lib):
    assert lib.dbf_mx4_code_bytes(3, 33) == 3 * 32 and lib.dbf_mx4_scale_bytes(3, 33) == 512
    assert lib.dbf_mx4_code_bytes(11008, 4096) == 11008 * 2048
    assert lib.dbf_mx4_scale_bytes(129, 129) == 2 * 2 * 512
    assert lib.dbf_act8_code_bytes(3, 33) == 3 * 64 and lib.dbf_act8_scale_bytes(3, 33) == 6
    for f in (lib.dbf_mx4_code_bytes, lib.dbf_mx4_scale_bytes, lib.dbf_act8_code_bytes, lib.dbf_act8_scale_bytes):
        assert f(0, 5) == 0 and f(5, 0) == 0 and f(-1, 5) == 0


def test_workspaces_grow_with_the_tokens(dbf, lib):
    by = ctypes.byref
    for M, N in ((1, 1), (520, 1352), (4096, 11008), (8192, 8192)):
        L = dbf.DbfMx4LayerC(M, N, P, P)
        qs = [lambda T: lib.dbf_mx4_workspace_bytes(by(L), T), lambda T: lib.dbf_mx4_gated_workspace_bytes(by(L), by(L), T)]
        for d in (dbf.F32, dbf.BF16):
            qs += [lambda T, d=d: lib.dbf_mx4_backward_workspace_bytes(by(L), T, d),
                   lambda T, d=d: lib.dbf_mx4_gated_backward_workspace_bytes(by(L), by(L), T, d)]
        for q in qs:
            got = [q(T) for T in (0, 1, 2, 15, 16, 17, 63, 64, 65, 128, 200, 224, 225, 511, 512, 513, 2048, 8191, 8192)]
            assert got[0] >= 256 and got == sorted(got)
    L = dbf.DbfMx4LayerC(0, 4, P, P)
    assert lib.dbf_mx4_workspace_bytes(by(L), 4) == 0 and lib.dbf_mx4_workspace_bytes(None, 4) == 0
    L = dbf.DbfMx4LayerC(4, 4, P, P)
    assert lib.dbf_mx4_workspace_bytes(by(L), -1) == 0
    assert lib.dbf_mx4_backward_workspace_bytes(by(L), 4, dbf.F16) == 0
    assert lib.dbf_mx4_gated_workspace_bytes(by(L), by(dbf.DbfMx4LayerC(4, 5, P, P)), 4) == 0


def test_quantize_refusals(dbf, lib):
    q, d = lib.dbf_mx4_quantize, lib.dbf_mx4_dequantize
    cb, sb = lib.dbf_mx4_code_bytes(4, 40), lib.dbf_mx4_scale_bytes(4, 40)
    assert q(None, dbf.F32, 4, 40, P, cb, P, sb, None, None) == dbf.ERR_INVALID_ARG
    assert q(P, dbf.I8, 4, 40, P, cb, P, sb, None, None) == dbf.ERR_INVALID_ARG
    assert q(P, dbf.F32, 0, 40, P, cb, P, sb, None, None) == dbf.ERR_INVALID_ARG
    assert q(P, dbf.F32, 4, 40, P, cb - 1, P, sb, None, None) == dbf.ERR_INVALID_ARG
    assert q(P, dbf.F32, 4, 40, P, cb, P, sb - 1, None, None) == dbf.ERR_INVALID_ARG
    assert q(P, dbf.F32, 4, 65535 * 256 + 1, P, 1 << 40, P, 1 << 40, None, None) == dbf.ERR_UNSUPPORTED
    assert q(P + 2, dbf.F32, 4, 40, P, cb, P, sb, None, None) == dbf.ERR_ALIGNMENT
    assert q(P, dbf.F32, 4, 40, P + 8, cb, P, sb, None, None) == dbf.ERR_ALIGNMENT
    assert q(P, dbf.F32, 4, 40, P, cb, P + 4, sb, None, None) == dbf.ERR_ALIGNMENT
    assert q(P, dbf.F32, 4, 40, P, cb, P, sb, P + 1, None) == dbf.ERR_ALIGNMENT
    assert d(P, None, 4, 40, P, dbf.F32, None) == dbf.ERR_INVALID_ARG
    assert d(P, P, 4, 40, P + 1, dbf.BF16, None) == dbf.ERR_ALIGNMENT
    a = dbf.DbfAct8C(P, P)
    assert lib.dbf_act8_save(P, dbf.F32, 4, 40, None, None, None) == dbf.ERR_INVALID_ARG
    assert lib.dbf_act8_save(P, dbf.F32, -1, 40, ctypes.byref(a), None, None) == dbf.ERR_INVALID_ARG
    assert lib.dbf_act8_save(None, dbf.F32, 0, 40, ctypes.byref(a), None, None) == dbf.OK
    assert lib.dbf_act8_load(ctypes.byref(dbf.DbfAct8C(P, None)), 4, 40, P, dbf.F32, None) == dbf.ERR_INVALID_ARG
    assert lib.dbf_act8_load(ctypes.byref(dbf.DbfAct8C(P + 8, P)), 4, 40, P, dbf.F32, None) == dbf.ERR_ALIGNMENT


def test_product_refusals(dbf, lib):
    by = ctypes.byref
    L = dbf.DbfMx4LayerC(96, 64, P, P)
    for f, need in ((lib.dbf_mx4_forward, lib.dbf_mx4_workspace_bytes(by(L), 4)),
                    (lib.dbf_mx4_backward, lib.dbf_mx4_backward_workspace_bytes(by(L), 4, dbf.F32))):
        call = lambda L=L, x=P, xd=dbf.F32, y=P, yd=dbf.F32, T=4, flags=0, ws=P, n=need: f(by(L) if L else None, x, xd, y, yd, T, flags, ws, n, None)
        assert call(L=None) == dbf.ERR_INVALID_ARG
        assert call(L=dbf.DbfMx4LayerC(96, 0, P, P)) == dbf.ERR_INVALID_ARG
        assert call(L=dbf.DbfMx4LayerC(96, 64, None, P)) == dbf.ERR_INVALID_ARG
        assert call(L=dbf.DbfMx4LayerC(96, 64, P + 8, P)) == dbf.ERR_ALIGNMENT
        assert call(L=dbf.DbfMx4LayerC(96, 64, P, P + 8)) == dbf.ERR_ALIGNMENT
        assert call(L=dbf.DbfMx4LayerC(65535 * 256 + 1, 64, P, P)) == dbf.ERR_UNSUPPORTED
        assert call(x=None) == call(y=None) == dbf.ERR_INVALID_ARG
        assert call(xd=dbf.F16) == call(yd=dbf.F16) == call(xd=7) == dbf.ERR_INVALID_ARG
        assert call(T=-1) == call(flags=4) == dbf.ERR_INVALID_ARG
        assert call(T=1 << 40) == dbf.ERR_UNSUPPORTED
        assert call(x=P + 8) == call(y=P + 4) == call(ws=P + 64) == dbf.ERR_ALIGNMENT
        assert call(ws=None) == call(n=need - 1) == dbf.ERR_WORKSPACE
        assert call(T=0, x=None, y=None, ws=None, n=0) == dbf.OK


def test_gated_refusals(dbf, lib):
    by = ctypes.byref
    L, other, A = dbf.DbfMx4LayerC(96, 64, P, P), dbf.DbfMx4LayerC(96, 65, P, P), dbf.DbfAct8C(P, P)
    need = lib.dbf_mx4_gated_workspace_bytes(by(L), by(L), 4)

    def fwd(up=L, act=0, x=P, xd=dbf.F32, g=None, u=None, ad=dbf.F32, h=P, hd=dbf.F32, sg=None, su=None, T=4, flags=0, ws=P, n=need):
        return lib.dbf_mx4_gated_forward(by(L), by(up), act, x, xd, g, u, ad, h, hd, sg and by(sg), su and by(su), T, flags, ws, n, None)

    assert fwd(up=other) == fwd(act=2) == fwd(xd=dbf.F16) == fwd(hd=dbf.I8) == dbf.ERR_INVALID_ARG
    assert fwd(g=P, ad=dbf.F16) == fwd(u=P, ad=9) == dbf.ERR_INVALID_ARG
    assert fwd(sg=A) == fwd(su=A) == fwd(sg=A, su=dbf.DbfAct8C(P, None)) == dbf.ERR_INVALID_ARG
    assert fwd(flags=dbf.ACCUMULATE) == fwd(x=None) == fwd(h=None) == dbf.ERR_INVALID_ARG
    assert fwd(g=P + 8) == fwd(h=P + 8) == fwd(sg=A, su=dbf.DbfAct8C(P + 4, P)) == fwd(ws=P + 16) == dbf.ERR_ALIGNMENT
    assert fwd(n=need - 1) == fwd(ws=None) == dbf.ERR_WORKSPACE
    assert fwd(T=0, x=None, h=None, ws=None) == dbf.OK
    need = lib.dbf_mx4_gated_backward_workspace_bytes(by(L), by(L), 4, dbf.BF16)

    def bwd(up=L, act=0, sg=A, su=A, dh=P, dt=dbf.BF16, dg=P, du=P, dx=P, xd=dbf.F32, T=4, flags=0, ws=P, n=need):
        return lib.dbf_mx4_gated_backward(by(L), by(up), act, sg and by(sg), su and by(su), dh, dt, dg, du, dx, xd, T, flags, ws, n, None)

    assert bwd(up=other) == bwd(act=-1) == bwd(dt=dbf.F16) == bwd(xd=dbf.F16) == bwd(flags=8) == dbf.ERR_INVALID_ARG
    assert bwd(sg=None) == bwd(su=dbf.DbfAct8C(None, P)) == bwd(dh=None) == bwd(dg=None) == bwd(du=None) == dbf.ERR_INVALID_ARG
    assert bwd(dh=P + 8) == bwd(dg=P + 8) == bwd(dx=P + 8) == bwd(ws=P + 16) == dbf.ERR_ALIGNMENT
    assert bwd(up=dbf.DbfMx4LayerC(96, 64, P + 4, P)) == dbf.ERR_ALIGNMENT
    assert bwd(n=need - 1) == bwd(ws=None) == dbf.ERR_WORKSPACE
    assert bwd(T=0, dh=None) == dbf.OK


def test_python_refuses_host_tensors(dbf):
    x = torch.ones(4, 96)
    with pytest.raises(ValueError):
        dbf.mx4_quantize(x)
    with pytest.raises(ValueError):
        dbf.act8_save(x)
    codes, scales = torch.zeros(64, 48, dtype=torch.uint8), torch.zeros(1, 1, 32, 4, 4, dtype=torch.uint8)
    with pytest.raises(ValueError):
        dbf.mx4_dequantize(codes, scales, 64, 96)
    layer = dbf.Mx4Layer(96, 64, codes, scales)
    with pytest.raises(ValueError):
        dbf.mx4_forward(layer, x)
    with pytest.raises(ValueError):   # codes of another width
        dbf.Mx4Layer(128, 64, codes, scales)


def test_sizes_that_32_bits_cannot_count(dbf, lib):
    by = ctypes.byref
    big = 2 ** 31 - 1
    L = dbf.DbfMx4LayerC(32, big, P, P)
    assert lib.dbf_mx4_workspace_bytes(by(L), 1) == 0
    assert lib.dbf_mx4_forward(by(L), P, dbf.F32, P, dbf.F32, 1, 0, P, 1 << 40, None) == dbf.ERR_UNSUPPORTED
    assert lib.dbf_mx4_backward(by(L), P, dbf.F32, P, dbf.F32, 1, 0, P, 1 << 40, None) == dbf.ERR_UNSUPPORTED
    L = dbf.DbfMx4LayerC(32, 64, P, P)
    assert lib.dbf_mx4_forward(by(L), P, dbf.F32, P, dbf.F32, big, 0, P, 1 << 62, None) == dbf.ERR_UNSUPPORTED
    assert lib.dbf_mx4_backward(by(L), P, dbf.F32, P, dbf.F32, big // 3, 0, P, 1 << 62, None) == dbf.ERR_UNSUPPORTED


def test_a_stream_of_another_device_is_refused(dbf):
    from types import SimpleNamespace
    on0 = SimpleNamespace(get_device=lambda: 0)
    with pytest.raises(ValueError, match="stream"):
        dbf._enter(on0, SimpleNamespace(device=torch.device("cuda", 1)))
    with pytest.raises(ValueError, match="CUDA"):
        dbf._enter(SimpleNamespace(get_device=lambda: -1), None)
