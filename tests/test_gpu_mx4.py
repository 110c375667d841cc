"""The 4-bit base layer, its gated block and the 8-bit activations on the GPU
against plain 64-bit forms (tests/mx_ref.py).

Tolerances. Quantising is exact: a division by a power of two and one
rounding, so codes and scales are compared for equality. A product of
microscaled operands whose scales lie within a factor of 8 has terms that are
multiples of one unit and sums below 2^24 units: fp32 accumulation is exact
whatever its order, and y is compared for equality. On other data each of the K
additions may be off by one unit of fp32 (2^-23, truncation included) of a
partial sum that S = sum |terms| bounds: K 2^-23 S. Rounding to bf16 adds
2^-8 |y|."""
import ctypes

import numpy as np
import pytest
import torch

import mx_ref as R

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


@pytest.fixture(scope="module")
def dbf():
    import double_binary_rank_b200 as m
    return m


def host(t):
    return t.double().cpu().numpy()


# ---- formats
SHAPES = [(1, 1), (1, 32), (3, 33), (5, 31), (33, 256), (129, 72), (128, 1024), (31, 1371), (130, 2056), (257, 40)]


@pytest.mark.parametrize("rows,k", SHAPES)
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_quantize_is_exact(dbf, rows, k, kind):
    rng = np.random.default_rng(rows * 1000 + k)
    x = rng.standard_normal((rows, k)) * np.exp2(rng.integers(-8, 8, (rows, 1)))
    x[rng.random((rows, k)) < 0.1] = 0
    x[0, : min(k, 8)] = [0.25, 0.75, -1.25, 1.75, 2.5, -3.5, 5.0, 6.0][: min(k, 8)]   # ties when amax is 6
    t = torch.tensor(x).to(DT[kind]).cuda()
    val, codes, byte = R.mx4(host(t))
    packed, scales = R.pack4(codes, byte)
    gc, gs = dbf.mx4_quantize(t)
    assert torch.equal(gc.cpu(), torch.from_numpy(packed)) and torch.equal(gs.cpu(), torch.from_numpy(scales))
    for out in ("f32", "bf16"):
        assert np.array_equal(host(dbf.mx4_dequantize(gc, gs, rows, k, dtype=DT[out])), val)
    f16 = host(dbf.mx4_dequantize(gc, gs, rows, k, dtype=torch.float16))
    assert np.array_equal(f16, val.astype(np.float16).astype(np.float64))


@pytest.mark.parametrize("rows,k", SHAPES)
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
def test_act8_is_exact(dbf, rows, k, kind):
    rng = np.random.default_rng(rows * 999 + k)
    x = rng.standard_normal((rows, k)) * np.exp2(rng.integers(-8, 6, (rows, 1)))
    x[0, : min(k, 3)] = [448.0, 449.0, -1.0][: min(k, 3)]
    t = torch.tensor(x).to(DT[kind]).cuda()
    val, codes, byte = R.act8(host(t))
    a = dbf.act8_save(t)
    assert np.array_equal(a.codes.cpu().numpy(), codes.reshape(rows, -1).astype(np.uint8))
    assert np.array_equal(a.scales.cpu().numpy(), byte.T.astype(np.uint8))
    for out in ("f32", "bf16"):
        assert np.array_equal(host(dbf.act8_load(a, dtype=DT[out])), val)
    assert np.array_equal(host(dbf.act8_load(a, dtype=torch.float16)), val.astype(np.float16).astype(np.float64))


@pytest.mark.parametrize("f", ["mx4", "act8"])
def test_extreme_blocks(dbf, f):
    """Subnormals, the largest values, zeros, negative zeros, NaN and infinities."""
    tiny, big = 2.0 ** -149, float(np.finfo(np.float32).max)
    x = np.zeros((9, 64))
    x[0, 3], x[1, 40], x[2, :], x[3, :], x[4, :4] = np.nan, np.inf, -0.0, tiny, [2.0 ** -126, 2.0 ** -127, -(2.0 ** -125), tiny]
    x[5, :3], x[6, 0], x[7, :2], x[8, 63] = [big, -big, 1.0], -np.inf, [2.0 ** -120, 2.0 ** -119 * 1.75], 2.0 ** -118 * 1.8
    t = torch.tensor(x, dtype=torch.float32).cuda()
    val, codes, byte = getattr(R, f)(host(t))
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    if f == "mx4":
        gc, gs = dbf.mx4_quantize(t, status=status)
        packed, scales = R.pack4(codes, byte)
        assert np.array_equal(gs.cpu().numpy(), scales) and np.array_equal(gc.cpu().numpy(), packed)
        back = host(dbf.mx4_dequantize(gc, gs, 9, 64, dtype=torch.float32))
    else:
        a = dbf.act8_save(t, status=status)
        assert np.array_equal(a.scales.cpu().numpy(), byte.T.astype(np.uint8))
        assert np.array_equal(a.codes.cpu().numpy(), codes.reshape(9, -1).astype(np.uint8))
        back = host(dbf.act8_load(a, dtype=torch.float32))
    # the largest fp32 value / 2^120 is 2^8 (1 - 2^-24), whose nearest E4M3 code is 256: it stands for 2^128,
    # which fp32 reads as infinity
    with np.errstate(over="ignore"):
        val = val.astype(np.float32).astype(np.float64)
    assert np.array_equal(back, val, equal_nan=True)
    assert status.item() == dbf.ERR_INVALID_ARG
    status.zero_()
    ok = torch.ones(3, 5, device="cuda")
    dbf.mx4_quantize(ok, status=status) if f == "mx4" else dbf.act8_save(ok, status=status)
    assert status.item() == 0


# ---- products
def exact_operand(rng, rows, k):
    """Values that quantise to themselves, of scales 1 to 4: every block holds a code of 4 or 6."""
    v = R.E2M1[rng.integers(0, 8, (rows, k))] * rng.choice([-1.0, 1.0], (rows, k))
    v[:, ::32] = rng.choice([4.0, -6.0], v[:, ::32].shape)
    scale = np.repeat(np.exp2(rng.integers(0, 3, (rows, -(-k // 32)))), 32, axis=1)[:, :k]
    return v * scale


def layer_of(dbf, w):
    return dbf.Mx4Layer.quantize(torch.tensor(w, dtype=torch.float32).cuda())


PRODUCTS = [(1, 1, 1), (1, 32, 1), (2, 33, 5), (3, 64, 129), (16, 256, 128), (17, 1000, 130), (33, 2048, 257), (64, 4096, 300),
            (48, 520, 128), (64, 96, 640), (65, 512, 512), (77, 1000, 2200), (100, 300, 1030), (130, 288, 640), (241, 2048, 513),
            (257, 1, 3), (300, 95, 511), (1000, 768, 1537)]


@pytest.mark.parametrize("T,M,N", PRODUCTS)
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_forward_is_exact(dbf, T, M, N, kind):
    rng = np.random.default_rng(T * 7 + M * 3 + N)
    w, x = exact_operand(rng, N, M), exact_operand(rng, T, M)
    assert np.array_equal(R.mx4(x[: min(T, 5)])[0], x[: min(T, 5)])
    ref = x @ w.T
    L = layer_of(dbf, w)
    t = torch.tensor(x).to(DT[kind]).cuda()
    y = dbf.mx4_forward(L, t, y_dtype=torch.float32)
    assert np.array_equal(host(y), ref)
    y2 = dbf.mx4_forward(L, t, y=torch.full((T, N), 8.0, device="cuda"), accumulate=True)
    assert np.array_equal(host(y2), ref + 8)
    yb = dbf.mx4_forward(L, t, y_dtype=torch.bfloat16)
    assert torch.equal(yb.cpu(), torch.tensor(ref).float().to(torch.bfloat16))


@pytest.mark.parametrize("T,M,N", [(1, 4096, 384), (40, 1000, 200), (300, 2048, 1000)])
def test_forward_on_normal_data(dbf, T, M, N):
    rng = np.random.default_rng(T)
    w = rng.standard_normal((N, M)).astype(np.float32)
    x = (rng.standard_normal((T, M)) * np.exp2(rng.integers(-6, 6, (1, M)))).astype(np.float32)
    wq, xq = R.mx4(w)[0], R.mx4(x)[0]
    ref, S = xq @ wq.T, np.abs(xq) @ np.abs(wq.T)
    L = layer_of(dbf, w)
    for out in ("f32", "bf16"):
        y = host(dbf.mx4_forward(L, torch.from_numpy(x).cuda(), y_dtype=DT[out]))
        tol = M * 2.0 ** -23 * S
        assert np.all(np.abs(y - ref) <= tol + STEP[out] * (np.abs(ref) + tol))


# ---- gated block
# act(g) u from exact g and u: e^-g and its reciprocal are each off by at most
# 2 units of fp32 plus |g| 2^-23 from the argument's scaling by log2(e); with
# the products and sums of the formulas, 16 units and 4 |g| units cover both
# activations' values and slopes (relative to |g| + 1 for slopes and GELU,
# whose terms cancel) for the |g| below 60 that the tests reach.
def gate_tol(g):
    return (16 + 4 * np.abs(g)) * 2.0 ** -23


@pytest.mark.parametrize("T,M,N", [(1, 32, 1), (1, 4096, 256), (3, 33, 5), (17, 1000, 130), (64, 2048, 257), (65, 512, 512),
                                   (100, 300, 1030), (241, 1024, 513), (300, 95, 511)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("add", ["none", "both", "up"])
def test_gated_forward(dbf, T, M, N, act, add):
    rng = np.random.default_rng(T + M + N)
    # exact products, scaled by a power of two to the gate's working range
    down = 2.0 ** -np.ceil(np.log2(12 * np.sqrt(M)) - 1)
    wg, wu = exact_operand(rng, N, M) * down, exact_operand(rng, N, M) * down
    x = exact_operand(rng, T, M) * 0.25
    g, u = x @ wg.T, x @ wu.T
    ga, ua = (torch.randint(-8, 9, (T, N), generator=torch.Generator().manual_seed(i)).to(torch.bfloat16).cuda() for i in (1, 2))
    kw = {"none": {}, "both": {"g_add": ga, "u_add": ua}, "up": {"u_add": ua}}[add]
    if add != "none":
        u = u + host(ua)
    if add == "both":
        g = g + host(ga)
    gl, ul = layer_of(dbf, wg), layer_of(dbf, wu)
    t = torch.tensor(x).to(torch.bfloat16).cuda()
    save = dbf.Act8.empty(T, N, "cuda"), dbf.Act8.empty(T, N, "cuda")
    h = dbf.mx4_gated_forward(gl, ul, t, act=act, save=save, h_dtype=torch.float32, **kw)
    ref = R.gate(act, g) * u
    tol = gate_tol(g) * (1 + np.abs(g)) * np.abs(u) + 1e-30
    assert np.all(np.abs(host(h) - ref) <= tol)
    # g and u are exact in fp32 here (the addends are whole numbers of the same unit), so their 8-bit form is too
    for a, v in zip(save, (g, u)):
        val, codes, byte = R.act8(v)
        assert np.array_equal(a.codes.cpu().numpy(), codes.reshape(T, -1).astype(np.uint8))
        assert np.array_equal(a.scales.cpu().numpy(), byte.T.astype(np.uint8))
    hb = dbf.mx4_gated_forward(gl, ul, t, act=act, h_dtype=torch.bfloat16, **kw)
    assert np.all(np.abs(host(hb) - ref) <= tol + 2.0 ** -8 * (np.abs(ref) + tol))


# ---- gradients
@pytest.mark.parametrize("T,M,N", [(1, 1, 1), (1, 32, 8), (2, 33, 5), (3, 64, 129), (16, 256, 128), (17, 1000, 130), (33, 2048, 257),
                                   (65, 512, 512), (77, 1000, 2200), (130, 288, 640), (257, 520, 64), (300, 95, 511), (1000, 768, 1536)])
@pytest.mark.parametrize("kind", ["f32", "bf16"])
def test_backward_is_exact(dbf, T, M, N, kind):
    """Whole-number gradients (up to 100, or up to 2^15 + 1 in fp32, which needs three pieces) and exact weights."""
    rng = np.random.default_rng(T * 7 + M * 3 + N)
    w = exact_operand(rng, N, M)
    dy = rng.integers(-100, 101, (T, N)).astype(np.float64)
    if kind == "f32" and N <= 512:   # terms below 2^15 * 24, sums below 2^24 units of 0.5 for a handful of them
        big = rng.random((T, N)) < 1.0 / N
        dy = np.where(big, rng.integers(-(2 ** 15) - 1, 2 ** 15 + 2, (T, N)), np.sign(dy))
    ref = dy @ w
    assert np.max(np.abs(dy) @ np.abs(w)) < 2 ** 23   # every partial sum is a multiple of 0.5 below 2^23
    t = torch.tensor(dy).to(DT[kind]).cuda()
    L = layer_of(dbf, w)
    assert np.array_equal(host(dbf.mx4_backward(L, t, dx_dtype=torch.float32)), ref)
    acc = dbf.mx4_backward(L, t, dx=torch.full((T, M), -3.0, device="cuda"), accumulate=True)
    assert np.array_equal(host(acc), ref - 3)
    b = dbf.mx4_backward(L, t, dx_dtype=torch.bfloat16)
    assert torch.equal(b.cpu(), torch.tensor(ref).float().to(torch.bfloat16))


@pytest.mark.parametrize("kind", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("T,M,N", [(1, 32, 8), (2, 33, 5), (70, 300, 1000), (129, 512, 264), (33, 95, 255)])
def test_gated_backward(dbf, T, M, N, act, kind):
    rng = np.random.default_rng(T + N)
    wg, wu = (rng.standard_normal((N, M)) / np.sqrt(N) for _ in range(2))
    g, u, dh = rng.standard_normal((T, N)) * 3, rng.standard_normal((T, N)), rng.standard_normal((T, N))
    g[0, 0], u[0, 0] = 0.0, 0.0
    saved = tuple(dbf.act8_save(torch.tensor(v, dtype=torch.float32).cuda()) for v in (g, u))
    t = torch.tensor(dh).to(DT[kind]).cuda()
    g, u = (R.act8(v.astype(np.float32))[0] for v in (g, u))
    dh = host(t)
    dg, du = dh * u * R.gate_slope(act, g), dh * R.gate(act, g)
    gl, ul = layer_of(dbf, wg), layer_of(dbf, wu)
    dx, gg, gu = dbf.mx4_gated_backward(gl, ul, t, saved, act=act, dx_dtype=torch.float32)
    tol = gate_tol(g) * (1 + np.abs(g)) * np.abs(dh)
    for got, ref, by in ((gg, dg, np.abs(u)), (gu, du, 1.0)):
        assert got.dtype == DT[kind]
        assert np.all(np.abs(host(got) - ref) <= tol * by + STEP[kind] * (np.abs(ref) + tol * by) + 1e-37)
    # dx is the gradient of what the block hands on
    gg, gu = host(gg), host(gu)
    wgq, wuq = R.mx4(wg.astype(np.float32))[0], R.mx4(wu.astype(np.float32))[0]
    ref, S = gg @ wgq + gu @ wuq, np.abs(gg) @ np.abs(wgq) + np.abs(gu) @ np.abs(wuq)
    pieces = 3 if kind == "f32" else 1
    assert np.all(np.abs(host(dx) - ref) <= 2 * pieces * N * 2.0 ** -23 * S + 1e-37)
    none, g2, u2 = dbf.mx4_gated_backward(gl, ul, t, saved, act=act, want_dx=False)
    assert none is None and np.array_equal(host(g2), gg) and np.array_equal(host(u2), gu)
