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


@pytest.mark.parametrize("rows,k", [(3, 33), (5, 31), (7, 250), (9, 255), (66, 257), (130, 511), (37, 1371), (65, 2050)])
@pytest.mark.parametrize("kind", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("first", [0, 1, 3])
def test_rows_that_start_anywhere(dbf, rows, k, kind, first):
    """Rows that are no whole vectors, in tensors that start anywhere: the shifted loads and stores of all formats, and
    nothing in front of or behind the tensor is touched."""
    rng = np.random.default_rng(rows * 77 + k)
    x = rng.standard_normal((rows, k)) * np.exp2(rng.integers(-8, 6, (rows, 1)))

    def place(fill=None):
        buf = torch.full((first + rows * k + 16,), -7.0, device="cuda", dtype=DT[kind])
        view = buf[first:first + rows * k].view(rows, k)
        if fill is not None:
            view.copy_(torch.tensor(fill).to(DT[kind]))
        return buf, view

    buf, t = place(x)
    val4, codes, byte = R.mx4(host(t))
    packed, scales = R.pack4(codes, byte)
    gc, gs = dbf.mx4_quantize(t)
    assert torch.equal(gc.cpu(), torch.from_numpy(packed)) and torch.equal(gs.cpu(), torch.from_numpy(scales))
    val8, codes8, byte8 = R.act8(host(t))
    a = dbf.act8_save(t)
    assert np.array_equal(a.codes.cpu().numpy(), codes8.reshape(rows, -1).astype(np.uint8))
    assert np.array_equal(a.scales.cpu().numpy(), byte8.T.astype(np.uint8))
    for load, val in ((lambda o: dbf.mx4_dequantize(gc, gs, rows, k, out=o), val4), (lambda o: dbf.act8_load(a, out=o), val8)):
        buf, o = place()
        load(o)
        want = val.astype(np.float16).astype(np.float64) if kind == "f16" else val
        assert np.array_equal(host(o), want)
        assert (buf[:first] == -7.0).all().item() and (buf[first + rows * k:] == -7.0).all().item()


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
    """Whole-number gradients (up to 100, or up to 2^15 + 1 in fp32, which needs three pieces) and exact weights; a bf16
    dx of an fp32 gradient within its tolerance."""
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
    if kind == "bf16":
        assert torch.equal(b.cpu(), torch.tensor(ref).float().to(torch.bfloat16))
    else:   # two pieces of an fp32 gradient: each value off by at most 2^-16 of itself
        tol = (2.0 ** -16 + N * 2.0 ** -23) * (np.abs(dy) @ np.abs(w))
        assert np.all(np.abs(host(b) - ref) <= tol + STEP["bf16"] * (np.abs(ref) + tol))


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
    low = host(dbf.mx4_gated_backward(gl, ul, t, saved, act=act, dx_dtype=torch.bfloat16)[0])
    tol = (2.0 ** -16 + 4 * N * 2.0 ** -23) * S + 1e-37
    assert np.all(np.abs(low - ref) <= tol + STEP["bf16"] * (np.abs(ref) + tol))
    none, g2, u2 = dbf.mx4_gated_backward(gl, ul, t, saved, act=act, want_dx=False)
    assert none is None and np.array_equal(host(g2), gg) and np.array_equal(host(u2), gu)


# ---- values that are not finite, and the limits of the format
@pytest.mark.parametrize("T,M,N", [(3, 100, 40), (70, 300, 260), (90, 520, 130)])
def test_not_finite_values_stay_where_they_are(dbf, T, M, N):
    """A NaN or infinity in x spoils its token alone, one in W its output column alone (and, in the gradient, the 32
    columns of its block)."""
    rng = np.random.default_rng(5)
    w, x = exact_operand(rng, N, M), exact_operand(rng, T, M)
    ref = x @ w.T
    w[N // 2, 33], x[T - 1, 5], x[1, M - 1] = np.nan, np.inf, np.nan
    L = layer_of(dbf, w)
    y = host(dbf.mx4_forward(L, torch.tensor(x).to(torch.bfloat16).cuda(), y_dtype=torch.float32))
    bad = np.zeros((T, N), bool)
    bad[:, N // 2] = bad[T - 1] = bad[1] = True
    assert np.isnan(y[bad]).all() and np.array_equal(y[~bad], ref[~bad])
    gl = layer_of(dbf, np.nan_to_num(w, nan=4.0))
    saved = dbf.Act8.empty(T, N, "cuda"), dbf.Act8.empty(T, N, "cuda")
    h = host(dbf.mx4_gated_forward(L, gl, torch.tensor(x).to(torch.bfloat16).cuda(), save=saved, h_dtype=torch.float32))
    assert np.array_equal(np.isnan(h), bad)
    # in 8 bits the whole block of 32 is spoiled
    blocks = np.zeros((T, -(-N // 32) * 32), bool)
    blocks[:, :N] = bad
    spread = np.repeat(blocks.reshape(T, -1, 32).any(2), 32, axis=1)[:, :N]
    assert np.array_equal(np.isnan(host(dbf.act8_load(saved[0], dtype=torch.float32))), spread)
    dy = torch.ones(T, N, device="cuda", dtype=torch.bfloat16)
    dx = host(dbf.mx4_backward(L, dy, dx_dtype=torch.float32))
    col = np.zeros(M, bool)
    col[32:64] = True
    assert np.isnan(dx[:, col]).all() and np.isfinite(dx[:, ~col]).all()
    dyn = dy.clone()
    dyn[0, N - 1] = float("inf")
    for t in (dyn, dyn.float()):
        dx = host(dbf.mx4_backward(gl, t, dx_dtype=torch.float32))
        assert not np.isfinite(dx[0]).any() and np.isfinite(dx[1:]).all()


def test_every_code_and_scale(dbf):
    """All 16 codes at every scale that the bf16 expansion of the gradient and fp32 can hold, one term per output."""
    codes = np.arange(16, dtype=np.uint8)
    table = np.concatenate([R.E2M1, -R.E2M1])
    bytes_ = np.arange(0, 253)
    N, M = len(bytes_), 32
    packed = torch.from_numpy(np.tile((codes[0::2] | codes[1::2] << 4).astype(np.uint8), (N, 2))).cuda()
    scales = np.zeros((2, 1, 32, 4, 4), np.uint8)
    for r, b in enumerate(bytes_):
        scales[r // 128, 0, r % 32, r % 128 // 32, 0] = b
    L = dbf.Mx4Layer(M, N, packed, torch.from_numpy(scales).cuda())
    value = np.tile(table, 2)[None, :] * np.exp2(bytes_[:, None] - 127.0)
    assert np.array_equal(host(L.dequantize(torch.float32)), value.astype(np.float32).astype(np.float64))
    dy = np.eye(N)
    dx = host(dbf.mx4_backward(L, torch.tensor(dy).to(torch.bfloat16).cuda(), dx_dtype=torch.float32))
    # products below the smallest normal fp32 may be flushed
    ok = (np.abs(value) >= 2.0 ** -126) | (value == 0)
    assert np.array_equal(dx[ok], value[ok]) and np.all(np.abs(dx[~ok]) <= np.abs(value[~ok]))


# ---- how calls may be made
def test_empty_batches(dbf):
    L = layer_of(dbf, np.ones((64, 32)))
    x = torch.empty(0, 32, device="cuda")
    assert dbf.mx4_forward(L, x).shape == (0, 64)
    assert dbf.mx4_backward(L, torch.empty(0, 64, device="cuda")).shape == (0, 32)
    saved = dbf.Act8.empty(0, 64, "cuda"), dbf.Act8.empty(0, 64, "cuda")
    assert dbf.mx4_gated_forward(L, L, x, save=saved).shape == (0, 64)
    dx, dg, du = dbf.mx4_gated_backward(L, L, torch.empty(0, 64, device="cuda"), saved)
    assert dx.shape == (0, 32) and dg.shape == du.shape == (0, 64)
    assert dbf.act8_load(dbf.act8_save(x)).shape == (0, 32)


def test_rows_behind_the_last_token_are_left(dbf):
    rng = np.random.default_rng(3)
    for T, M, N in ((5, 64, 72), (70, 64, 520), (230, 256, 264)):
        L = layer_of(dbf, exact_operand(rng, N, M))
        big = torch.full((T + 40, N), 7.0, device="cuda", dtype=torch.bfloat16)
        x = torch.tensor(exact_operand(rng, T, M)).to(torch.bfloat16).cuda()
        dbf.mx4_forward(L, x, y=big[:T])
        assert (big[T:] == 7).all() and not (big[:T] == 7).all()
        bx = torch.full((T + 40, M), 7.0, device="cuda", dtype=torch.bfloat16)
        dbf.mx4_backward(L, torch.ones(T, N, device="cuda", dtype=torch.bfloat16), dx=bx[:T])
        assert (bx[T:] == 7).all()


@pytest.mark.parametrize("T", [1, 24, 200])
def test_graph_replays_on_new_inputs(dbf, T):
    """Forward, gated forward and backward captured once and replayed on other inputs, two graphs on one workspace."""
    M, N = 520, 1000
    rng = np.random.default_rng(T)
    wg, wu = exact_operand(rng, N, M), exact_operand(rng, N, M)
    gl, ul = layer_of(dbf, wg), layer_of(dbf, wu)
    x = torch.zeros(T, M, device="cuda", dtype=torch.bfloat16)
    y = torch.zeros(T, N, device="cuda")
    dx = torch.zeros(T, M, device="cuda")
    ws = dbf.alloc_workspace(max(dbf.mx4_workspace_bytes(gl, T), dbf.mx4_gated_workspace_bytes(gl, ul, T),
                                 dbf.mx4_backward_workspace_bytes(gl, T, torch.float32)), "cuda")
    h = torch.zeros(T, N, device="cuda")
    graphs = []
    s = torch.cuda.Stream()
    for f in (lambda: (dbf.mx4_forward(gl, x, y=y, ws=ws), dbf.mx4_backward(gl, y, dx=dx, ws=ws)),
              lambda: dbf.mx4_gated_forward(gl, ul, x, h=h, ws=ws)):
        with torch.cuda.stream(s):
            f()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            f()
        graphs.append(g)
    for seed in (1, 2, 3):
        xv = exact_operand(np.random.default_rng(seed), T, M)
        x.copy_(torch.tensor(xv).to(torch.bfloat16))
        graphs[1].replay()
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        ref = xv @ wg.T
        assert np.array_equal(host(y), ref)
        eager = dbf.mx4_gated_forward(gl, ul, x, h_dtype=torch.float32)
        assert torch.equal(h, eager)
        assert torch.equal(dx, dbf.mx4_backward(gl, y, dx_dtype=torch.float32))
    assert dbf.workspace_status(ws) == 0


def test_calls_follow_what_was_enqueued_before(dbf):
    """x, and without static_weights the weights too, may be written by the work just before the call; y may be read
    by it. Long chains of launches on one stream, each depending on the last."""
    M = N = 512
    rng = np.random.default_rng(9)
    ws_ = [exact_operand(rng, N, M) / 16 for _ in range(2)]
    for T in (1, 20, 90):
        src = [dbf.mx4_quantize(torch.tensor(w, dtype=torch.float32).cuda()) for w in ws_]
        L = dbf.Mx4Layer(M, N, src[0][0].clone(), src[0][1].clone())
        x = torch.tensor(exact_operand(rng, T, M)).to(torch.bfloat16).cuda()
        want = []
        for w in src:
            want.append([dbf.mx4_forward(dbf.Mx4Layer(M, N, *w), x.clone(), y_dtype=torch.float32),
                         dbf.mx4_backward(dbf.Mx4Layer(M, N, *w), x.clone(), dx_dtype=torch.float32)])
        torch.cuda.synchronize()
        y, dx, cur = torch.empty(T, N, device="cuda"), torch.empty(T, M, device="cuda"), torch.empty_like(x)
        outs = []
        for i in range(24):
            L.codes.copy_(src[i % 2][0])
            L.scales.copy_(src[i % 2][1])
            cur.zero_()
            cur.copy_(x)
            dbf.mx4_forward(L, cur, y=y)
            dbf.mx4_backward(L, cur, dx=dx)
            outs.append((y.clone(), dx.clone()))
            y.fill_(-1.0)
        for i, (a, b) in enumerate(outs):
            assert torch.equal(a, want[i % 2][0]) and torch.equal(b, want[i % 2][1])


def test_two_streams_at_once(dbf):
    """Calls on two streams with workspaces of their own give what they give alone."""
    rng = np.random.default_rng(4)
    jobs = []
    for T, M, N in ((1, 2048, 4096), (33, 1000, 3000), (300, 1024, 2048), (2, 4096, 11008)):
        L = layer_of(dbf, exact_operand(rng, N, M))
        x = torch.tensor(exact_operand(rng, T, M)).to(torch.bfloat16).cuda()
        jobs.append((L, x, dbf.mx4_forward(L, x, y_dtype=torch.float32), dbf.mx4_gated_forward(L, L, x)))
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    wss = [dbf.alloc_workspace(max(dbf.mx4_gated_workspace_bytes(j[0], j[0], j[1].shape[0]) for j in jobs), "cuda") for _ in streams]
    torch.cuda.synchronize()
    got = []
    for rep in range(6):
        for k, st in enumerate(streams):
            L, x, ref, href = jobs[(rep + k) % len(jobs)]
            y, h = torch.empty_like(ref), torch.empty_like(href)
            st.wait_stream(torch.cuda.current_stream())
            dbf.mx4_forward(L, x, y=y, ws=wss[k], static_weights=True, stream=st)
            dbf.mx4_gated_forward(L, L, x, h=h, ws=wss[k], static_weights=True, stream=st)
            got.append((y, ref, h, href))
    torch.cuda.synchronize()
    for y, ref, h, href in got:
        assert torch.equal(y, ref) and torch.equal(h, href)
    assert all(dbf.workspace_status(w) == 0 for w in wss)


def test_base_and_adapter_kernels_on_two_streams(dbf):
    """The base's kernels on one stream while the adapter's run on another (both kinds hold tensor memory, in
    clusters): the same results as alone. The adapter's fp32 sums may meet in another order: a bf16 step."""
    from gpu_util import dev_layer, random_layer
    rng = np.random.default_rng(12)
    T, M, N, r = 600, 1024, 2048, 512
    L = layer_of(dbf, exact_operand(rng, N, M))
    ad = dev_layer(random_layer(rng, M, N, r, 1))
    x = torch.tensor(exact_operand(rng, T, M)).to(torch.bfloat16).cuda()
    dy = torch.tensor(rng.integers(-3, 4, (T, N)).astype(np.float64)).to(torch.bfloat16).cuda()
    wss = [dbf.alloc_workspace(n, "cuda") for n in (max(dbf.mx4_gated_workspace_bytes(L, L, T),
                                                        dbf.mx4_backward_workspace_bytes(L, T, torch.bfloat16)),
                                                    max(dbf.workspace_bytes(ad, t) for t in (1, T)))]
    base = (lambda st: dbf.mx4_forward(L, x[:1], ws=wss[0], stream=st), lambda st: dbf.mx4_gated_forward(L, L, x, ws=wss[0], stream=st),
            lambda st: dbf.mx4_backward(L, dy, ws=wss[0], stream=st), lambda st: dbf.mx4_forward(L, x[:20], ws=wss[0], stream=st))
    other = (lambda st: dbf.forward(ad, x, ws=wss[1], stream=st), lambda st: dbf.forward(ad, x[:1], ws=wss[1], stream=st))
    own = torch.cuda.current_stream()
    want = [[f(own) for f in fs] for fs in (base, other)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        got.append([[f(st) for f in fs] for fs, st in zip((base, other), streams)])
    torch.cuda.synchronize()
    for b, o in got:
        assert all(torch.equal(a, w) for a, w in zip(b, want[0]))
        assert all(((a.float() - w.float()).norm() <= 2.0 ** -7 * w.float().norm()).item() for a, w in zip(o, want[1]))
    assert all(dbf.workspace_status(w) == 0 for w in wss)


def test_an_explicit_stream_orders_the_copies_and_workspaces_too(dbf):
    """The input is written late on the stream that is passed: the contiguous copy of a
    strided input, the new outputs and the workspace's header belong on it as well."""
    rng = np.random.default_rng(6)
    T, M, N = 37, 96, 160
    L = layer_of(dbf, exact_operand(rng, N, M))
    late = torch.tensor(exact_operand(rng, T, M)).float().cuda()
    want = dbf.mx4_quantize(late), dbf.act8_save(late), dbf.mx4_forward(L, late), dbf.mx4_gated_forward(L, L, late)
    x, wide = torch.zeros(T, M, device="cuda"), torch.zeros(T, 2 * M, device="cuda")
    busy = torch.ones(1 << 27, device="cuda")
    st, own = torch.cuda.Stream(), torch.cuda.current_stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(st):
        for _ in range(40):   # several milliseconds
            busy.mul_(1.0)
        x.copy_(late)
        wide[:, ::2].copy_(late)
    got = (dbf.mx4_quantize(wide[:, ::2], stream=st), dbf.act8_save(wide[:, ::2], stream=st), dbf.mx4_forward(L, x, stream=st),
           dbf.mx4_gated_forward(L, L, x, stream=st))
    assert torch.cuda.current_stream() == own
    st.synchronize()
    assert torch.equal(got[0][0], want[0][0]) and torch.equal(got[0][1], want[0][1])
    assert torch.equal(got[1].codes, want[1].codes) and torch.equal(got[1].scales, want[1].scales)
    assert torch.equal(got[2], want[2]) and torch.equal(got[3], want[3])


def test_offsets_past_32_bits(dbf):
    """y, x and an 8-bit activation of more than 2^31 elements (and more than 2^32 bytes)."""
    T, M, N = 270_001, 32, 8192
    rng = np.random.default_rng(2)
    w, row = exact_operand(rng, N, M), exact_operand(rng, 5, M)
    L = layer_of(dbf, w)
    pick = [0, 1, 131_071, 262_143, 262_144, 265_000, 269_999, 270_000]
    x = torch.tensor(row).to(torch.bfloat16).cuda()[torch.arange(T, device="cuda") % 5].contiguous()
    y = dbf.mx4_forward(L, x)
    ref = torch.tensor(row @ w.T).float().to(torch.bfloat16)
    for t in pick:
        assert torch.equal(y[t].cpu(), ref[t % 5])
    a = dbf.act8_save(y)
    codes, scales = dbf.mx4_quantize(y)
    small = y[pick].contiguous()
    back, want = dbf.act8_load(a), dbf.act8_load(dbf.act8_save(small))
    assert torch.equal(back[pick], want)
    del back
    want4 = dbf.mx4_dequantize(*dbf.mx4_quantize(small), len(pick), N)
    assert torch.equal(dbf.mx4_dequantize(codes, scales, T, N)[pick], want4)
    del codes, scales, a
    dx = dbf.mx4_backward(L, y, dx_dtype=torch.float32)
    for t in pick:
        assert torch.equal(dx[t], dx[t % 5])
    # these sums pass 2^24 units (9.4e6 in units of 0.5 or less), so they are not exact
    y5 = host(y[:5])
    assert np.all(np.abs(host(dx[:5]) - y5 @ w) <= N * 2.0 ** -23 * (np.abs(y5) @ np.abs(w)))


def test_refusals(dbf):
    L = layer_of(dbf, np.ones((64, 96)))
    x = torch.ones(4, 96, device="cuda")
    for bad in (x[:, :64], x.t(), x.half(), x.double(), x.cpu(), torch.ones(4, 192, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            dbf.mx4_forward(L, bad)
    with pytest.raises(ValueError):
        dbf.mx4_forward(L, x, y=torch.empty(4, 65, device="cuda"))
    with pytest.raises(ValueError):
        dbf.mx4_forward(L, x, accumulate=True)
    with pytest.raises(ValueError):
        dbf.Mx4Layer(96, 64, L.codes[:, :32], L.scales)
    with pytest.raises(ValueError):
        dbf.Mx4Layer(96, 64, L.codes, L.scales.view(-1))
    with pytest.raises(dbf.DbfError) as e:
        dbf.mx4_forward(L, x, ws=torch.zeros(128, dtype=torch.uint8, device="cuda"))
    assert e.value.status == dbf.ERR_WORKSPACE
    with pytest.raises(dbf.DbfError) as e:   # rows that start off a 16-byte boundary
        dbf.mx4_forward(L, torch.ones(4 * 96 + 1, device="cuda")[1:].view(4, 96))
    assert e.value.status == dbf.ERR_ALIGNMENT
    with pytest.raises(ValueError):
        dbf.mx4_gated_forward(L, L, x, g_add=torch.ones(4, 63, device="cuda"))
    with pytest.raises(KeyError):
        dbf.mx4_gated_forward(L, L, x, act="relu")
    with pytest.raises(ValueError):
        dbf.mx4_gated_forward(L, L, x, save=(dbf.Act8.empty(4, 64, "cuda"), dbf.Act8.empty(5, 64, "cuda")))
    with pytest.raises(ValueError):
        dbf.act8_save(x, out=dbf.Act8.empty(4, 95, "cuda"))


# ---- together: an adapter on a 4-bit gated block, trained with 8-bit checkpoints
def test_adapter_training_step_on_a_4bit_block(dbf):
    """The step of one block: adapter branches from dbf_forward are added inside the gated kernel, x, g and u are kept
    in 8 bits, dg and du feed dbf_backward of both adapters, dx collects the base's and the adapters' parts. Against
    the same step in 64 bits."""
    import dbf_synth as S
    import oracle
    from gpu_util import dev_layer, random_layer, rel_err
    T, M, N, r = 200, 256, 384, 128
    rng = np.random.default_rng(11)
    wg, wu = (rng.standard_normal((N, M)) / np.sqrt(M) for _ in range(2))
    gl, ul = layer_of(dbf, wg), layer_of(dbf, wu)
    ad = [random_layer(rng, M, N, r, 1) for _ in range(2)]
    for L in ad:   # a branch as large as the base's output
        L.alpha[:] = S.to_f16_bits(np.full(N, 2.0 ** -7))
    dev = [dev_layer(L) for L in ad]
    x = torch.tensor(rng.standard_normal((T, M))).to(torch.bfloat16).cuda()
    dh = torch.tensor(rng.standard_normal((T, N))).to(torch.bfloat16).cuda()
    # forward
    add = [dbf.forward(d, x) for d in dev]
    saved = dbf.Act8.empty(T, N, "cuda"), dbf.Act8.empty(T, N, "cuda")
    h = dbf.mx4_gated_forward(gl, ul, x, g_add=add[0], u_add=add[1], save=saved)
    x8 = dbf.act8_save(x)
    # backward
    dx, dg, du = dbf.mx4_gated_backward(gl, ul, dh, saved, dx_dtype=torch.float32)
    xr = dbf.act8_load(x8)
    grads = [dbf.backward(d, xr, dd) for d, dd in zip(dev, (dg, du))]
    total = dx + grads[0].dx + grads[1].dx
    # 64 bits: every stored value rounded where the step rounds it
    xq = R.mx4(host(x))[0]
    g, u = (xq @ R.mx4(w.astype(np.float32))[0].T + host(a) for w, a in zip((wg, wu), add))
    tol = 2.0 ** -8
    assert np.all(np.abs(host(h) - R.gate("silu", g) * u) <= (tol + 2.0 ** -12) * np.abs(R.gate("silu", g) * u) + 1e-5)
    # g and u may round to the neighbouring 8-bit code where fp32 and fp64 sums lie on two sides of a border
    g8, u8 = (host(dbf.act8_load(a, dtype=torch.float32)) for a in saved)
    for got, want in ((g8, g), (u8, u)):
        val, _, byte = R.act8(want.astype(np.float32))
        step = np.exp2(byte.repeat(32, axis=1)[:, :N] - 127.0) * 2.0 ** -9 + np.abs(want) / 8
        assert np.all(np.abs(got - val) <= step) and np.mean(got != val) < 1e-3
    h64 = host(dh)
    rdg, rdu = h64 * u8 * R.gate_slope("silu", g8), h64 * R.gate("silu", g8)
    for got, want in ((dg, rdg), (du, rdu)):
        assert np.all(np.abs(host(got) - want) <= (tol + 2.0 ** -12) * np.abs(want) + 1e-6)
    xr64 = R.act8(host(x))[0]
    assert np.array_equal(host(xr), xr64)
    base = host(dg) @ R.mx4(wg.astype(np.float32))[0] + host(du) @ R.mx4(wu.astype(np.float32))[0]
    refs = [oracle.backward(L, xr64.astype(np.float32), host(d).astype(np.float32)) for L, d in zip(ad, (dg, du))]
    assert rel_err(host(total), base + refs[0].dx + refs[1].dx) < 2e-3   # the adapters' tolerance
