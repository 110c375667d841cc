"""The 4-bit layer's calls over the variants that their plans choose: one or two
accumulators, one or two sets of them, narrow and wide token tiles, one and several
tiles to a CTA pair, x quantised ahead of the few-token kernel, parts of the
gradient's contraction. Each shape says which variant it is there for; that the
plans still choose it is checked on the host, so that a change of their costs
cannot leave a variant untested.

Operands quantise to themselves and their sums are whole units below 2^24 (see
tests/test_gpu_mx4.py), so products are compared for equality with 64-bit ones.
The gate is compared relative to its value: see tests/test_gpu_mx4_gate.py for the
units, and 2 (2 + 1.173 |z|) of them instead of 4 for the exponential of results
rounded to bf16. The reciprocal of 1 + e^-z is 0 where it would be below 2^-126:
what is lost of s g u there is below 2^-126 (1 + 2^-12) |g u|, the sum being off by
as little."""
import ctypes

import numpy as np
import pytest
import torch

import mx_ref as R

gpu = pytest.mark.gpu
FORWARD, GATED, GATED_ADD, GATED_SAVE, BACKWARD, GATED_BACKWARD = range(6)
FEW, MANY, GRADIENT = range(3)
PAIRS = 74
UNIT = 2.0 ** -24 * (1 + 2.0 ** -12)
FLUSH = 2.0 ** -126 * (1 + 2.0 ** -12)
C2, K = 2 * np.sqrt(2 / np.pi), 0.044715

# (T, M, N): what the plan is on 148 SMs
MANY_PLAIN = {
    (40, 4100, 200): dict(accs=1, sets=1, wide=False, waves=1),
    (4100, 264, 520): dict(accs=1, sets=1, wide=True, waves=1),
    (3003, 520, 1352): dict(accs=1, sets=2, wide=False, waves=2),
    (3003, 64, 2101): dict(accs=1, sets=2, wide=True, waves=2),
    (3003, 2056, 1352): dict(accs=2, sets=1, wide=False, waves=1),
    (2100, 1100, 2099): dict(accs=2, sets=1, wide=True, waves=1),
    (2500, 2056, 6001): dict(accs=2, sets=1, wide=True, waves=2),
    (3003, 2056, 4104): dict(accs=2, sets=1, wide=True, waves=2),
    (1000, 64, 8201): dict(accs=2, sets=2, wide=False, waves=3),
    (4100, 300, 6000): dict(accs=2, sets=2, wide=False, waves=6),
}
MANY_GATED = {
    (33, 2056, 200): dict(sets=1, wide=False, waves=1),
    (70, 300, 261): dict(sets=1, wide=False, waves=1),
    (4100, 1100, 520): dict(sets=1, wide=True, waves=1),
    (3003, 1100, 1352): dict(sets=1, wide=False, waves=2),
    (2100, 264, 3000): dict(sets=1, wide=True, waves=2),
    (2100, 264, 3001): dict(sets=1, wide=True, waves=2),
    (701, 300, 8199): dict(sets=2, wide=False, waves=5),
    (4100, 64, 1000): dict(sets=2, wide=False, waves=2),
    (4100, 64, 3001): dict(sets=2, wide=False, waves=6),
}
FEW_PLAIN = {
    (1, 28672, 128): dict(pre=0, split=5, over=True),
    (17, 520, 130): dict(pre=0, split=3, over=False),
    (32, 4096, 384): dict(pre=1, split=4, over=False),
    (20, 3000, 130): dict(pre=1, split=4, over=False),
    (17, 3000, 8192): dict(pre=1, split=2, over=True),
    (9, 4096, 11008): dict(pre=1, split=3, over=True),
    (17, 28672, 130): dict(pre=1, split=8, over=True),
}
FEW_GATED = {
    (1, 16384, 128): dict(pre=0, split=5, over=True),
    (16, 520, 72): dict(pre=0, split=3, over=False),
    (13, 4100, 257): dict(pre=1, split=4, over=True),
    (16, 4096, 11008): dict(pre=1, split=3, over=True),
    (10, 2056, 8200): dict(pre=1, split=2, over=True),
    (4, 28672, 136): dict(pre=1, split=8, over=True),
}
GRADIENTS = {   # with an fp32 gradient
    (1, 64, 2056): dict(halves=1, parts=True, waves=1),
    (17, 8201, 200): dict(halves=1, parts=False, waves=1),
    (2050, 520, 4104): dict(halves=2, parts=True, waves=1),
    (2050, 2056, 520): dict(halves=2, parts=False, waves=1),
    (2050, 4100, 201): dict(halves=2, parts=False, waves=2),
    (6000, 2056, 64): dict(halves=2, parts=False, waves=2),
}


@pytest.fixture(scope="module")
def dbf():
    import double_binary_rank_b200 as m
    return m


def cut(dbf, call, shape, dy=None):
    T, M, N = shape
    out = (ctypes.c_int64 * 8)()
    assert dbf._lib.dbf_debug_mx4_cut(call, M, N, T, dbf.BF16 if dy is None else dy, 2 * PAIRS, out) == dbf.OK
    return list(out)


def test_shapes_reach_their_variants(dbf):
    for calls, shapes in (((FORWARD,), MANY_PLAIN), ((GATED, GATED_ADD, GATED_SAVE), MANY_GATED)):
        for shape, want in shapes.items():
            assert all(cut(dbf, call, shape)[0] == MANY for call in calls), shape
            c = cut(dbf, calls[0], shape)
            has = dict(accs=c[2], sets=c[3], wide=c[1] > 128, waves=-(-c[6] // PAIRS))
            assert {k: has[k] for k in want} == want, (shape, c)
    # what the gated plans choose for addends or copies, over all the shapes
    for call in (GATED_ADD, GATED_SAVE):
        seen = {(c[3], c[1] > 128, c[6] > PAIRS) for c in (cut(dbf, call, s) for s in MANY_GATED)}
        assert {(1, False, False), (1, True, False), (1, True, True), (2, False, True)} <= seen
    for call, shapes in ((FORWARD, FEW_PLAIN), (GATED, FEW_GATED)):
        for shape, want in shapes.items():
            c = cut(dbf, call, shape)
            assert c[0] == FEW and dict(pre=c[3], split=c[2], over=c[5] > c[4]) == want, (shape, c)
    for shape, want in GRADIENTS.items():
        for call in (BACKWARD, GATED_BACKWARD):
            c = cut(dbf, call, shape, dbf.F32)
            assert c[0] == GRADIENT and dict(halves=c[2], parts=c[3] > 1, waves=-(-c[6] // PAIRS)) == want, (shape, c)


# ---- operands
def codes(rng, rows, k, scales=3):
    """Values that quantise to themselves: every block holds a code of 4 or 6, times 1, 2 or 4."""
    t = torch.tensor(np.concatenate([R.E2M1, -R.E2M1])[rng.integers(0, 16, (rows, k))])
    t[:, ::32] = torch.tensor(rng.choice([4.0, -6.0], t[:, ::32].shape))
    s = torch.tensor(np.exp2(rng.integers(0, scales, (rows, -(-k // 32)))))
    return (t * s.repeat_interleave(32, dim=1)[:, :k]).cuda()


def quantized(dbf, w):
    return dbf.Mx4Layer.quantize(w.float())


@gpu
@pytest.mark.parametrize("T,M,N", list(MANY_PLAIN) + list(FEW_PLAIN))
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_forward(dbf, T, M, N, kind):
    rng = np.random.default_rng(T + M + N)
    w, x = codes(rng, N, M), codes(rng, T, M)
    L, x16 = quantized(dbf, w), x.to(kind)
    ref = x @ w.t()
    assert ref.abs().max().item() < 2 ** 21   # in units of 1/4: below 2^23
    assert torch.equal(dbf.mx4_forward(L, x16, y_dtype=torch.float32).double(), ref)
    assert torch.equal(dbf.mx4_forward(L, x16, y_dtype=torch.bfloat16), ref.to(torch.bfloat16))
    start = torch.randint(-50, 50, (T, N), device="cuda", generator=torch.Generator("cuda").manual_seed(T))
    for out in (torch.float32, torch.bfloat16):   # one rounding of the exact sum
        y = dbf.mx4_forward(L, x16, y=start.to(out), accumulate=True)
        assert torch.equal(y, (ref + start).to(out))


def gate_ref(act, g):
    z = g if act == "silu" else C2 * (g + K * g ** 3)
    return g / (1 + torch.exp(-z)), z.abs()


@gpu
@pytest.mark.parametrize("T,M,N", list(MANY_GATED) + list(FEW_GATED))
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("add", ["none", "both", "g", "u", "both f32", "g f32"])
def test_gated_forward(dbf, T, M, N, act, add):
    """Every kind of addends with both types of h, copies kept or not: h relative to the value, the copies exact."""
    rng = np.random.default_rng(T + M + N)
    down = 2.0 ** -np.ceil(np.log2(12 * np.sqrt(M)) - 1)   # products scaled by a power of two to the gate's range
    wg, wu, x = codes(rng, N, M, 2) * down, codes(rng, N, M, 2) * down, codes(rng, T, M, 2) * 0.25
    gl, ul, xb = quantized(dbf, wg), quantized(dbf, wu), x.to(torch.bfloat16)
    g, u = x @ wg.t(), x @ wu.t()
    kind = torch.float32 if add.endswith("f32") else torch.bfloat16
    made = [torch.randint(-8, 9, (T, N), device="cuda", generator=torch.Generator("cuda").manual_seed(i)).to(kind) for i in (1, 2)]
    kw = {}
    if add[0] in "bg":
        kw["g_add"], g = made[0], g + made[0].double()
    if add[0] in "bu":
        kw["u_add"], u = made[1], u + made[1].double()
    assert torch.equal(g.float().double(), g) and torch.equal(u.float().double(), u)
    value, z = gate_ref(act, g)
    ref = value * u
    moved = 7 * z if act == "gelu" else 0
    keep = [dbf.act8_save(v.float()) for v in (g, u)]
    for out in (torch.float32, torch.bfloat16):
        units = 9 + moved + (0 if out == torch.float32 else 2.35 * z)
        tol = units * UNIT * ref.abs() + FLUSH * (g * u).abs()
        if out == torch.bfloat16:
            tol = tol + 2.0 ** -8 * (ref.abs() + tol)
        saved = dbf.Act8.empty(T, N, "cuda"), dbf.Act8.empty(T, N, "cuda")
        for a in saved:
            a.codes.fill_(0x5A)
            a.scales.fill_(0x5A)
        plain = dbf.mx4_gated_forward(gl, ul, xb, act=act, h_dtype=out, **kw)
        kept = dbf.mx4_gated_forward(gl, ul, xb, act=act, h_dtype=out, save=saved, **kw)
        for h in (plain, kept):
            assert ((h.double() - ref).abs() <= tol).all().item()
        for a, b in zip(saved, keep):
            assert torch.equal(a.codes, b.codes) and torch.equal(a.scales, b.scales)


@gpu
@pytest.mark.parametrize("act,most", [("silu", 72.0), ("gelu", 8.5)])
@pytest.mark.parametrize("T,N", [(3, 96), (16, 97), (70, 520), (300, 1352), (70, 261)])
def test_small_values_of_a_bf16_gate(dbf, T, N, act, most):
    """g from its addend, down to where the value is 1e-29: relative to the value, also with copies."""
    g_add = torch.empty(T, N, device="cuda").uniform_(-most, most, generator=torch.Generator("cuda").manual_seed(N)).to(torch.bfloat16)
    u_add = torch.ones(T, N, device="cuda", dtype=torch.bfloat16)
    Z = dbf.Mx4Layer.quantize(torch.zeros(N, 64, device="cuda"))
    x = torch.ones(T, 64, device="cuda", dtype=torch.bfloat16)
    ref, z = gate_ref(act, g_add.double())
    tol = (9 + 2.35 * z + (7 * z if act == "gelu" else 0)) * UNIT * ref.abs()
    tol = tol + 2.0 ** -8 * (ref.abs() + tol)
    for save in (None, (dbf.Act8.empty(T, N, "cuda"), dbf.Act8.empty(T, N, "cuda"))):
        h = dbf.mx4_gated_forward(Z, Z, x, act=act, g_add=g_add, u_add=u_add, h_dtype=torch.bfloat16, save=save)
        assert ((h.double() - ref).abs() <= tol).all().item()
    # du = dh act(g) from the same g as 8 bits hold it
    g8, dh = dbf.act8_load(save[0], dtype=torch.float32).double(), torch.ones(T, N, device="cuda", dtype=torch.bfloat16)
    ref, z = gate_ref(act, g8)
    tol = (9 + 2.35 * z + (7 * z if act == "gelu" else 0)) * UNIT * ref.abs()
    du = dbf.mx4_gated_backward(Z, Z, dh, save, act=act, want_dx=False)[2]
    assert ((du.double() - ref).abs() <= tol + 2.0 ** -8 * (ref.abs() + tol)).all().item()


# ---- gradients
@gpu
@pytest.mark.parametrize("T,M,N", list(GRADIENTS))
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_backward(dbf, T, M, N, kind):
    rng = np.random.default_rng(T + M + N)
    w = codes(rng, N, M)
    dy = torch.randint(-100, 101, (T, N), device="cuda", generator=torch.Generator("cuda").manual_seed(N)).double()
    L, ref = quantized(dbf, w), dy @ w
    assert (dy.abs() @ w.abs()).max().item() < 2 ** 23   # units of 1/2, any order
    start = torch.randint(-50, 50, (T, M), device="cuda", generator=torch.Generator("cuda").manual_seed(T))
    for out in (torch.float32, torch.bfloat16):
        assert torch.equal(dbf.mx4_backward(L, dy.to(kind), dx_dtype=out), ref.to(out))
        dx = dbf.mx4_backward(L, dy.to(kind), dx=start.to(out), accumulate=True)
        assert torch.equal(dx, (ref + start).to(out))


@gpu
@pytest.mark.parametrize("T,M,N", [s for s in GRADIENTS if s != (17, 8201, 200)] + [(33, 95, 255)])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gated_backward(dbf, T, M, N, kind, act):
    """dx of what dg and du hold, 64 bits, each of 2 N terms off by a unit of fp32 at most (three pieces of fp32 ones:
    six times), and added to what is there in one rounding more."""
    rng = np.random.default_rng(T + M + N)
    gl, ul = (quantized(dbf, codes(rng, N, M)) for _ in range(2))
    r = torch.Generator("cuda").manual_seed(T)
    saved = tuple(dbf.act8_save(torch.randn(T, N, device="cuda", generator=r) * 3) for _ in range(2))
    dh = torch.randn(T, N, device="cuda", generator=r).to(kind)
    dx, dg, du = dbf.mx4_gated_backward(gl, ul, dh, saved, act=act, dx_dtype=torch.float32)
    wg, wu, dg64, du64 = gl.dequantize(torch.float32).double(), ul.dequantize(torch.float32).double(), dg.double(), du.double()
    ref = dg64 @ wg + du64 @ wu
    S = dg64.abs() @ wg.abs() + du64.abs() @ wu.abs()
    assert ((dx.double() - ref).abs() <= (6 if kind == torch.float32 else 2) * N * 2.0 ** -23 * S + 2.0 ** -140).all().item()
    start = torch.randn(T, M, device="cuda", generator=r)
    for out in (torch.float32, torch.bfloat16):
        first = start.to(out)
        got = dbf.mx4_gated_backward(gl, ul, dh, saved, act=act, dx=first.clone(), accumulate=True)
        assert torch.equal(got[0], (dx + first.float()).to(out))
        assert torch.equal(got[1], dg) and torch.equal(got[2], du)


# ---- order of work
@gpu
@pytest.mark.parametrize("T,M,N,gated", [(20, 3000, 130, False), (32, 4096, 384, False), (13, 4100, 257, True)])
def test_few_tokens_quantised_ahead_follow_what_was_enqueued(dbf, T, M, N, gated):
    """x and the weights are written just before the call, without static_weights; the workspace is the same each time."""
    rng = np.random.default_rng(T)
    ws_ = [codes(rng, N, M) / 16 for _ in range(2)]
    xs = [codes(rng, T, M).to(torch.bfloat16) for _ in range(2)]
    src = [dbf.mx4_quantize(w.float()) for w in ws_]
    assert cut(dbf, GATED if gated else FORWARD, (T, M, N))[3] == 1
    ws = dbf.alloc_workspace(dbf.mx4_workspace_bytes(dbf.Mx4Layer(M, N, *src[0]), T), "cuda")
    call = (lambda L, x: dbf.mx4_gated_forward(L, L, x, ws=ws, h_dtype=torch.float32)) if gated else \
           (lambda L, x: dbf.mx4_forward(L, x, ws=ws, y_dtype=torch.float32))
    want = [[call(dbf.Mx4Layer(M, N, *s), x).clone() for x in xs] for s in src]
    if not gated:
        assert all(torch.equal(want[i][j].double(), xs[j].double() @ ws_[i].t()) for i in range(2) for j in range(2))
    torch.cuda.synchronize()
    L, cur, outs = dbf.Mx4Layer(M, N, src[0][0].clone(), src[0][1].clone()), torch.empty_like(xs[0]), []
    for i in range(24):
        L.codes.copy_(src[i % 2][0])
        L.scales.copy_(src[i % 2][1])
        cur.copy_(xs[i // 2 % 2])
        outs.append(call(L, cur))
    for i, y in enumerate(outs):
        assert torch.equal(y, want[i % 2][i // 2 % 2])
    assert dbf.workspace_status(ws) == 0


@gpu
@pytest.mark.parametrize("T,M,N", [(3, 64, 96), (16, 520, 73), (70, 300, 264), (70, 300, 261), (2100, 264, 3000), (4100, 64, 1000)])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kept", [False, True])
def test_h_in_the_place_of_an_addend(dbf, T, M, N, kind, kept):
    rng = np.random.default_rng(T)
    gl, ul = (quantized(dbf, codes(rng, N, M) / 64) for _ in range(2))
    x = codes(rng, T, M).to(torch.bfloat16)
    add = [torch.randn(T, N, device="cuda", generator=torch.Generator("cuda").manual_seed(i)).to(kind) for i in (1, 2)]
    save = (lambda: (dbf.Act8.empty(T, N, "cuda"), dbf.Act8.empty(T, N, "cuda"))) if kept else (lambda: None)
    first = save()
    want = dbf.mx4_gated_forward(gl, ul, x, g_add=add[0], u_add=add[1], h_dtype=kind, save=first)
    for i in range(2):
        a = [t.clone() for t in add]
        again = save()
        h = dbf.mx4_gated_forward(gl, ul, x, g_add=a[0], u_add=a[1], h=a[i], save=again)
        assert h is a[i] and torch.equal(h, want) and torch.equal(a[1 - i], add[1 - i])
        assert not kept or all(torch.equal(p.codes, q.codes) and torch.equal(p.scales, q.scales) for p, q in zip(first, again))


@gpu
@pytest.mark.parametrize("T,N", [(1, 64), (33, 95), (600, 520), (2050, 1032)])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_dx_in_the_place_of_dh(dbf, T, N, kind):
    """dh is read before dx is written, also where the contraction is in parts and where dx is added to what dh was."""
    rng = np.random.default_rng(T)
    gl, ul = (quantized(dbf, codes(rng, N, N)) for _ in range(2))
    r = torch.Generator("cuda").manual_seed(T)
    saved = tuple(dbf.act8_save(torch.randn(T, N, device="cuda", generator=r)) for _ in range(2))
    dh = torch.randn(T, N, device="cuda", generator=r).to(kind)
    for accumulate in (False, True):
        want = dbf.mx4_gated_backward(gl, ul, dh, saved, dx=dh.clone(), accumulate=accumulate)
        here = dh.clone()
        got = dbf.mx4_gated_backward(gl, ul, here, saved, dx=here, accumulate=accumulate)
        assert got[0] is here and all(torch.equal(a, b) for a, b in zip(got, want))
