"""The gate of the 4-bit block where its result is fp32: relative to the value,
also where it is small.

Tolerances, in units of 2^-24 (half a step of fp32). expf is off by at most 2
steps, 4 units, the reciprocal by one, 2 units; 1 + e, the product with g and that
with u are a rounding each: SiLU's sigmoid 7 units, its value 9. GELU's argument z = 2c (g +
k g^3) has seven roundings, the two constants' among them, that move e^-z by |z|
each: 7 |z| units more. Slopes, with s the sigmoid, E its units and 1 - s off by E s
+ (1 - s): SiLU s (1 + a), a = g (1 - s), off by s (E |g| s + 2 |g| (1 - s) +
(E + 2) |1 + a|); GELU s + f d, d = s (1 - s), f = g 2c (1 + 3 k g^2) of six
roundings: s E + |f| (d (E + 8) + s (E s + 1)) + |s + f d|. Products with dh and u
add a rounding each."""
import numpy as np
import pytest
import torch

import mx_ref as R

pytestmark = pytest.mark.gpu
UNIT = 2.0 ** -24 * (1 + 2.0 ** -12)   # products of the units above
C2, K = 2 * np.sqrt(2 / np.pi), 0.044715


@pytest.fixture(scope="module")
def dbf():
    import double_binary_rank_b200 as m
    return m


def host(t):
    return t.double().cpu().numpy()


def sigmoid_units(act, g):
    return 7 + (7 * np.abs(C2 * (g + K * g ** 3)) if act == "gelu" else 0)


def value_units(act, g):
    return sigmoid_units(act, g) + 2


def slope_units(act, g):
    E = sigmoid_units(act, g)
    z = g if act == "silu" else C2 * (g + K * g ** 3)
    s = 1 / (1 + np.exp(-z))
    if act == "silu":
        return s * (E * np.abs(g) * s + 2 * np.abs(g) * (1 - s) + (E + 2) * np.abs(1 + g * (1 - s)))
    d, f = s * (1 - s), np.abs(g) * C2 * (1 + 3 * K * g * g)
    return s * E + f * (d * (E + 8) + s * (E * s + 1)) + np.abs(s + g * C2 * (1 + 3 * K * g * g) * d)


@pytest.mark.parametrize("T,N", [(3, 96), (3, 97), (16, 40), (70, 512), (70, 261), (300, 1032)])
@pytest.mark.parametrize("act,most", [("silu", 72.0), ("gelu", 9.0)])
def test_products_alone(dbf, T, N, act, most):
    """g and u are single products of codes, exact; every path that reads nothing else."""
    rng = np.random.default_rng(T + N)
    w, up, x = np.zeros((N, 32)), np.zeros((N, 32)), np.zeros((T, 32))
    w[:, 3] = R.E2M1[rng.integers(1, 8, N)] * rng.choice([-1.0, 1.0], N)
    up[:, 3] = R.E2M1[rng.integers(1, 8, N)]
    x[:, 3] = R.E2M1[rng.integers(1, 8, T)] * most / 36
    g, u = x @ w.T, x @ up.T
    assert np.array_equal(R.mx4(x)[0], x) and g.min() < -most / 4
    gl, ul = (dbf.Mx4Layer.quantize(torch.tensor(a, dtype=torch.float32).cuda()) for a in (w, up))
    h = host(dbf.mx4_gated_forward(gl, ul, torch.tensor(x, dtype=torch.float32).cuda(), act=act, h_dtype=torch.float32))
    ref = R.gate(act, g) * u
    if act == "gelu":   # the tanh form in 64 bits cancels below g = -5: its sigmoid form does not
        ref = g * u / (1 + np.exp(-C2 * (g + K * g ** 3)))
    assert np.all(np.abs(h - ref) <= value_units(act, g) * UNIT * np.abs(ref))


@pytest.mark.parametrize("T,N", [(3, 96), (3, 97), (70, 512), (70, 261)])
@pytest.mark.parametrize("act,most", [("silu", 80.0), ("gelu", 9.0)])
@pytest.mark.parametrize("which", ["both", "g"])
@pytest.mark.parametrize("kind", [torch.float32, torch.bfloat16])
def test_addends(dbf, T, N, act, most, which, kind):
    """Weights of zero in the gate: g is its addend (one of two, or the only one, of either type)."""
    rng = np.random.default_rng(T + N)
    ga = torch.tensor(rng.uniform(-most, most, (T, N))).to(kind).cuda()
    ua = torch.tensor(rng.uniform(1, 2, (T, N))).to(kind).cuda()
    gl, ul = dbf.Mx4Layer.quantize(torch.zeros(N, 64, device="cuda")), dbf.Mx4Layer.quantize(torch.ones(N, 64, device="cuda"))
    x = torch.ones(T, 64, device="cuda")
    kw = {"g_add": ga, "u_add": ua} if which == "both" else {"g_add": ga}
    h = host(dbf.mx4_gated_forward(gl, ul, x, act=act, h_dtype=torch.float32, **kw))
    g, u = host(ga), np.full((T, N), 64.0)
    if which == "both":
        u = (u + host(ua)).astype(np.float32).astype(np.float64)   # the sum's own rounding
    ref = g * u / (1 + np.exp(-(g if act == "silu" else C2 * (g + K * g ** 3))))
    assert np.all(np.abs(h - ref) <= value_units(act, g) * UNIT * np.abs(ref))


@pytest.mark.parametrize("T,N", [(1, 32), (40, 264), (33, 95)])
@pytest.mark.parametrize("act,most", [("silu", 72.0), ("gelu", 9.0)])
def test_gradients(dbf, T, N, act, most):
    rng = np.random.default_rng(T + N)
    g, u = (torch.tensor(rng.uniform(-m, m, (T, N)), dtype=torch.float32).cuda() for m in (most, 2.0))
    saved = tuple(dbf.act8_save(v) for v in (g, u))
    g, u = (R.act8(host(v))[0] for v in (g, u))
    dh = torch.tensor(rng.standard_normal((T, N)), dtype=torch.float32).cuda()
    L = dbf.Mx4Layer.quantize(torch.ones(N, 32, device="cuda"))
    _, dg, du = dbf.mx4_gated_backward(L, L, dh, saved, act=act, want_dx=False)
    d = host(dh)
    z = g if act == "silu" else C2 * (g + K * g ** 3)
    s = 1 / (1 + np.exp(-z))
    ref = d * g * s
    assert np.all(np.abs(host(du) - ref) <= value_units(act, g) * UNIT * np.abs(ref))
    slope = s * (1 + g * (1 - s)) if act == "silu" else s + g * s * (1 - s) * C2 * (1 + 3 * K * g * g)
    ref = d * u * slope
    assert np.all(np.abs(host(dg) - ref) <= (slope_units(act, g) * np.abs(d * u) + 2 * np.abs(ref)) * UNIT)
