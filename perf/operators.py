"""The 4-bit base layer and its gated feed-forward block: measured cases.

Operators, each with its plain form in elementary torch operations:

  quantize     dbf.mx4_quantize, dbf.mx4_dequantize: a matrix to microscaled 4-bit floats (E2M1 codes, one
               E8M0 scale per 32 consecutive columns of a row) and back.
  forward      dbf.mx4_forward: y = W q(x), W and q(x) microscaled 4-bit, fp32 sums.
  backward     dbf.mx4_backward: dx = dy W, the gradient of the product with respect to q(x).
  gated        dbf.mx4_gated_forward: h = silu(g) . u with g = Wg q(x) [+ g_add], u = Wu q(x) [+ u_add].
  gated_train  the same with g and u kept in 8 bits, then dbf.mx4_gated_backward: dg, du and dx from dh and
               the 8-bit g and u.
  act8         dbf.act8_save, dbf.act8_load: an activation to 8 bits (E4M3 codes, one E8M0 scale per 32
               columns) and back.

Layouts (shared by both sides): 4-bit codes are rows of ceil(k/32) * 16 bytes, column 2j in the low nibble of
byte j; their scales lie in tiles of 128 rows x 4 blocks, [row tile][block tile][32][4][4], row r and block b
at [r // 128][b // 4][r % 32][r % 128 // 32][b % 4].
"""
import math

import torch

own = False

BLOCK = 32
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ---- cases ---------------------------------------------------------------------------------------
def listed():
    return [
        # the base weight of an MLP projection, quantised when a model is loaded, read back for a merge
        {"name": "quantize 11008x4096 bf16", "op": "quantize", "N": 11008, "M": 4096, "x": "bf16"},
        # a ragged batch of fp32 activations whose width ends inside a block of 32
        {"name": "quantize 333x1371 f32", "op": "quantize", "N": 333, "M": 1371, "x": "f32"},
        # one decoding step through the up projection: latency
        {"name": "forward T=1 4096->11008", "op": "forward", "T": 1, "M": 4096, "N": 11008, "x": "bf16", "y": "bf16"},
        # a batch of decoding sequences or a short prompt, odd sizes, fp32 in and out
        {"name": "forward T=77 1000->2200 f32", "op": "forward", "T": 77, "M": 1000, "N": 2200, "x": "f32", "y": "f32"},
        # the largest layer of the benchmark at its prefill size
        {"name": "forward T=8192 8192->8192", "op": "forward", "T": 8192, "M": 8192, "N": 8192, "x": "bf16", "y": "bf16"},
        # the gradient through the frozen base of the MLP projection: adapter training
        {"name": "backward T=2048 4096->11008", "op": "backward", "T": 2048, "M": 4096, "N": 11008, "x": "bf16", "y": "bf16"},
        # one decoding step through gate and up projections
        {"name": "gated T=1 4096->11008", "op": "gated", "T": 1, "M": 4096, "N": 11008, "x": "bf16", "y": "bf16", "add": False},
        # prefill with an adapter's branch added to both projections
        {"name": "gated T=2048 4096->11008 +adapter", "op": "gated", "T": 2048, "M": 4096, "N": 11008, "x": "bf16", "y": "bf16", "add": True},
        # a small training step with odd sizes
        {"name": "gated_train T=301 520->1352", "op": "gated_train", "T": 301, "M": 520, "N": 1352, "x": "bf16", "y": "bf16", "add": False},
        # the training step of the MLP block at the benchmark's token count
        {"name": "gated_train T=2048 4096->11008", "op": "gated_train", "T": 2048, "M": 4096, "N": 11008, "x": "bf16", "y": "bf16", "add": False},
        # the block's input kept for an adapter's backward pass
        {"name": "act8 2048x4096 bf16", "op": "act8", "N": 2048, "M": 4096, "x": "bf16"},
        # the MLP's hidden activations of a long batch
        {"name": "act8 8191x11000 f32", "op": "act8", "N": 8191, "M": 11000, "x": "f32"},
    ]


def _log(rng, low, high):
    return max(low, min(high, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(("quantize", "forward", "forward", "backward", "gated", "gated", "gated_train", "act8"))
    kind = rng.choice(("bf16", "bf16", "f32"))
    if op in ("quantize", "act8"):
        return {"op": op, "N": _log(rng, 1, 11008), "M": _log(rng, 24, 11008), "x": rng.choice(("bf16", "f32", "f16") if op == "quantize" else ("bf16", "f32"))}
    M, N, T = _log(rng, 128, 8192), _log(rng, 128, 11008), _log(rng, 1, 8192)
    if rng.random() < 0.5:  # widths of real layers are mostly multiples of 64, the others odd
        M, N = -(-M // 64) * 64, -(-N // 64) * 64
    most = 0.9 * 8192 ** 3 / {"forward": 1, "backward": 1, "gated": 2, "gated_train": 4}[op]
    T = max(1, min(T, int(most / (M * N))))
    case = {"op": op, "T": T, "M": M, "N": N, "x": kind, "y": "bf16" if op != "forward" else kind}
    if op in ("gated", "gated_train"):
        case["add"] = rng.random() < 0.5
        case["x"] = "bf16" if op == "gated_train" else kind
    return case


# ---- formats, plain ------------------------------------------------------------------------------
def _blocks(x):
    """x [rows, k] as fp32 [rows, ceil(k/32), 32], zeros behind the last column."""
    rows, k = x.shape
    nb = -(-k // BLOCK)
    x = x.float()
    if nb * BLOCK != k:
        x = torch.cat([x, x.new_zeros(rows, nb * BLOCK - k)], 1)
    return x.view(rows, nb, BLOCK)


def _pow2(byte):
    """2^(byte - 127) in fp32, exact; byte 255 is NaN."""
    b = byte.to(torch.int32)
    v = torch.where(b == 0, 0x00400000, b << 23).to(torch.int32).view(torch.float32)
    return torch.where(b == 255, float("nan"), v)


def _mx4(x):
    """(magnitude values, sign bit, scale bytes) of x in blocks: scale 2^(floor(log2 amax) - 2), codes to nearest even, at most 6."""
    v = _blocks(x)
    amax = v.abs().amax(2)
    byte = (torch.frexp(amax)[1] - 1 - 2).clamp(-127, 127) + 127
    byte = torch.where(amax == 0, 0, byte)
    byte = torch.where(torch.isfinite(amax), byte, 255)
    w = v.abs() * _pow2(torch.where(byte == 255, 127, 254 - byte))[:, :, None]
    step = torch.where(w < 2, 0.5, torch.where(w < 4, 1.0, 2.0))
    return (torch.round(w / step) * step).clamp(max=6.0), torch.signbit(v), byte


def _mx4_values(x):
    """q(x): what x's microscaled 4-bit form stands for, fp32."""
    mag, neg, byte = _mx4(x)
    v = torch.where(neg, -mag, mag) * _pow2(byte)[:, :, None]
    return v.flatten(1)[:, : x.shape[1]]


def _pack(mag, neg, byte):
    """Codes and tiled scales of _mx4's answer in the layouts of this file's head."""
    rows, nb = byte.shape
    code = torch.bucketize(mag, torch.tensor(E2M1, device=mag.device)).to(torch.uint8) | (neg.to(torch.uint8) << 3)
    code = code.flatten(1)
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    rt, ct = -(-rows // 128), -(-nb // 4)
    full = torch.zeros(rt * 128, ct * 4, dtype=torch.uint8, device=mag.device)
    full[:rows, :nb] = byte.to(torch.uint8)
    return codes, full.view(rt, 4, 32, ct, 4).permute(0, 3, 2, 1, 4).contiguous()


def _scale_rows(scales, rows, nb):
    rt, ct = scales.shape[:2]
    return scales.permute(0, 3, 2, 1, 4).reshape(rt * 128, ct * 4)[:rows, :nb]


def _weight(codes, scales, rows, k):
    """The fp32 matrix that codes and tiled scales stand for."""
    nb = codes.shape[1] // 16
    nibble = torch.stack([codes & 15, codes >> 4], 2).view(rows, nb, BLOCK)
    table = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    return (table[nibble.int()] * _pow2(_scale_rows(scales, rows, nb))[:, :, None]).flatten(1)[:, :k]


def _act8_values(x):
    """What x's 8-bit form stands for, fp32: the smallest scale 2^s with amax <= 448 2^s, E4M3 to nearest even."""
    v = _blocks(x)
    amax = v.abs().amax(2)
    frac, e = torch.frexp(amax)
    byte = (e - 1 - 8 + (frac > 0.875).int()).clamp(-127, 127) + 127
    byte = torch.where(amax == 0, 0, byte)
    byte = torch.where(torch.isfinite(amax), byte, 255)
    w = v * _pow2(torch.where(byte == 255, 127, 254 - byte))[:, :, None]
    step = _pow2((torch.frexp(w)[1] - 1).clamp(min=-6) - 3 + 127)
    return (torch.round(w / step) * step * _pow2(byte)[:, :, None]).flatten(1)[:, : x.shape[1]]


# ---- inputs --------------------------------------------------------------------------------------
def _activation(gen, rows, cols, kind):
    """Normal values with a few channels that are much larger, as hidden states have."""
    x = torch.randn(rows, cols, device="cuda", generator=gen)
    big = torch.rand(cols, device="cuda", generator=gen) < 0.01
    return (x * torch.where(big, 12.0, 1.0)).to(TYPES[kind])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, M, N = case["op"], case["M"], case["N"]
    s = {"case": case}
    if op in ("quantize", "act8"):
        s["x"] = _activation(gen, N, M, case["x"])
        return s
    T = case["T"]
    for name in ("w",) if op in ("forward", "backward") else ("gate", "up"):
        w = torch.randn(N, M, device="cuda", generator=gen) / math.sqrt(M if op != "backward" else N)
        s[name] = _pack(*_mx4(w))
        del w
    if op == "backward":
        s["dy"] = torch.randn(T, N, device="cuda", generator=gen).to(TYPES[case["x"]])
        return s
    s["x"] = _activation(gen, T, M, case["x"])
    if case.get("add"):
        s["g_add"], s["u_add"] = ((0.3 * torch.randn(T, N, device="cuda", generator=gen)).to(torch.bfloat16) for _ in range(2))
    if op == "gated_train":
        s["dh"] = torch.randn(T, N, device="cuda", generator=gen).to(TYPES[case["x"]])
    return s


# ---- one pass ------------------------------------------------------------------------------------
def run(s):
    return _own(s) if own else _plain(s)


def _plain(s):
    case = s["case"]
    op, M, N = case["op"], case["M"], case["N"]
    if op == "quantize":
        codes, scales = _pack(*_mx4(s["x"]))
        return _weight(codes, scales, N, M).to(torch.bfloat16)
    if op == "act8":
        return _act8_values(s["x"]).to(torch.bfloat16)
    out = TYPES[case["y"]]
    if op == "forward":
        return (_mx4_values(s["x"]) @ _weight(*s["w"], N, M).t()).to(out)
    if op == "backward":
        return (s["dy"].float() @ _weight(*s["w"], N, M)).to(out)
    x, wg, wu = _mx4_values(s["x"]), _weight(*s["gate"], N, M), _weight(*s["up"], N, M)
    g, u = x @ wg.t(), x @ wu.t()
    if case.get("add"):
        g, u = g + s["g_add"].float(), u + s["u_add"].float()
    h = (g / (1 + torch.exp(-g)) * u).to(out)
    if op == "gated":
        return h
    g, u, dh = _act8_values(g), _act8_values(u), s["dh"].float()
    sig = 1 / (1 + torch.exp(-g))
    dg = (dh * u * sig * (1 + g * (1 - sig))).to(s["dh"].dtype)
    du = (dh * g * sig).to(s["dh"].dtype)
    return {"h": h, "dg": dg, "du": du, "dx": (dg.float() @ wg + du.float() @ wu).to(out)}


def _own(s):
    import double_binary_rank_b200 as dbf

    case = s["case"]
    op, M, N = case["op"], case["M"], case["N"]
    if op == "quantize":
        codes, scales = dbf.mx4_quantize(s["x"])
        return dbf.mx4_dequantize(codes, scales, N, M, dtype=torch.bfloat16)
    if op == "act8":
        return dbf.act8_load(dbf.act8_save(s["x"]), dtype=torch.bfloat16)
    T, out = case["T"], TYPES[case["y"]]
    if "layers" not in s:  # a program makes its layers and workspaces once
        s["layers"] = [dbf.Mx4Layer(M, N, *s[n]) for n in ("w", "gate", "up") if n in s]
        if op == "forward":
            s["ws"] = dbf.alloc_workspace(dbf.mx4_workspace_bytes(s["layers"][0], T), "cuda")
        elif op == "backward":
            s["ws"] = dbf.alloc_workspace(dbf.mx4_backward_workspace_bytes(s["layers"][0], T, s["dy"].dtype), "cuda")
        else:
            s["ws"] = dbf.alloc_workspace(dbf.mx4_gated_workspace_bytes(*s["layers"], T), "cuda")
        if op == "gated_train":
            s["ws_back"] = dbf.alloc_workspace(dbf.mx4_gated_backward_workspace_bytes(*s["layers"], T, s["dh"].dtype), "cuda")
            s["saved"] = dbf.Act8.empty(T, N, "cuda"), dbf.Act8.empty(T, N, "cuda")
    if op == "forward":
        return dbf.mx4_forward(s["layers"][0], s["x"], ws=s["ws"], y_dtype=out, static_weights=True)
    if op == "backward":
        return dbf.mx4_backward(s["layers"][0], s["dy"], ws=s["ws"], dx_dtype=out)
    h = dbf.mx4_gated_forward(*s["layers"], s["x"], act="silu", g_add=s.get("g_add"), u_add=s.get("u_add"),
                              save=s.get("saved"), ws=s["ws"], h_dtype=out, static_weights=True)
    if op == "gated":
        return h
    dx, dg, du = dbf.mx4_gated_backward(*s["layers"], s["dh"], s["saved"], act="silu", ws=s["ws_back"], dx_dtype=out)
    return {"h": h, "dg": dg, "du": du, "dx": dx}


# ---- what a pass cannot do without -----------------------------------------------------------------
def work(case):
    op, M, N = case["op"], case["M"], case["N"]
    four = N * -(-M // BLOCK) * 17  # a 4-bit matrix with its scales
    if op == "quantize":
        return {"bytes": N * M * SIZE[case["x"]] + 2 * four + N * M * 2, "flops": 0}
    if op == "act8":
        return {"bytes": N * M * SIZE[case["x"]] + 2 * N * -(-M // BLOCK) * 33 + N * M * 2, "flops": 0}
    T, x, y = case["T"], SIZE[case["x"]], SIZE[case["y"]]
    if op in ("forward", "backward"):
        a, b = (M, N) if op == "forward" else (N, M)
        return {"bytes": four + T * a * x + T * b * y, "flops": 2 * T * M * N}
    total = 2 * four + T * M * x + T * N * y + (4 * T * N if case.get("add") else 0)
    if op == "gated":
        return {"bytes": total, "flops": 4 * T * M * N}
    kept = 2 * T * -(-N // BLOCK) * 33
    return {"bytes": total + 2 * kept + 2 * four + T * N * x + 2 * T * N * x + T * M * y, "flops": 8 * T * M * N}


# ---- in 64 bits, from the definition ----------------------------------------------------------------
def _two(e):
    """2^e in fp64, exact, for whole e in [-1022, 1023]."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _scale64(x, most, top):
    """x in fp64 blocks and their scales: the largest power of two 2^s with 2^s * 2^top <= amax (most None), or
    the smallest one with amax <= most * 2^s."""
    rows, k = x.shape
    pad = -k % BLOCK
    v = torch.nn.functional.pad(x.double(), (0, pad)).view(rows, -1, BLOCK)
    amax = v.abs().max(2, keepdim=True).values
    tiny = 2.0 ** -127
    if most is None:
        s = torch.floor(torch.log2(amax.clamp(min=2.0 ** -160))) - top
        s = torch.where(_two(s + top) > amax, s - 1, s)
        s = torch.where(_two(s + 1 + top) <= amax, s + 1, s)
    else:
        s = torch.ceil(torch.log2(amax.clamp(min=2.0 ** -160) / most))
        s = torch.where(most * _two(s) < amax, s + 1, s)
        s = torch.where(most * _two(s - 1) >= amax, s - 1, s)
    return v, _two(s).clamp(min=tiny)


def _mx4_exact(x):
    v, scale = _scale64(x, None, 2)
    w = v / scale
    a, mid = w.abs(), (0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0)
    up = (0.5, 0.5, 0.5, 0.5, 1.0, 1.0, 2.0)
    q = torch.zeros_like(a)
    for i in range(7):  # ties go to the even code
        q += up[i] * ((a > mid[i]) if i % 2 == 0 else (a >= mid[i]))
    return (torch.sign(w) * q * scale).flatten(1)[:, : x.shape[1]]


def _act8_exact(x):
    v, scale = _scale64(x, 448.0, 8)
    w = v / scale
    e = torch.floor(torch.log2(w.abs().clamp(min=2.0 ** -6)))
    e = torch.where(_two(e) > w.abs().clamp(min=2.0 ** -6), e - 1, e)
    e = torch.where(_two(e + 1) <= w.abs(), e + 1, e)
    magic = 1.5 * 2.0 ** 52 * _two(e - 3)  # adding it leaves multiples of 2^(e - 3), ties to even
    return (((w + magic) - magic) * scale).flatten(1)[:, : x.shape[1]]


def _weight_exact(codes, scales, rows, k):
    c = torch.empty(rows, codes.shape[1] * 2, dtype=torch.uint8, device=codes.device)
    c[:, 0::2], c[:, 1::2] = codes % 16, codes // 16
    c = c[:, :k].double()
    sign, c = 1 - 2 * torch.floor(c / 8), c % 8
    e, m = torch.floor(c / 2), c % 2
    value = torch.where(e == 0, 0.5 * m, (1 + 0.5 * m) * _two(e - 1))
    r, b = torch.arange(rows, device=codes.device)[:, None], torch.arange(k, device=codes.device)[None, :] // BLOCK
    byte = scales[r // 128, b // 4, r % 32, r % 128 // 32, b % 4]
    return sign * value * _two(byte.int() - 127)


def exact(case, seed):
    s = prepare(case, seed)
    op, M, N = case["op"], case["M"], case["N"]
    if op == "quantize":
        return _mx4_exact(s["x"])
    if op == "act8":
        return _act8_exact(s["x"])
    if op == "forward":
        return _mx4_exact(s["x"]) @ _weight_exact(*s["w"], N, M).t()
    if op == "backward":
        return s["dy"].double() @ _weight_exact(*s["w"], N, M)
    x = _mx4_exact(s["x"])
    wg, wu = _weight_exact(*s["gate"], N, M), _weight_exact(*s["up"], N, M)
    g, u = x @ wg.t(), x @ wu.t()
    if case.get("add"):
        g, u = g + s["g_add"].double(), u + s["u_add"].double()
    h = g * torch.sigmoid(g) * u
    if op == "gated":
        return h
    g, u, dh = _act8_exact(g), _act8_exact(u), s["dh"].double()
    sig = torch.sigmoid(g)
    dg, du = dh * u * (sig + g * sig * (1 - sig)), dh * g * sig
    # the block hands on dg and du in dh's type, and dx is the gradient of what it hands on
    dg16, du16 = dg.to(s["dh"].dtype).double(), du.to(s["dh"].dtype).double()
    return {"h": h, "dg": dg, "du": du, "dx": dg16 @ wg + du16 @ wu}
