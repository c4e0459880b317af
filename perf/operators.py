"""Cases of the MXFP4 operators: the cast to microscaled 4-bit floats and back, the products of 4-bit
operands (forward, input gradient, weight gradient into fp32), the products of bf16 activations with
4-bit weights, and the linear layer's training step built from them.

A block is 32 elements along the contraction axis: packed E2M1 codes (element 2j in the low nibble of
byte j) and one E8M0 scale byte s, standing for E2M1(code) * 2^(s - 127).
"""
import math

import numpy as np
import torch

own = False

# Shards of the repository's workloads: 1B-class fc1 [8192, 2048], fc2 [2048, 4096], qkv [1536, 2048];
# 7B-class qkv [6144, 4096], fc1 [11008, 4096], fc2 [4096, 5504]; 8192 tokens to a micro-batch.
_CASES = [
    # one token through a layer whose weight is kept in 4 bits: decoding one sequence
    {"name": "w4 1 token 1B fc1", "op": "fwd4w", "T": 1, "in": 2048, "out": 8192},
    # a decoding batch of 16 sequences
    {"name": "w4 16 tokens 7B fc1", "op": "fwd4w", "T": 16, "in": 4096, "out": 11008},
    # input gradient through a frozen 4-bit weight, a short odd batch
    {"name": "w4 dgrad 200 7B fc2", "op": "dgrad4w", "T": 200, "in": 5504, "out": 4096},
    # one token with both operands in 4 bits
    {"name": "fwd 1 token 7B qkv", "op": "fwd", "T": 1, "in": 4096, "out": 6144},
    # ragged sizes: no extent fills its last tile
    {"name": "fwd ragged", "op": "fwd", "T": 1000, "in": 1056, "out": 776},
    # a training micro-batch forward
    {"name": "fwd 8192 1B fc1", "op": "fwd", "T": 8192, "in": 2048, "out": 8192},
    # its input gradient on the widest layer
    {"name": "dgrad 8192 7B fc1", "op": "dgrad", "T": 8192, "in": 4096, "out": 11008},
    # weight gradients of two micro-batches: few output tiles and a long contraction, and the widest layer
    {"name": "wgrad 8192 1B qkv", "op": "wgrad", "T": 8192, "in": 2048, "out": 1536},
    {"name": "wgrad 8192 7B fc1", "op": "wgrad", "T": 8192, "in": 4096, "out": 11008},
    # casting a short ragged activation, and the widest gradient with stochastic rounding
    {"name": "cast ragged", "op": "cast", "rows": 1000, "cols": 2064, "stochastic": False},
    {"name": "cast 8192 7B fc1 dY", "op": "cast", "rows": 8192, "cols": 11008, "stochastic": True},
    # the whole training step of a layer from bf16 tensors: three casts and three products
    {"name": "step 8192 1B fc2", "op": "step", "T": 8192, "in": 4096, "out": 2048},
]


def listed():
    return [dict(c) for c in _CASES]


def _log(rng, lo, hi, mult):
    return max(mult, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / mult)) * mult)


def draw(rng):
    op = rng.choice(["fwd4w", "fwd4w", "dgrad4w", "fwd", "fwd", "dgrad", "wgrad", "cast", "step"])
    if op == "cast":
        return {"op": op, "rows": _log(rng, 1, 8192, 1), "cols": _log(rng, 32, 11008, 8), "stochastic": rng.random() < 0.5}
    n_in = _log(rng, 256, 8192, 32 if op in ("fwd", "fwd4w", "dgrad4w") else 8)
    n_out = _log(rng, 256, 8192, 32 if op == "dgrad" else 8)
    # no more multiplications than in the widest layer's two weight gradients
    most = 2 * 8192 * 4096 * 11008 // ({"wgrad": 2, "step": 3}.get(op, 1) * n_in * n_out)
    T = _log(rng, 1, min(8192, most // 32 * 32), 32 if op == "wgrad" else 1)
    return {"op": op, "T": T, "in": n_in, "out": n_out}


def _up32(n):
    return (n + 31) // 32 * 32


def work(case):
    if case["op"] == "cast":
        R, C = case["rows"], case["cols"]
        elems = R * _up32(C) + C * _up32(R)
        return {"bytes": 2 * R * C + elems * (0.5 + 1 / 32) + 2 * elems, "flops": 0}
    T, i, o = case["T"], case["in"], case["out"]
    b4 = 0.5 + 1 / 32
    one = 2 * T * i * o
    if case["op"] == "fwd4w":
        return {"bytes": o * i * b4 + 2 * T * (i + o), "flops": one}
    if case["op"] == "dgrad4w":
        return {"bytes": o * i * b4 + 2 * T * (i + o), "flops": one}
    if case["op"] == "fwd":
        return {"bytes": (T + o) * i * b4 + 2 * T * o, "flops": one}
    if case["op"] == "dgrad":
        return {"bytes": (T + i) * o * b4 + 2 * T * i, "flops": one}
    if case["op"] == "wgrad":
        return {"bytes": 2 * (o + i) * T * b4 + 4 * o * i, "flops": 2 * one}
    return {"bytes": 2 * (T * i + o * i + T * o) + 2 * T * (o + i) + 4 * o * i, "flops": 3 * one}


# ---- plain form ---------------------------------------------------------------------------------

def _power(e):
    """2^e as float32, e an integer tensor in -127 .. 127."""
    return torch.where(e == -127, torch.full_like(e, 1 << 22), (e + 127) << 23).to(torch.int32).view(torch.float32)


def _mul32(m, c):
    """High and low 32-bit words of m * c, both below 2^32, in 64-bit integers."""
    low, high = c & 0xFFFF, c >> 16
    return ((m * high + ((m * low) >> 16)) >> 16) & 0xFFFFFFFF, (m * c) & 0xFFFFFFFF


def _draws(rows, cols, seed, device):
    """The 16-bit draw of each element [rows, cols]: Philox4x32 of 7 rounds, the group of 8 elements as its counter."""
    n = rows * cols // 8
    c0 = torch.arange(n, dtype=torch.int64, device=device)
    c0, c1 = c0 & 0xFFFFFFFF, c0 >> 32
    c2, c3 = torch.zeros_like(c0), torch.zeros_like(c0)
    k0, k1 = seed & 0xFFFFFFFF, (seed >> 32) & 0xFFFFFFFF
    for _ in range(7):
        h0, l0 = _mul32(0xD2511F53, c0)
        h1, l1 = _mul32(0xCD9E8D57, c2)
        c0, c1, c2, c3 = h1 ^ c1 ^ k0, l1, h0 ^ c3 ^ k1, l0
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    w = torch.stack([c0, c1, c2, c3], -1)
    return torch.stack([w & 0xFFFF, w >> 16], -1).reshape(rows, cols)


def _codes(x, draws=None):
    """Codes [R, C'] (0..15) and scale bytes [R, C'/32] of x [R, C], C' the next multiple of 32."""
    R, C = x.shape
    x = torch.nn.functional.pad(x.float(), (0, -C % 32)).reshape(R, -1, 32)
    mant, exp = torch.frexp(x.abs().amax(-1))
    exp = exp.to(torch.int64) - 3
    if draws is not None:
        exp = exp + (mant > 0.75)
    exp = torch.where(mant == 0, torch.full_like(exp, -127), exp.clamp(-127, 127))
    v = x.abs() * _power(-exp)[..., None]
    if draws is None:
        code = ((v > 0.25).to(torch.uint8) + (v >= 0.75) + (v > 1.25) + (v >= 1.75) + (v > 2.5) + (v >= 3.5) + (v > 5.0))
    else:
        r = torch.nn.functional.pad(draws.float(), (0, -C % 32)).reshape(R, -1, 32)
        up = (v >= 2).float() + (v >= 4)
        n = torch.floor((torch.floor(v * torch.exp2(1 - up) * 65536) + r) / 65536)
        code = (n + 2 * up).to(torch.uint8)
    code = code + 8 * (x < 0).to(torch.uint8)
    return code.reshape(R, -1), (exp + 127).to(torch.uint8)


def _pack(code):
    return code[:, 0::2] | (code[:, 1::2] << 4)


def _values(code, scale):
    """float32 values of codes [R, C] and scale bytes [R, C/32]."""
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6], device=code.device)
    v = table[code.to(torch.int32)].reshape(scale.shape[0], -1, 32)
    return (v * _power(scale.to(torch.int64) - 127)[..., None]).reshape(code.shape)


def _unpack(q, s):
    return _values(torch.stack([q & 15, q >> 4], -1).reshape(q.shape[0], -1), s)


def _cast(x, seed=None):
    """x's rowwise and columnwise values in float32."""
    d = None if seed is None else _draws(*x.shape, seed, x.device)
    return _values(*_codes(x, d)), _values(*_codes(x.t(), None if d is None else d.t()))


# ---- inputs -------------------------------------------------------------------------------------

def _normal(gen, shape, std):
    """bf16 normal values whose columns differ in size, as activations' channels do."""
    x = torch.randn(shape, generator=gen, device="cuda")
    x *= std * torch.exp(0.5 * torch.randn(shape[1], generator=gen, device="cuda"))
    return x.to(torch.bfloat16)


def _quantised(gen, shape, std):
    code, s = _codes(_normal(gen, shape, std))
    return _pack(code), s


_STD = {"X": 1.0, "W": 0.02, "dY": 0.001}


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case)
    if case["op"] == "cast":
        st["x"] = _normal(gen, (case["rows"], case["cols"]), _STD["dY"] if case["stochastic"] else _STD["X"])
        st["seed"] = 0x5EED00000000 + seed if case["stochastic"] else None
        return st
    T, i, o = case["T"], case["in"], case["out"]
    if case["op"] in ("fwd4w", "dgrad4w"):
        st["W"] = _quantised(gen, (o, i), _STD["W"])
        st["x"] = _normal(gen, (T, i), _STD["X"]) if case["op"] == "fwd4w" else _normal(gen, (T, o), _STD["dY"])
    elif case["op"] == "fwd":
        st["X"], st["W"] = _quantised(gen, (T, i), _STD["X"]), _quantised(gen, (o, i), _STD["W"])
    elif case["op"] == "dgrad":
        st["dY"], st["WT"] = _quantised(gen, (T, o), _STD["dY"]), _quantised(gen, (i, o), _STD["W"])
    elif case["op"] == "wgrad":
        st["dYT"] = [_quantised(gen, (o, T), _STD["dY"]) for _ in range(2)]
        st["XT"] = [_quantised(gen, (i, T), _STD["X"]) for _ in range(2)]
        st["main_grad"] = torch.zeros((o, i), device="cuda")
    else:
        st["x"] = _normal(gen, (T, i), _STD["X"]).requires_grad_()
        st["weight"] = torch.nn.Parameter(_normal(gen, (o, i), _STD["W"]))
        st["weight"].main_grad = st["main_grad"] = torch.zeros((o, i), device="cuda")
        st["dy"] = _normal(gen, (T, o), _STD["dY"])
        st["seed"] = 0x5EED00000000 + seed
    return st


# ---- one pass -----------------------------------------------------------------------------------

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import sharded_linear_amd as sl
    op = st["op"]
    if op == "cast":
        qr, sr, qc, sc = sl.sl_mxfp4_quantize(st["x"], seed=st["seed"])
        return sl.sl_mxfp4_dequantize(qr, sr), sl.sl_mxfp4_dequantize(qc, sc)
    if op == "fwd4w":
        return sl.sl_linear_fwd_mxfp4w(st["x"], *st["W"])
    if op == "dgrad4w":
        return sl.sl_linear_dgrad_mxfp4w(st["x"], *st["W"])
    if op == "fwd":
        return sl.sl_linear_fwd_mxfp4(*st["X"], *st["W"])
    if op == "dgrad":
        return sl.sl_linear_dgrad_mxfp4(*st["dY"], *st["WT"])
    sl.sl_grad_buffer_zero(st["main_grad"].view(-1))
    if op == "wgrad":
        for dy, x in zip(st["dYT"], st["XT"]):
            sl.sl_linear_wgrad_accum_mxfp4(*dy, *x, st["main_grad"])
        return st["main_grad"]
    y = sl.linear_mxfp4_with_grad_accumulation(st["x"], st["weight"], seed=st["seed"])
    dx, = torch.autograd.grad(y, st["x"], st["dy"])
    return y.detach(), dx, st["main_grad"]


def _run_plain(st):
    op = st["op"]
    if op == "cast":
        r, c = _cast(st["x"], st["seed"])
        return r.to(torch.bfloat16), c.to(torch.bfloat16)
    if op == "fwd4w":
        return (st["x"].float() @ _unpack(*st["W"]).t()).to(torch.bfloat16)
    if op == "dgrad4w":
        return (st["x"].float() @ _unpack(*st["W"])).to(torch.bfloat16)
    if op == "fwd":
        return (_unpack(*st["X"]) @ _unpack(*st["W"]).t()).to(torch.bfloat16)
    if op == "dgrad":
        return (_unpack(*st["dY"]) @ _unpack(*st["WT"]).t()).to(torch.bfloat16)
    g = st["main_grad"].zero_()
    if op == "wgrad":
        for dy, x in zip(st["dYT"], st["XT"]):
            g += _unpack(*dy) @ _unpack(*x).t()
        return g
    x, w, dy = st["x"].detach(), st["weight"].detach(), st["dy"]
    xr, xc = _cast(x)
    wr, wc = _cast(w)
    dr, dc = _cast(dy, st["seed"])
    y = xr @ wr.t()
    dx = dr @ wc.t()
    g += dc @ xc.t()
    return y.to(torch.bfloat16), dx.to(torch.bfloat16), g


# ---- the definition in 64 bits ------------------------------------------------------------------

def _philox_draws(rows, cols, seed):
    u, low = np.uint64, np.uint64(0xFFFFFFFF)
    g = np.arange(rows * cols // 8, dtype=u)
    c = [g & low, g >> u(32), np.zeros_like(g), np.zeros_like(g)]
    k = [u(seed & 0xFFFFFFFF), u(seed >> 32 & 0xFFFFFFFF)]
    for n in range(7):
        a, b = c[0] * u(0xD2511F53), c[2] * u(0xCD9E8D57)
        c = [(b >> u(32)) ^ c[1] ^ k[0], b & low, (a >> u(32)) ^ c[3] ^ k[1], a & low]
        k = [(k[0] + u(0x9E3779B9)) & low, (k[1] + u(0xBB67AE85)) & low]
    words = np.stack(c, 1).astype("<u4")
    return torch.from_numpy(words.view("<u2").astype(np.int32).reshape(rows, cols)).cuda()


def _rounded(x, draws=None):
    """What x [R, C] stands for after the cast along its rows, in float64 [R, C']."""
    R, C = x.shape
    n = _up32(C)
    full = torch.zeros((R, n), dtype=torch.float64, device=x.device)
    full[:, :C] = x.double()
    b = full.view(R, n // 32, 32)
    amax = b.abs().amax(2, keepdim=True)
    safe = torch.where(amax > 0, amax, torch.ones_like(amax))
    e = torch.floor(torch.log2(safe))
    e = torch.where(torch.exp2(e) > safe, e - 1, torch.where(torch.exp2(e + 1) <= safe, e + 1, e))   # log2 rounded across
    X = e - 2
    if draws is not None:
        X = torch.where(safe > 6 * torch.exp2(X), X + 1, X)
    unit = torch.exp2(X.clamp(-127, 127))
    v = b.abs() / unit
    step = torch.where(v < 2, 0.5, torch.where(v < 4, 1.0, 2.0)).double()
    if draws is None:
        out = (torch.round(v / step) * step).clamp(max=6.0)
    else:
        r = torch.zeros((R, n), dtype=torch.float64, device=x.device)
        r[:, :C] = draws
        out = torch.floor((torch.floor(v / step * 65536) + r.view_as(b)) / 65536) * step
    return (torch.sign(b) * out * unit).view(R, n)


def _decoded(packed, scale):
    q = packed.to(torch.int64)
    nib = torch.empty((q.shape[0], q.shape[1] * 2), dtype=torch.int64, device=q.device)
    nib[:, 0::2], nib[:, 1::2] = q % 16, q // 16
    mag = nib % 8
    m = torch.where(mag < 2, mag.double() / 2, (1 + (mag % 2).double() / 2) * torch.exp2((mag // 2 - 1).double()))
    m = torch.where(nib >= 8, -m, m)
    return m * torch.exp2(scale.double() - 127).repeat_interleave(32, dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("cast", "step"):
        x = (st["x"] if op == "cast" else st["dy"]).detach()
        d = None if st["seed"] is None else _philox_draws(*x.shape, st["seed"])
        r, c = _rounded(x, d), _rounded(x.t(), None if d is None else d.t())
        if op == "cast":
            return r, c
        a, w = st["x"].detach(), st["weight"].detach()
        y = _rounded(a) @ _rounded(w).t()
        dx = r @ _rounded(w.t())[:, :r.shape[1]].t()
        return y, dx, c @ _rounded(a.t()).t()
    if op == "fwd4w":
        return st["x"].double() @ _decoded(*st["W"]).t()
    if op == "dgrad4w":
        return st["x"].double() @ _decoded(*st["W"])
    if op == "fwd":
        return _decoded(*st["X"]) @ _decoded(*st["W"]).t()
    if op == "dgrad":
        return _decoded(*st["dY"]) @ _decoded(*st["WT"]).t()
    return sum(_decoded(*dy) @ _decoded(*x).t() for dy, x in zip(st["dYT"], st["XT"]))
