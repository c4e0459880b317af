"""Cases of the operators around a sharded linear layer: the vocabulary-parallel embedding and its
gradient, the root-mean-square norm with the residual's addition (bf16 and MXFP8 results) and its
gradient, and the orthogonalised update (Newton-Schulz) of a weight from its accumulated gradient.

MXFP8 is E4M3 codes with one E8M0 scale byte s per 32 elements, standing for E4M3(code) * 2^(s - 127).
"""
import math

import torch

own = False

_COEFFS = (3.4445, -4.7750, 2.0315)
_STEPS = 5
_EPS = 1e-5
_LR, _MOMENTUM, _DECAY = 0.02, 0.95, 0.01

_CASES = [
    # one token of a sequence being decoded, through a shard of the table (1B-class vocabulary of 128256, two ranks)
    {"name": "embed 1 token", "op": "embed", "T": 1, "V": 64128, "H": 2048, "scale": 1.0},
    # a training micro-batch; the rank's half of the ids, zeros for the others
    {"name": "embed 8192 1B", "op": "embed", "T": 8192, "V": 64128, "H": 2048, "scale": 1.0},
    # its gradient into the fp32 buffer: a few tokens take most places, one of them pads
    {"name": "embed grad 8192 1B", "op": "embed_grad", "T": 8192, "V": 64128, "H": 2048, "scale": 1.0},
    # a ragged batch on a small table, embeddings scaled by sqrt(H)
    {"name": "embed grad ragged", "op": "embed_grad", "T": 1013, "V": 4999, "H": 1032, "scale": 32.125},
    # decoding: the block's input and its residual for one token, MXFP8 for the projection that follows
    {"name": "norm mxfp8 1 token 7B", "op": "norm8", "T": 1, "H": 4096, "residual": True, "cols": False},
    # training forward of the all-MXFP8 layer: both copies, the sum kept for the residual stream
    {"name": "norm mxfp8 8192 1B", "op": "norm8", "T": 8192, "H": 2048, "residual": True, "cols": True},
    # its gradient on the 7B-class width, the residual stream's gradient added
    {"name": "norm grad 8192 7B", "op": "norm_grad", "T": 8192, "H": 4096, "residual": True},
    # a ragged bf16 layer, forward and gradient, first norm of a model (no residual yet)
    {"name": "norm both ragged", "op": "norm_both", "T": 1003, "H": 2056, "residual": False},
    # the smallest weight's update: latency of a chain of small products
    {"name": "orth 512x256", "op": "orth", "L": 1, "rows": 512, "cols": 256},
    # the qkv weights of a model's 16 layers, one call
    {"name": "orth 16x 1B qkv", "op": "orth", "L": 16, "rows": 1536, "cols": 2048},
    # one tall weight alone
    {"name": "orth 1B fc1", "op": "orth", "L": 1, "rows": 8192, "cols": 2048},
    # a whole optimiser step of two 7B-class fc2 weights: momentum, products, weights
    {"name": "muon 2x 7B fc2", "op": "muon", "L": 2, "rows": 4096, "cols": 5504},
]


def listed():
    return [dict(c) for c in _CASES]


def _log(rng, lo, hi, mult=1):
    return max(mult, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / mult)) * mult)


def _products(L, rows, cols):
    m, n = min(rows, cols), max(rows, cols)
    return L * _STEPS * (3 * m * m * n + m * m * m)


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "norm", "norm8", "norm_grad", "norm_both", "orth", "orth", "muon"])
    if op in ("embed", "embed_grad"):
        return {"op": op, "T": _log(rng, 1, 16384), "V": _log(rng, 100, 64128), "H": _log(rng, 64, 4096, 8),
                "scale": rng.choice([1.0, 1.0, 22.625, 0.37])}
    if op in ("norm", "norm_grad", "norm_both"):
        return {"op": op, "T": _log(rng, 1, 8192), "H": _log(rng, 64, 8192, 8), "residual": rng.random() < 0.7}
    if op == "norm8":
        cols = rng.random() < 0.5
        return {"op": op, "T": _log(rng, 32, 8192, 32) if cols else _log(rng, 1, 8192), "H": _log(rng, 64, 8192, 32),
                "residual": rng.random() < 0.7, "cols": cols}
    while True:
        rows, cols = _log(rng, 16, 8192), _log(rng, 16, 8192)
        one = _products(1, rows, cols)
        most = _products(2, 4096, 5504)
        if one <= most:
            return {"op": op, "L": _log(rng, 1, max(1, min(16, most // one))), "rows": rows, "cols": cols}


def work(case):
    op = case["op"]
    if op in ("orth", "muon"):
        elems = case["L"] * case["rows"] * case["cols"]
        return {"bytes": elems * (6 if op == "orth" else 16), "flops": _products(case["L"], case["rows"], case["cols"])}
    T, H = case["T"], case["H"]
    if op == "embed":
        return {"bytes": 4 * T + 2 * T * H + 2 * min(T, case["V"]) * H // 2, "flops": 0}
    if op == "embed_grad":       # about half of the places are this rank's, about a third of those another row
        return {"bytes": 4 * T + T * H + 8 * min(T // 6 + 1, case["V"]) * H, "flops": T * H}
    r = 2 if case["residual"] else 0
    forward = T * H * (2 + 2 * r) + 2 * H + 4 * T
    backward = T * H * (6 + r) + 10 * H + 4 * T
    if op == "norm":
        return {"bytes": forward + 2 * T * H, "flops": 4 * T * H}
    if op == "norm8":
        copies = 2 if case["cols"] else 1
        return {"bytes": forward + T * H * copies * (1 + 1 / 32) * 2 + 2 * T * H * copies, "flops": 4 * T * H}
    if op == "norm_grad":
        return {"bytes": backward, "flops": 10 * T * H}
    return {"bytes": forward + 2 * T * H + backward, "flops": 14 * T * H}


# ---- inputs -------------------------------------------------------------------------------------

def _normal(gen, shape, std, dtype=torch.bfloat16):
    return (torch.randn(shape, generator=gen, device="cuda") * std).to(dtype)


def _ids(gen, T, vocab):
    """Places of text: the r-th most frequent token with probability near 1 / r, spread over the
    vocabulary; one place in 16 holds the padding token 0."""
    u = torch.rand(T, generator=gen, device="cuda", dtype=torch.float64)
    rank = (torch.exp(u * math.log(vocab)) - 1).to(torch.int64).clamp(0, vocab - 1)
    ids = (rank * 1000003 + 7) % vocab
    pad = torch.rand(T, generator=gen, device="cuda") < 1 / 16
    return torch.where(pad, torch.zeros_like(ids), ids).to(torch.int32)


def _gradient(gen, L, rows, cols):
    """A weight's accumulated gradient: directions of falling strength and noise of full rank."""
    r = max(1, min(rows, cols) // 8)
    g = 0.01 * torch.randn((L, rows, cols), generator=gen, device="cuda")
    a = torch.randn((L, rows, r), generator=gen, device="cuda")
    b = torch.randn((L, r, cols), generator=gen, device="cuda")
    a = a / (1 + torch.arange(r, device="cuda", dtype=torch.float32))
    return (g + 0.02 * torch.bmm(a, b)) * 1e-3


def prepare(case, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    st = dict(case)
    op = case["op"]
    if op in ("orth", "muon"):
        L, R, C = case["L"], case["rows"], case["cols"]
        st["G"] = _gradient(gen, L, R, C)
        if op == "muon":
            st["W"] = [_normal(gen, (R, C), 0.02) for _ in range(L)]
            st["M"] = list((10 * _gradient(gen, L, R, C)).unbind(0))
            st["G"] = list(st["G"].unbind(0))
        return st
    T, H = case["T"], case["H"]
    if op in ("embed", "embed_grad"):
        vocab = 2 * case["V"]
        st["ids"] = _ids(gen, T, vocab)
        st["start"] = int(st["ids"][0]) // case["V"] * case["V"]       # the rank that holds the first token
        if op == "embed":
            st["W"] = _normal(gen, (case["V"], H), 0.02)
        else:
            st["dY"] = _normal(gen, (T, H), 1e-3)
            st["grad"] = 1e-3 * torch.randn((case["V"], H), generator=gen, device="cuda")
        return st
    x = torch.randn((T, H), generator=gen, device="cuda") * torch.exp(0.5 * torch.randn(H, generator=gen, device="cuda"))
    st["w"] = (1 + 0.1 * torch.randn(H, generator=gen, device="cuda")).to(torch.bfloat16)
    st["x"] = x.to(torch.bfloat16)
    if op != "norm_grad" and case["residual"]:
        st["r"] = _normal(gen, (T, H), 2.0)
    if op in ("norm_grad", "norm_both"):
        st["dY"] = _normal(gen, (T, H), 1e-3)
        st["dH"] = _normal(gen, (T, H), 1e-3) if case["residual"] else None
        st["grad"] = torch.zeros(H, device="cuda")
    if op == "norm_grad":            # what the forward keeps: the normalised rows' inputs and 1 / rms
        st["rstd"] = torch.rsqrt(st["x"].float().square().mean(1) + _EPS)
    return st


# ---- one pass -----------------------------------------------------------------------------------

def run(st):
    return _run_own(st) if own else _run_plain(st)


def _run_own(st):
    import sharded_linear_amd as sl
    op = st["op"]
    if op == "embed":
        return sl.sl_embedding_fwd(st["ids"], st["W"], vocab_start=st["start"], scale=st["scale"])
    if op == "embed_grad":
        return sl.sl_embedding_wgrad_accum(st["ids"], st["dY"], st["grad"], vocab_start=st["start"], scale=st["scale"])
    if op == "norm":
        return sl.sl_rmsnorm_fwd(st["x"], st["w"], _EPS, residual=st.get("r"))
    if op == "norm8":
        qr, sr, qc, sc, h, rstd = sl.sl_rmsnorm_fwd_mxfp8(st["x"], st["w"], _EPS, residual=st.get("r"), cols=st["cols"])
        y = [sl.sl_mxfp8_dequantize(qr, sr)] + ([sl.sl_mxfp8_dequantize(qc, sc)] if st["cols"] else [])
        return y, h, rstd
    if op == "norm_grad":
        return sl.sl_rmsnorm_bwd(st["dY"], st["x"], st["w"], st["rstd"], st["grad"], dresidual=st["dH"]), st["grad"]
    if op == "norm_both":
        y, h, rstd = sl.sl_rmsnorm_fwd(st["x"], st["w"], _EPS, residual=st.get("r"))
        return y, h, rstd, sl.sl_rmsnorm_bwd(st["dY"], h, st["w"], rstd, st["grad"], dresidual=st["dH"]), st["grad"]
    if op == "orth":
        return sl.sl_orthogonalize(st["G"])
    sl.sl_muon_step(st["W"], st["G"], st["M"], _LR, momentum=_MOMENTUM, weight_decay=_DECAY)
    return st["W"], st["M"]


def _plain_codes(y):
    """y [R, C] in float32, rounded to MXFP8 along C."""
    b = y.reshape(y.shape[0], -1, 32)
    _, e = torch.frexp(b.abs().amax(-1, keepdim=True))
    e = (e - 9).clamp(-126, 127)                       # 2^-127 is no normal number; no block here is that small
    unit = ((e + 127) << 23).view(torch.float32)
    v = b / unit
    _, k = torch.frexp(v)
    step = torch.ldexp(torch.ones_like(v), k.clamp(min=-5) - 4)
    q = (torch.round(v / step) * step).clamp(-448, 448)
    return (q * unit).reshape(y.shape)


def _plain_norm(st):
    x = st["x"].float()
    if "r" in st:
        x = (x + st["r"].float()).to(torch.bfloat16).float()
    rstd = torch.rsqrt(x.square().mean(1) + _EPS)
    return x * rstd[:, None] * st["w"].float(), x.to(torch.bfloat16), rstd


def _plain_norm_grad(st, h, rstd):
    n = h.float() * rstd[:, None]
    dy = st["dY"].float()
    g = dy * st["w"].float()
    dx = (g - n * (g * n).mean(1, keepdim=True)) * rstd[:, None]
    if st["dH"] is not None:
        dx = dx + st["dH"].float()
    st["grad"] += (dy * n).sum(0)
    return dx.to(torch.bfloat16)


def _plain_orth(g):
    """[L, m, n] float32."""
    x = g / torch.linalg.vector_norm(g, dim=(1, 2), keepdim=True).clamp_min(1e-30)
    if g.shape[1] > g.shape[2]:
        x = x.transpose(1, 2).contiguous()
    a, b, c = _COEFFS
    for _ in range(_STEPS):
        A = torch.bmm(x, x.transpose(1, 2).contiguous())
        x = a * x + torch.bmm(b * A + c * torch.bmm(A, A), x)
    return x.transpose(1, 2) if g.shape[1] > g.shape[2] else x


def _run_plain(st):
    op = st["op"]
    if op in ("embed", "embed_grad"):
        at = st["ids"].to(torch.int64) - st["start"]
        here = (at >= 0) & (at < st["V"])
        at = torch.where(here, at, torch.zeros_like(at))
        if op == "embed":
            y = (st["W"][at].float() * st["scale"]).to(torch.bfloat16)
            return torch.where(here[:, None], y, torch.zeros_like(y))
        d = st["dY"].float() * st["scale"]
        return st["grad"].index_add_(0, at, torch.where(here[:, None], d, torch.zeros_like(d)))
    if op in ("norm", "norm8", "norm_both"):
        y, h, rstd = _plain_norm(st)
        if op == "norm":
            return y.to(torch.bfloat16), h, rstd
        if op == "norm8":
            return [_plain_codes(v).to(torch.bfloat16) for v in ([y, y.t().contiguous()] if st["cols"] else [y])], h, rstd
        return y.to(torch.bfloat16), h, rstd, _plain_norm_grad(st, h, rstd), st["grad"]
    if op == "norm_grad":
        return _plain_norm_grad(st, st["x"], st["rstd"]), st["grad"]
    if op == "orth":
        return _plain_orth(st["G"]).to(torch.bfloat16).contiguous()
    u = []
    for m, g in zip(st["M"], st["G"]):
        m.mul_(_MOMENTUM).add_(g)
        u.append(g + _MOMENTUM * m)
    o = _plain_orth(torch.stack(u))
    s = max(1.0, st["rows"] / st["cols"]) ** 0.5
    for k, w in enumerate(st["W"]):
        v = w.float()
        w.copy_(v - _LR * (s * o[k] + _DECAY * v))
    return st["W"], st["M"]


# ---- the definitions in 64 bits -----------------------------------------------------------------

def _exact_mx(y):
    """MXFP8 of y [R, C] (float64) along C, by the exponents of the block's largest and of each value."""
    b = y.view(y.shape[0], y.shape[1] // 32, 32)
    floor2 = lambda v: torch.floor(torch.log2(torch.where(v > 0, v, torch.ones_like(v))))  # noqa: E731

    def exponent(v):
        e = floor2(v)
        return torch.where(torch.exp2(e) > v, e - 1, torch.where(torch.exp2(e + 1) <= v, e + 1, e))

    top = b.abs().amax(2, keepdim=True)
    unit = torch.exp2((exponent(torch.where(top > 0, top, torch.ones_like(top))) - 8).clamp(-127, 127))
    mag = b.abs() / unit
    grain = torch.exp2(exponent(torch.where(mag > 0, mag, torch.ones_like(mag))).clamp(min=-6) - 3)
    out = torch.minimum(torch.round(mag / grain) * grain, torch.full_like(mag, 448.0))
    return (torch.sign(b) * out * unit).view(y.shape)


def _exact_orth(g):
    """One matrix in float64: U p(S) V^T by products on the other side of the iteration, X (a + b X'X + c (X'X)^2)."""
    norm = g.square().sum().sqrt()
    x = g / norm if norm > 0 else g.clone()
    tall = x.shape[0] > x.shape[1]
    x = x if tall else x.t().contiguous()
    eye = torch.eye(x.shape[1], dtype=torch.float64, device=x.device)
    a, b, c = _COEFFS
    for _ in range(_STEPS):
        s = x.t().contiguous() @ x
        x = x @ (s @ (c * s + b * eye) + a * eye)
    return x if tall else x.t().contiguous()


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("embed", "embed_grad"):
        V = case["V"]
        ids = st["ids"].long()
        mine = torch.nonzero((ids >= st["start"]) & (ids < st["start"] + V)).flatten()
        if op == "embed":
            y = torch.zeros((case["T"], case["H"]), dtype=torch.float64, device="cuda")
            y[mine] = st["W"].double().index_select(0, ids[mine] - st["start"]) * case["scale"]
            return y
        grad = st["grad"].double()
        rows, where = torch.unique(ids[mine] - st["start"], return_inverse=True)
        sums = torch.zeros((rows.numel(), case["H"]), dtype=torch.float64, device="cuda")
        sums.index_put_((where,), st["dY"].double()[mine], accumulate=True)
        grad[rows] += case["scale"] * sums
        return grad
    if op in ("orth", "muon"):
        if op == "orth":
            return torch.stack([_exact_orth(g) for g in st["G"].double()])
        moved, weights = [], []
        for w, g, m in zip(st["W"], st["G"], st["M"]):
            g = g.double()
            m = _MOMENTUM * m.double() + g
            moved.append(m)
            step = _exact_orth(g + _MOMENTUM * m) * max(1.0, case["rows"] / case["cols"]) ** 0.5
            weights.append(w.double() * (1 - _LR * _DECAY) - _LR * step)
        return weights, moved
    h = st["x"].double()
    total = h
    if "r" in st:
        total = h + st["r"].double()
        h = total.to(torch.bfloat16).double()          # the norm is of the sum as it is kept
    w = st["w"].double()
    inv = st["rstd"].double() if op == "norm_grad" else 1 / torch.sqrt((h * h).sum(1) / h.shape[1] + _EPS)
    y = h * w * inv[:, None]
    if op == "norm":
        return y, total, inv
    if op == "norm8":
        return [_exact_mx(y)] + ([_exact_mx(y.t().contiguous())] if case["cols"] else []), total, inv
    dy = st["dY"].double()
    mean = (dy * w * h).sum(1) / h.shape[1]
    dx = inv[:, None] * dy * w - h * (inv ** 3 * mean)[:, None]
    if st["dH"] is not None:
        dx = dx + st["dH"].double()
    grad = st["grad"].double() + (dy * h * inv[:, None]).sum(0)
    return (dx, grad) if op == "norm_grad" else (y, total, inv, dx, grad)
