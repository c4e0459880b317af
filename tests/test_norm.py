"""The root-mean-square norm with the residual's addition: refusals on the CPU, results and gradients on the GPU against 64 bits."""
import math
from fractions import Fraction

import numpy as np
import pytest
import torch

import sharded_linear_amd as sl
from oracle import numerics
from sharded_linear_amd import _lib
from tests.gpu_util import say

OK, EINVAL, EALIGN, ESHAPE, EWORKSPACE = 0, -1, -2, -3, -4
A = 1 << 20          # an aligned fake device address, never dereferenced
BF16, F32, U8 = torch.bfloat16, torch.float32, torch.uint8
U = 2.0 ** -24       # half a step of fp32
HALF = 2.0 ** -8     # half a step of bf16
# 1 / rms: a sum of squares over at most 32 elements of a lane, 6 halvings of a wave and 15 further waves, each addition and
# product half a step at most (all terms are positive), the mean, the root and the quotient
RSTD = (32 + 6 + 15 + 4) / 2 * U + 4 * U


def test_forward_validation():
    f = _lib.lib().sl_rmsnorm_fwd
    assert f(None, A, A, A, 1e-5, A, A, A, 4, 20) == ESHAPE
    assert f(None, A, A, A, 1e-5, A, A, A, 4, 16392) == ESHAPE
    assert f(None, A, A, A, 1e-5, A, A, A, 1 << 31, 16) == ESHAPE
    assert f(None, A, A, A, 1e-5, A, A, A, -1, 16) == EINVAL
    for eps in (-1e-5, float("inf"), float("nan")):
        assert f(None, A, A, A, eps, A, A, A, 4, 16) == EINVAL
    assert f(None, None, A, A, 1e-5, A, A, A, 4, 16) == EINVAL
    assert f(None, A, A, None, 1e-5, A, A, A, 4, 16) == EINVAL
    assert f(None, A, A, A, 1e-5, None, A, A, 4, 16) == EINVAL
    assert f(None, A, A, A, 1e-5, A, None, A, 4, 16) == EINVAL              # a residual without h
    assert f(None, A, A, A, 1e-5, A, A, None, 4, 16) == EINVAL
    for k in (1, 2, 3, 5, 6):
        args = [None, A, A, A, 1e-5, A, A, A, 4, 16]
        args[k] = A + 8
        assert f(*args) == EALIGN, k
    assert f(None, A, A, A, 1e-5, A, A, A + 2, 4, 16) == EALIGN
    assert f(None, None, None, None, 1e-5, None, None, None, 0, 16) == OK
    assert f(None, None, None, None, 1e-5, None, None, None, 4, 0) == OK


def test_mxfp8_forward_validation():
    f = _lib.lib().sl_rmsnorm_fwd_mxfp8
    assert f(None, A, A, A, 1e-5, A, A, None, None, A, A, 4, 48) == ESHAPE              # rows need whole blocks
    assert f(None, A, A, A, 1e-5, None, None, A, A, A, A, 33, 64) == ESHAPE
    assert f(None, A, A, A, 1e-5, A, None, A, A, A, A, 32, 64) == EINVAL
    assert f(None, A, A, A, 1e-5, A, A, A, None, A, A, 32, 64) == EINVAL
    assert f(None, A, A, A, 1e-5, A, A, A, A, None, A, 32, 64) == EINVAL
    assert f(None, A, A, A, -1.0, A, A, A, A, A, A, 32, 64) == EINVAL
    assert f(None, A, A, A, 1e-5, A + 8, A, A, A, A, A, 32, 64) == EALIGN
    assert f(None, A, A, A, 1e-5, A, A, A + 8, A, A, A, 32, 64) == EALIGN
    assert f(None, A, None, A, 1e-5, A, A, A, A, None, A, (1 << 31) - 32, 16384) == ESHAPE
    assert f(None, None, None, None, 1e-5, None, None, None, None, None, None, 0, 64) == OK


def test_gradient_validation():
    L = _lib.lib()
    f, ws = L.sl_rmsnorm_bwd, L.sl_rmsnorm_bwd_workspace_bytes
    need = ws(40, 64)
    assert need >= 64 * 4 and ws(0, 64) == 0 and ws(4, 0) == 0 and ws(4, 12) == 0 and ws(4, 16392) == 0
    assert ws(1 << 20, 64) <= 1 << 20                                                   # planes of a bounded number of workgroups
    base = [None, A, A, A, A, A, A, A, 40, 64, A, need]
    for k in (1, 2, 3, 4, 6):
        args = list(base)
        args[k] = None
        assert f(*args) == EINVAL, k
    for k in (1, 2, 3, 5, 6):
        args = list(base)
        args[k] = A + 8
        assert f(*args) == EALIGN, k
    for k in (4, 7):
        args = list(base)
        args[k] = A + 2
        assert f(*args) == EALIGN, k
    assert f(*base[:9], 60, A, need) == ESHAPE
    assert f(*base[:10], None, 0) == EWORKSPACE
    assert f(*base[:10], A, need - 1) == EWORKSPACE
    assert f(*base[:10], A + 4, need) == EWORKSPACE
    assert f(None, None, None, None, None, None, None, None, 0, 64, None, 0) == OK


def test_binding_refusals(monkeypatch):
    from sharded_linear_amd import ops
    x, w = torch.zeros(4, 64, dtype=BF16), torch.zeros(64, dtype=BF16)
    with pytest.raises(ValueError, match="GPU tensors"):
        sl.sl_rmsnorm_fwd(x, w, 1e-5)
    monkeypatch.setattr(ops, "_device", lambda t: t.device)
    with pytest.raises(ValueError, match="matrix"):
        sl.sl_rmsnorm_fwd(x[None], w, 1e-5)
    with pytest.raises(ValueError, match="w has shape"):
        sl.sl_rmsnorm_fwd(x, w[:32], 1e-5)
    with pytest.raises(TypeError, match="w must"):
        sl.sl_rmsnorm_fwd(x, w.float(), 1e-5)
    with pytest.raises(ValueError, match="residual"):
        sl.sl_rmsnorm_fwd(x, w, 1e-5, residual=x[:3])
    with pytest.raises(ValueError, match="h is the sum"):
        sl.sl_rmsnorm_fwd(x, w, 1e-5, h=x)
    with pytest.raises(ValueError, match="rstd"):
        sl.sl_rmsnorm_bwd(x, x, w, torch.zeros(5), torch.zeros(64))
    with pytest.raises(TypeError, match="w_grad"):
        sl.sl_rmsnorm_bwd(x, x, w, torch.zeros(4), w)
    p = torch.nn.Parameter(w)
    with pytest.raises(ValueError, match="main_grad"):
        sl.rmsnorm_with_grad_accumulation(x, p)
    with pytest.raises(ValueError, match="features"):
        sl.rmsnorm_with_grad_accumulation(x[:, :32], w)
    with pytest.raises(ValueError, match="residual"):
        sl.rmsnorm_with_grad_accumulation(x, w, x[:2])
    W = torch.nn.Parameter(torch.zeros(128, 64, dtype=BF16))
    with pytest.raises(ValueError, match="main_grad"):
        sl.norm_linear_mxfp8_with_grad_accumulation(x, w, W)
    W.main_grad = torch.zeros(128, 64)
    with pytest.raises(ValueError, match="128"):
        sl.norm_linear_mxfp8_with_grad_accumulation(x, w, W)


# ---- on the GPU -----------------------------------------------------------------------------------

EPS = 1e-5
# a wave to a row and a workgroup to a row, whole chunks and part of the last one, one token to many
SHAPES = [(1, 8), (1, 64), (1, 4096), (2, 520), (3, 16384), (5, 2056), (70, 1032), (129, 8192), (1024, 512), (1030, 2048), (1027, 1544),
          (1500, 4104), (3000, 64), (64, 10240)]


def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


def _inputs(T, H, residual, seed):
    g = _gen(seed)
    x = _bf16(g, T, H)
    r = _bf16(g, T, H, std=3.0) if residual else None
    return x, r, (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(BF16)


def _check_stats(x, r, h, rstd, eps=EPS):
    """h against the sum, rstd against h; returns the exact 1 / rms."""
    if r is None:
        assert h is x
    else:
        exact = x.double() + r.double()
        assert ((h.double() - exact).abs() <= exact.abs() * (HALF * (1 + 2 * U) + U)).all()
    inv = 1 / torch.sqrt(h.double().square().mean(1) + eps)
    assert ((rstd.double() - inv).abs() <= RSTD * inv).all()
    return inv


@pytest.mark.gpu
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", SHAPES)
def test_forward(T, H, residual):
    say(f"case norm T={T} H={H} residual={residual}")
    x, r, w = _inputs(T, H, residual, T + H)
    y, h, rstd = sl.sl_rmsnorm_fwd(x, w, EPS, residual=r)
    inv = _check_stats(x, r, h, rstd)
    ref = h.double() * inv[:, None] * w.double()
    assert ((y.double() - ref).abs() <= ref.abs() * (HALF * (1 + 1e-5) + RSTD + 2 * U)).all()


def _values(q, s):
    """float64 of MXFP8 codes and scales."""
    return torch.from_numpy(numerics.mxfp8_dequant(q.cpu().numpy(), s.cpu().numpy())).cuda()


def _e4m3(v):
    """|v| rounded to E4M3, saturating (float64)."""
    e = torch.floor(torch.log2(torch.where(v > 0, v, torch.ones_like(v)))).clamp(min=-6)
    step = torch.exp2(e - 3)
    return (torch.round(v / step) * step).clamp(max=448.0)


def _check_mx(q, s, y, off):
    """Codes of y [R, C] (float64) along C: what the rule gives for some value within `off` (relative) of each."""
    b = y.view(y.shape[0], -1, 32)
    top = b.abs().amax(2)
    byte = lambda t: torch.where(t > 0, (torch.floor(torch.log2(torch.where(t > 0, t, torch.ones_like(t)))) - 8).clamp(-127, 127) + 127, 0.0)  # noqa: E731
    lo, hi = byte(top * (1 - off)), byte(top * (1 + off))
    sd = s.double()
    assert ((sd == lo) | (sd == hi)).all()
    unit = torch.exp2(sd - 127)[..., None]
    got = _values(q, s).view(b.shape)
    assert (torch.sign(got) * torch.sign(b) >= 0).all()
    mag = got.abs() / unit
    assert (mag >= _e4m3(b.abs() / unit * (1 - off))).all() and (mag <= _e4m3(b.abs() / unit * (1 + off))).all()


@pytest.mark.gpu
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", [(32, 32), (64, 4096), (96, 544), (160, 2080), (1024, 2048), (1056, 672), (256, 8224), (1, 64), (7, 4096), (1025, 96)])
def test_forward_mxfp8(T, H, residual):
    say(f"case norm mxfp8 T={T} H={H} residual={residual}")
    x, r, w = _inputs(T, H, residual, T + H)
    cols = T % 32 == 0
    qr, sr, qc, sc, h, rstd = sl.sl_rmsnorm_fwd_mxfp8(x, w, EPS, residual=r, cols=cols)
    inv = _check_stats(x, r, h, rstd)
    y = h.double() * inv[:, None] * w.double()
    off = RSTD + 2 * U
    _check_mx(qr, sr, y, off)
    only = sl.sl_rmsnorm_fwd_mxfp8(x, w, EPS, residual=r, cols=False)
    assert torch.equal(only[0], qr) and torch.equal(only[1], sr) and only[2] is None and torch.equal(only[5], rstd)
    if not cols:
        return
    _check_mx(qc, sc, y.t().contiguous(), off)
    only = sl.sl_rmsnorm_fwd_mxfp8(x, w, EPS, residual=r, rows=False)
    assert torch.equal(only[2], qc) and torch.equal(only[3], sc) and only[0] is None and torch.equal(only[4], h)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(2048, 2048), (64, 4096), (96, 544)])
def test_mxfp8_codes_are_those_of_the_exact_product(T, H):
    """Rows of small integers: sums of squares are exact, so rstd in two floats is off by less than 2^-45 and each code has to be the
    exact product's."""
    say(f"case norm mxfp8 exact codes T={T} H={H}")
    g = _gen(T)
    x = torch.randint(-15, 16, (T, H), generator=g, device="cuda").to(BF16)
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(BF16)
    qr, sr, qc, sc, _, rstd = sl.sl_rmsnorm_fwd_mxfp8(x, w, 2.0 ** -17)
    inv = 1 / torch.sqrt(x.double().square().mean(1) + 2.0 ** -17)
    assert torch.equal(rstd, inv.float())
    y = x.double() * w.double() * inv[:, None]
    _check_mx(qr, sr, y, 2.0 ** -45)
    _check_mx(qc, sc, y.t().contiguous(), 2.0 ** -45)


@pytest.mark.gpu
def test_columnwise_copy_alone_takes_any_width():
    say("case norm mxfp8 columns of width 1032")
    x, r, w = _inputs(96, 1032, True, 5)
    _, _, qc, sc, h, rstd = sl.sl_rmsnorm_fwd_mxfp8(x, w, EPS, residual=r, rows=False)
    inv = _check_stats(x, r, h, rstd)
    _check_mx(qc, sc, (h.double() * inv[:, None] * w.double()).t().contiguous(), RSTD + 2 * U)


@pytest.mark.gpu
def test_mxfp8_encode_over_the_whole_range():
    """y = w in every row (h = 1, eps = 0): blocks of every magnitude that bf16 has, subnormal ones and ties among them,
    against the quantiser's codes of the same values."""
    say("case norm mxfp8, every bf16 pattern")
    bits = np.arange(65536, dtype=np.uint16)
    bits = bits[(bits & 0x7F80) != 0x7F80].reshape(-1, 32)               # finite
    for block in (bits, bits.reshape(32, -1).T.reshape(-1, 32)):         # neighbours in a block, and all magnitudes in one
        for part in np.array_split(block.reshape(-1), 8):
            w = torch.from_numpy(np.ascontiguousarray(part).view(np.int16)).view(BF16).cuda()
            x = torch.ones((32, w.numel()), dtype=BF16, device="cuda")
            qr, sr, qc, sc, _, rstd = sl.sl_rmsnorm_fwd_mxfp8(x, w, 0.0)
            assert (rstd == 1).all()
            want = sl.sl_mxfp8_quantize(w.expand(32, -1).contiguous())
            for got, ref in zip((qr, sr, qc, sc), want):
                assert torch.equal(got, ref)


@pytest.mark.gpu
def test_rows_of_zeros_and_of_other_than_numbers():
    say("case norm of zeros, infinities and NaN")
    for T, H in ((40, 64), (1200, 256), (33, 4096)):
        g = _gen(T)
        x, w = _bf16(g, T, H), torch.ones(H, dtype=BF16, device="cuda")
        want = sl.sl_rmsnorm_fwd_mxfp8(x, w, EPS, cols=False)
        x[3], x[5, 7], x[8, H - 1] = 0, float("nan"), float("inf")
        y, h, rstd = sl.sl_rmsnorm_fwd(x, w, EPS)
        assert not y[3].any() and abs(rstd[3].item() * EPS ** 0.5 - 1) < 1e-6
        assert torch.isnan(y[5]).all() and torch.isnan(y[8, H - 1]) and not y[8, :H - 1].any()      # inf / inf, x / inf
        q, s, _, _, _, _ = sl.sl_rmsnorm_fwd_mxfp8(x, w, EPS, cols=False)
        assert (s[5] == 255).all() and not q[5].any() and s[8, -1] == 255 and not q[8, -32:].any()
        assert not s[3].any() and not q[3].any()
        others = [t for t in range(T) if t not in (3, 5, 8)]
        assert torch.equal(q[others], want[0][others]) and torch.equal(s[others], want[1][others])
        top = T // 32 * 32
        qc, sc = sl.sl_rmsnorm_fwd_mxfp8(x[:top], w, EPS, rows=False)[2:4]
        assert (sc[:, 0] == 255).all() and not qc[:, :32].any() and (sc[:, 1:] != 255).all()
    x = torch.full((2, 64), 2.0 ** -66, dtype=BF16, device="cuda")       # squares below fp32's range
    assert torch.equal(sl.sl_rmsnorm_fwd(x, w[:64], 1.0)[0], x)


@pytest.mark.gpu
@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("T,H", SHAPES + [(5000, 2048)])
def test_gradient(T, H, residual):
    say(f"case norm gradient T={T} H={H} residual={residual}")
    g = _gen(T * H)
    dy, h = _bf16(g, T, H), _bf16(g, T, H)
    dh = _bf16(g, T, H) if residual else None
    w = (1 + 0.2 * torch.randn(H, generator=g, device="cuda")).to(BF16)
    rstd = torch.rsqrt(h.float().square().mean(1) + EPS)
    grad = torch.randn(H, generator=g, device="cuda")
    old = grad.clone()
    dx = sl.sl_rmsnorm_bwd(dy, h, w, rstd, grad, dresidual=dh)
    i, d, hd = rstd.double()[:, None], dy.double(), h.double()
    gg, n = d * w.double(), hd * i
    mean = (gg * n).mean(1, keepdim=True)
    ref = i * (gg - n * mean)
    # the mean: terms of two roundings, at most 53 additions and the division; then two products, a difference, a product
    mean_off = (53 + 4) * U * (gg * n).abs().mean(1, keepdim=True)
    off = i * (n.abs() * (mean_off + 3 * U * mean.abs()) + 3 * U * (gg.abs() + (n * mean).abs()))
    if residual:
        ref = ref + dh.double()
        off = off + U * (ref.abs() + dh.double().abs())
    assert ((dx.double() - ref).abs() <= HALF * (ref.abs() + off) + off).all()
    total = old.double() + (d * n).sum(0)
    # products of two roundings, at most T additions in any order and that to the old value
    assert ((grad.double() - total).abs() <= (T + 3) * U * ((d * n).abs().sum(0) + old.double().abs())).all()
    # the same call gives the same bits; a frozen weight's call the same dX
    again = old.clone()
    assert torch.equal(sl.sl_rmsnorm_bwd(dy, h, w, rstd, again, dresidual=dh), dx) and torch.equal(again, grad)
    assert torch.equal(sl.sl_rmsnorm_bwd(dy, h, w, rstd, None, dresidual=dh), dx)
    if residual:                                                          # into the residual's gradient itself
        assert torch.equal(sl.sl_rmsnorm_bwd(dy, h, w, rstd, None, dresidual=dh, dX=dh), dx)


@pytest.mark.gpu
@pytest.mark.parametrize("T,H", [(1, 8), (100, 72), (1024, 2048), (2500, 264), (300, 4096)])
def test_weight_gradient_of_integers(T, H):
    """rstd = 1/2 and integers: every sum is exact in fp32."""
    say(f"case norm weight gradient of integers T={T} H={H}")
    g = _gen(T)
    dy, h = (torch.randint(-4, 5, (T, H), generator=g, device="cuda").to(BF16) for _ in range(2))
    grad = torch.randint(-4, 5, (H,), generator=g, device="cuda").float()
    want = grad.double() + (dy.double() * h.double()).sum(0) / 2
    sl.sl_rmsnorm_bwd(dy, h, torch.ones(H, dtype=BF16, device="cuda"), torch.full((T,), 0.5, device="cuda"), grad)
    assert torch.equal(grad.double(), want)


@pytest.mark.gpu
def test_gradient_against_differences():
    say("case norm gradient against differences")
    T, H = 6, 40
    x, r, w = _inputs(T, H, True, 2)
    y, h, rstd = sl.sl_rmsnorm_fwd(x, w, EPS, residual=r)
    c, k = _bf16(_gen(3), T, H), _bf16(_gen(4), T, H)                     # gradients of y and of h
    grad = torch.zeros(H, device="cuda")
    dx = sl.sl_rmsnorm_bwd(c, h, w, rstd, grad, dresidual=k).double()

    def loss(hh, ww):
        return ((hh / torch.sqrt(hh.square().mean(1, keepdim=True) + EPS) * ww) * c.double()).sum() + (hh * k.double()).sum()

    h64, w64, step = h.double(), w.double(), 1e-4
    for t, j in ((0, 0), (3, 17), (5, 39)):
        e = torch.zeros_like(h64)
        e[t, j] = step
        slope = ((loss(h64 + e, w64) - loss(h64 - e, w64)) / (2 * step)).item()
        assert abs(dx[t, j].item() - slope) <= HALF * abs(slope) + 1e-5     # differences are off by step^2 times a third derivative
        e = torch.zeros_like(w64)
        e[j] = step
        slope = ((loss(h64, w64 + e) - loss(h64, w64 - e)) / (2 * step)).item()
        assert abs(grad[j].item() - slope) <= 1e-5 * (1 + abs(slope))


@pytest.mark.gpu
def test_empty_extents():
    say("case norm of no tokens")
    w, x = torch.ones(64, dtype=BF16, device="cuda"), torch.zeros((0, 64), dtype=BF16, device="cuda")
    y, h, rstd = sl.sl_rmsnorm_fwd(x, w, EPS, residual=x)
    assert y.shape == h.shape == (0, 64) and rstd.shape == (0,)
    qr, sr, qc, sc, _, _ = sl.sl_rmsnorm_fwd_mxfp8(x, w, EPS)
    assert qr.shape == (0, 64) and sr.shape == (0, 2) and qc.shape == (64, 0) and sc.shape == (64, 0)
    grad = torch.ones(64, device="cuda")
    assert sl.sl_rmsnorm_bwd(x, x, w, rstd, grad).shape == (0, 64) and (grad == 1).all()


@pytest.mark.gpu
def test_autograd():
    say("case norm autograd")
    g = _gen(6)
    x, r = _bf16(g, 2, 50, 136).requires_grad_(), _bf16(g, 2, 50, 136).requires_grad_()
    w = torch.nn.Parameter((1 + 0.1 * torch.randn(136, generator=g, device="cuda")).to(BF16))
    w.main_grad = torch.zeros(136, device="cuda")
    cy, ch = _bf16(g, 2, 50, 136), _bf16(g, 2, 50, 136)
    y, h = sl.rmsnorm_with_grad_accumulation(x, w, r, EPS)
    dx, dr = torch.autograd.grad((y, h), (x, r), (cy, ch))
    assert torch.equal(dx, dr) and w.grad_added_to_main_grad
    _, h2, rstd = sl.sl_rmsnorm_fwd(x.detach().view(100, 136), w.detach(), EPS, residual=r.detach().view(100, 136))
    grad = torch.zeros(136, device="cuda")
    want = sl.sl_rmsnorm_bwd(cy.view(100, 136), h2, w.detach(), rstd, grad, dresidual=ch.view(100, 136))
    assert torch.equal(dx.view(100, 136), want) and torch.equal(w.main_grad, grad)
    # y alone, h alone, no residual, a frozen weight, no gradients at all
    y, h = sl.rmsnorm_with_grad_accumulation(x, w, r, EPS)
    dx, = torch.autograd.grad(y, x, cy)
    assert torch.equal(dx.view(100, 136), sl.sl_rmsnorm_bwd(cy.view(100, 136), h2, w.detach(), rstd, None))
    y, h = sl.rmsnorm_with_grad_accumulation(x, w, r, EPS)
    assert torch.equal(torch.autograd.grad(h, r, ch)[0], ch)
    y = sl.rmsnorm_with_grad_accumulation(x, w, eps=EPS)
    assert torch.autograd.grad(y, x, cy)[0].shape == x.shape
    frozen = w.detach()
    y = sl.rmsnorm_with_grad_accumulation(x, frozen, eps=EPS)
    y.backward(cy)
    assert x.grad is not None
    with torch.no_grad():
        assert not sl.rmsnorm_with_grad_accumulation(x, torch.nn.Parameter(frozen.clone()), r)[0].requires_grad


@pytest.mark.gpu
def test_norm_and_linear_in_mxfp8():
    """The step is the operators one after the other, bit for bit."""
    say("case norm and linear in MXFP8")
    g = _gen(7)
    T, H, O = 256, 384, 640
    x, r = _bf16(g, 2, 128, H).requires_grad_(), _bf16(g, 2, 128, H, std=2.0).requires_grad_()
    buf = sl.ParamAndGradBuffer({"norm": (H,), "fc": (O, H)}, "cuda", bucket_size=None)
    nw = buf.attach("norm", torch.nn.Parameter((1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(BF16)))
    W = buf.attach("fc", torch.nn.Parameter(_bf16(g, O, H, std=0.05)))
    cy, ch = _bf16(g, 2, 128, O), _bf16(g, 2, 128, H)
    y, h = sl.norm_linear_mxfp8_with_grad_accumulation(x, nw, W, r, EPS)
    dx, dr = torch.autograd.grad((y, h), (x, r), (cy, ch))
    got = buf.grad_data.clone()

    flat = lambda t: t.detach().reshape(T, -1)  # noqa: E731
    qr, sr, qc, sc, h2, rstd = sl.sl_rmsnorm_fwd_mxfp8(flat(x), nw.detach(), EPS, residual=flat(r))
    wr, wrs, wc, wcs = sl.sl_mxfp8_quantize(W.detach())
    assert torch.equal(flat(y), sl.sl_linear_fwd_mxfp8(qr, sr, wr, wrs)) and torch.equal(flat(h), h2)
    dq = sl.sl_mxfp8_quantize(flat(cy))
    buf.zero_grad_buffer()
    sl.sl_linear_wgrad_accum_mxfp8(dq[2], dq[3], qc, sc, buf.main_grad("fc"))
    dn = sl.sl_linear_dgrad_mxfp8(dq[0], dq[1], wc, wcs)
    want = sl.sl_rmsnorm_bwd(dn, h2, nw.detach(), rstd, buf.main_grad("norm"), dresidual=flat(ch))
    assert torch.equal(flat(dx), want) and torch.equal(flat(dr), want) and torch.equal(buf.grad_data, got)
    # against 64 bits: MXFP8 keeps 3 bits of mantissa (half a step 2^-4) of both operands, so a sum of K products is off by at
    # most 2 * 2^-4 + 2^-8 of the sum of their magnitudes, and the values that saturate by 1/8 of each more
    hd = h2.double()
    n = hd / torch.sqrt(hd.square().mean(1, keepdim=True) + EPS) * nw.double()
    assert ((flat(y).double() - n @ W.double().t()).abs() <= 0.4 * (n.abs() @ W.double().abs().t())).all()
    # frozen weights, kept copies, and no gradients
    kept = sl.sl_mxfp8_quantize(W.detach())
    buf.zero_grad_buffer()
    y2, _ = sl.norm_linear_mxfp8_with_grad_accumulation(x, nw.detach(), W.detach(), r, EPS, weight_mxfp8=kept)
    dx2, = torch.autograd.grad(y2, x, cy)
    assert torch.equal(y2, y) and not buf.grad_data.any()
    assert torch.equal(flat(dx2), sl.sl_rmsnorm_bwd(dn, h2, nw.detach(), rstd, None))
    with torch.no_grad():
        y3 = sl.norm_linear_mxfp8_with_grad_accumulation(x[:, :5], nw, W)             # 10 tokens: forward alone takes any number
    assert y3.shape == (2, 5, O) and not y3.requires_grad


@pytest.mark.gpu
def test_captured_and_replayed():
    say("case norm graphs")
    g = _gen(12)
    T, H = 1536, 1024
    x, r, w = _inputs(T, H, True, 1)
    dy, grads = _bf16(g, T, H), [torch.zeros(H, device="cuda") for _ in range(2)]

    def work(grad):
        out = sl.sl_rmsnorm_fwd_mxfp8(x, w, EPS, residual=r)
        return out + (sl.sl_rmsnorm_bwd(dy, out[4], w, out[5], grad),)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        work(torch.zeros(H, device="cuda"))
    torch.cuda.current_stream().wait_stream(s)
    graphs, outs = [], []
    for k in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(work(grads[k]))
        graphs.append(graph)
    for k in (0, 1, 1, 0):
        x.copy_(_bf16(g, T, H))
        before = grads[k].clone()
        graphs[k].replay()
        want = work(before)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs[k], want)) and torch.equal(grads[k], before)


def _row_of_integers(h, squares, H):
    """H integers of up to 255, h first, whose squares add up to ``squares``; zeros at the end."""
    row, left = [h], squares - h * h
    while left:
        row.append(min(math.isqrt(left), 100))
        left -= row[-1] ** 2
    return row + [0] * (H - len(row))


# Sums of squares S, h and w for which p = h w lies so that p rstd, S / 4096 + 2^-17 being 1 / rstd^2, is within 2^-25 of a border, and the
# fp32 product with the rounded rstd one unit in the last place away from it: below a power of two with the product above it, and
# above a tie of two codes with the product below it.
@pytest.mark.gpu
@pytest.mark.parametrize("S,h,w", [(126358, 130, 175), (604652, 149, 167), (2225318, 153, 156), (671613, 13, 197), (230861, 13, 231), (59898, 7, 236)])
def test_mxfp8_codes_beside_a_border(S, h, w):
    say(f"case norm mxfp8 beside a border S={S} h={h} w={w}")
    T, H, eps = 32, 4096, 2.0 ** -17
    x = torch.ones((T, H), dtype=BF16, device="cuda")
    x[3] = torch.tensor(_row_of_integers(h, S, H), dtype=BF16, device="cuda")
    weight = torch.full((H,), 2.0 ** -10, dtype=BF16, device="cuda")
    weight[0] = w
    square = Fraction(h * w) ** 2 / (Fraction(S, H) + Fraction(1, 1 << 17))
    exact = 1 / torch.sqrt(x.double().square().mean(1) + eps)[:, None] * x.double() * weight.double()
    v = exact[3, 0].item()
    unit = 2.0 ** (math.floor(math.log2(v)) - (0 if h > 100 else 4))      # borders are whole numbers of it, or twice it
    border = unit * round(v / unit) if round(v / unit) else unit
    assert 0 < abs(square / Fraction(border) ** 2 - 1) < 2.0 ** -24
    assert (square > Fraction(border) ** 2) == (v > border)
    qr, sr, qc, sc, _, _ = sl.sl_rmsnorm_fwd_mxfp8(x, weight, eps)
    _check_mx(qr, sr, exact, 2.0 ** -45)
    _check_mx(qc, sc, exact.t().contiguous(), 2.0 ** -45)


@pytest.mark.parametrize("other", [(256, 64), (128, 96), (64, 128)], ids=["out", "in", "turned"])
def test_mxfp8_copies_of_another_weight_are_refused(other, monkeypatch):
    """Before the norm or anything else runs."""
    from sharded_linear_amd import autograd
    ran = []

    def norm(x, w, eps, residual=None, rows=True, cols=True, out=None, h=None):
        ran.append("norm")
        T, H = x.shape
        return (*_copies(T, H)[:2], *((_copies(T, H)[2:]) if cols else (None, None)), x if h is None else h, torch.zeros(T))

    monkeypatch.setattr(autograd, "sl_rmsnorm_fwd_mxfp8", norm)
    monkeypatch.setattr(autograd, "sl_linear_fwd_mxfp8", lambda q, s, wq, ws, Y=None: torch.zeros((q.shape[0], wq.shape[0]), dtype=BF16) if Y is None else Y)
    monkeypatch.setattr(autograd, "sl_mxfp8_quantize", lambda *a, **k: ran.append("cast"))
    x = torch.zeros((128, 64), dtype=BF16, requires_grad=True)
    nw, w = torch.ones(64, dtype=BF16), torch.nn.Parameter(torch.zeros((128, 64), dtype=BF16))
    w.main_grad = torch.zeros((128, 64))
    call = lambda copies: sl.norm_linear_mxfp8_with_grad_accumulation(x, nw, w, weight_mxfp8=copies)  # noqa: E731
    good, bad = _copies(128, 64), _copies(*other)
    assert call(good).shape == (128, 128) and ran == ["norm"]
    del ran[:]
    for mixed in (bad, good[:2] + bad[2:], bad[:2] + good[2:], good[:3], (None, None) + good[2:]):
        with pytest.raises(ValueError, match="weight_mxfp8"):
            call(mixed)
    with pytest.raises(ValueError, match="columnwise MXFP8"):
        call(good[:2] + (None, None))
    assert not ran
    with torch.no_grad():
        assert call(good[:2] + (None, None)).shape == (128, 128)          # forward alone reads the rowwise copy


def _copies(rows, cols):
    """The shapes of a matrix's MXFP8 copies."""
    u = lambda *s: torch.zeros(s, dtype=U8)  # noqa: E731
    return u(rows, cols), u(rows, cols // 32), u(cols, rows), u(cols, rows // 32)
