"""Orthogonalised updates: refusals on the CPU, iterates and optimiser steps on the GPU against 64 bits."""
import ctypes

import pytest
import torch

import sharded_linear_amd as sl
from sharded_linear_amd import _lib
from tests.gpu_util import say

OK, EINVAL, EALIGN, ESHAPE, EWORKSPACE = 0, -1, -2, -3, -4
A = 1 << 20          # an aligned fake device address, never dereferenced
BF16, F32 = torch.bfloat16, torch.float32
COEFFS = (3.4445, -4.7750, 2.0315)
# The 2-norm of an iterate's error over that of the iterate.  An element is rounded to fp16 within half a step, 2^-11, so the
# roundings of one matrix are 2^-11 / sqrt(3) = 2.8e-4 of its norm.  With singular values near 1, X moves by at most
# |b + 2 c| = 0.7 .. 4.8 times what A moves by, by up to 2.8 times the relative change of b A + c A^2, and a change of X grows by
# up to a = 3.4 a step while its singular value is small and by less than 1 later: three last steps of 2.8e-4 (1 + 4.8 + 2.8), added
# as squares, are 4.2e-3 at most.
OFF = 4.2e-3
BF16_OFF = 2.0 ** -8 / 3 ** 0.5      # the rounding of the result, as a 2-norm


def _arr(*v):
    return (ctypes.c_float * len(v))(*v)


def test_orthogonalize_validation():
    L = _lib.lib()
    f, ws = L.sl_orthogonalize, L.sl_orthogonalize_workspace_bytes
    need = ws(2, 100, 60)
    k = _arr(*COEFFS * 5)
    assert need > 0 and ws(0, 5, 5) == 0 and ws(1, 0, 5) == 0 and ws(-1, 5, 5) == 0 and ws(1, 1 << 31, 5) == 0
    assert ws(1, (1 << 31) - 1, (1 << 31) - 1) == 0 and ws(1 << 30, 8, 8) == 0
    assert f(None, A, 4, A, 2, 100, 60, 5, k, A, need - 1) == EWORKSPACE
    assert f(None, A, 4, A, 2, 100, 60, 5, k, None, 0) == EWORKSPACE
    assert f(None, A, 4, A, 2, 100, 60, 5, k, A + 8, need) == EWORKSPACE
    assert f(None, A, 3, A, 2, 100, 60, 5, k, A, need) == EINVAL
    assert f(None, A, 4, A, 2, 100, 60, -1, k, A, need) == EINVAL
    assert f(None, A, 4, A, 2, 100, 60, 65, k, A, need) == EINVAL
    assert f(None, A, 4, A, 2, 100, 60, 5, None, A, need) == EINVAL
    assert f(None, A, 4, A, -1, 100, 60, 5, k, A, need) == EINVAL
    assert f(None, None, 4, A, 2, 100, 60, 5, k, A, need) == EINVAL
    assert f(None, A, 4, None, 2, 100, 60, 5, k, A, need) == EINVAL
    assert f(None, A + 4, 4, A, 2, 100, 60, 5, k, A, need) == EALIGN
    assert f(None, A, 4, A + 4, 2, 100, 60, 5, k, A, need) == EALIGN
    assert f(None, A, 4, A, 1, 1 << 20, 1 << 20, 5, k, A, 1 << 62) == ESHAPE
    assert f(None, A, 4, A, 70000, 8, 8, 5, k, A, 1 << 62) == ESHAPE
    assert f(None, None, 4, None, 0, 100, 60, 5, k, None, 0) == OK
    assert f(None, None, 4, None, 2, 0, 60, 5, k, None, 0) == OK


@pytest.mark.parametrize("k,ok", [((3.4445, -4.7750, 2.0315), True), ((1.5, -0.5, 0.0), True), ((1.875, -1.25, 0.375), True), ((1.0, 0.0, 0.0), True),
                                  ((8.28749, -23.5959, 17.3004), True), ((4.0, 0.0, 0.0), False), ((2.0, 1.5, 0.0), False), ((3.4445, -4.7750, 12.0), False),
                                  ((9.0, -20.0, 12.5), True), ((float("nan"), 0.0, 0.0), False), ((1.0, 30.0, -30.0), False)])
def test_coefficients_that_leave_the_range_are_refused(k, ok):
    """One step of each from singular values in [0, 1]: below 3, and a + b z + c z^2 below 15."""
    f = _lib.lib().sl_orthogonalize
    s = torch.linspace(0, 1, 100001, dtype=torch.float64)
    if ok:
        assert (k[0] * s + k[1] * s ** 3 + k[2] * s ** 5).abs().max() <= 3 and (k[0] + k[1] * s ** 2 + k[2] * s ** 4).abs().max() <= 15
    assert f(None, None, 4, None, 0, 8, 8, 1, _arr(*k), None, 0) == (OK if ok else EINVAL)


def test_coefficients_are_followed_over_the_steps():
    f = _lib.lib().sl_orthogonalize
    double = (2.0, 0.0, 0.0)
    assert f(None, None, 4, None, 0, 8, 8, 1, _arr(*double), None, 0) == OK
    assert f(None, None, 4, None, 0, 8, 8, 2, _arr(*double * 2), None, 0) == EINVAL        # singular values of 4
    assert f(None, None, 4, None, 0, 8, 8, 2, _arr(*double, 0.5, 0.0, 0.0), None, 0) == OK


def test_muon_validation():
    L = _lib.lib()
    f = L.sl_muon_step
    need = L.sl_orthogonalize_workspace_bytes(2, 100, 60)
    P = lambda *v: (ctypes.c_void_p * len(v))(*v)  # noqa: E731
    k = _arr(*COEFFS * 5)
    good = P(A, A)
    tail = (0.1, 0.9, 1, 0.0, 1.0, 5, k, A)
    assert f(None, good, None, good, good, 2, 100, 60, *tail, need - 1) == EWORKSPACE
    assert f(None, None, None, good, good, 2, 100, 60, *tail, need) == EINVAL
    assert f(None, good, None, None, good, 2, 100, 60, *tail, need) == EINVAL
    assert f(None, good, None, good, None, 2, 100, 60, *tail, need) == EINVAL
    assert f(None, P(A, None), None, good, good, 2, 100, 60, *tail, need) == EINVAL
    assert f(None, good, P(A, None), good, good, 2, 100, 60, *tail, need) == EINVAL
    assert f(None, P(A, A + 8), None, good, good, 2, 100, 60, *tail, need) == EALIGN
    assert f(None, good, P(A, A + 8), good, good, 2, 100, 60, *tail, need) == EALIGN
    for j in (0, 1, 3, 4):
        t = list(tail)
        t[j] = float("inf")
        assert f(None, good, None, good, good, 2, 100, 60, *t, need) == EINVAL, j
    assert f(None, None, None, None, None, 0, 100, 60, *tail, 0) == OK


def test_binding_refusals(monkeypatch):
    from sharded_linear_amd import ops
    with pytest.raises(ValueError, match="GPU tensors"):
        sl.sl_orthogonalize(torch.zeros(4, 4))
    monkeypatch.setattr(ops, "_device", lambda t: t.device)
    G = torch.zeros(4, 6)
    for bad in (G.half(), G[0], G[None, None]):
        with pytest.raises(ValueError, match="G must be"):
            sl.sl_orthogonalize(bad)
    with pytest.raises(ValueError, match="contiguous"):
        sl.sl_orthogonalize(G.t())
    with pytest.raises(ValueError, match="coefficients"):
        sl.sl_orthogonalize(G, steps=2, coefficients=[COEFFS] * 3)
    with pytest.raises(ValueError, match="steps"):
        sl.sl_orthogonalize(G, steps=-1)
    w, m = torch.zeros(4, 6, dtype=BF16), torch.zeros(4, 6)
    with pytest.raises(ValueError, match="number"):
        sl.sl_muon_step([w, w.clone()], [G], [m], 0.1)
    with pytest.raises(TypeError, match="main_grad"):
        sl.sl_muon_step(w, w, m, 0.1)
    with pytest.raises(ValueError, match="weight has shape"):
        sl.sl_muon_step([w, w[:3]], [G, G], [m, m.clone()], 0.1)
    with pytest.raises(ValueError, match="twice"):
        sl.sl_muon_step([w, w], [G, G], [m, m.clone()], 0.1)
    with pytest.raises(ValueError, match="twice"):
        sl.sl_muon_step([w], [G], [G], 0.1)
    assert sl.sl_muon_step([], [], [], 0.1) is None


@pytest.mark.parametrize("weights,grads,momenta,masters,ok", [
    ((0, 24), (0, 24), (100, 124), None, True),          # neighbours
    ((0, 24), (0, 0), (100, 124), None, True),           # one gradient for both
    ((0, 23), (0, 24), (100, 124), None, False),         # weights overlap
    ((0, 24), (0, 24), (100, 120), None, False),         # momenta overlap
    ((0, 24), (0, 24), (100, 47), None, False),          # a momentum over a gradient
    ((0, 24), (0, 24), (100, 124), (148, 172), True),
    ((0, 24), (0, 24), (100, 124), (148, 171), False),   # masters overlap
    ((0, 24), (0, 24), (100, 124), (76, 148), True),     # a master just before a momentum
    ((0, 24), (0, 24), (100, 124), (77, 148), False),    # and over its first element
])
def test_overlaps_are_refused(weights, grads, momenta, masters, ok, monkeypatch):
    """Matrices of 24 elements that begin at the given elements of one fp32 and one bf16 array."""
    from sharded_linear_amd import ops
    monkeypatch.setattr(ops, "_device", lambda t: t.device)
    monkeypatch.setattr(ops, "_scratch", lambda *a: (None, 0))
    monkeypatch.setattr(ops, "_launch", lambda *a: None)
    data, params = torch.zeros(300), torch.zeros(300, dtype=BF16)
    at = lambda a, starts: None if starts is None else [a[k:k + 24].view(4, 6) for k in starts]  # noqa: E731
    args = at(params, weights), at(data, grads), at(data, momenta), 0.1
    if ok:
        sl.sl_muon_step(*args, masters=at(data, masters))
    else:
        with pytest.raises(ValueError, match="overlaps"):
            sl.sl_muon_step(*args, masters=at(data, masters))


# ---- on the GPU -----------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def _iterate(u, steps=5, coefficients=COEFFS):
    """Newton-Schulz in float64 of one matrix."""
    u = u.double()
    n = u.norm()
    x = u / n if n > 0 else u
    tall = x.shape[0] > x.shape[1]
    x = x.t().contiguous() if tall else x
    ks = [coefficients] * steps if len(coefficients) == 3 and not isinstance(coefficients[0], (tuple, list)) else coefficients
    for a, b, c in ks:
        A = x @ x.t().contiguous()
        x = a * x + (b * A + c * (A @ A)) @ x
    return x.t() if tall else x


def _off(got, ref):
    return ((got.double() - ref).norm() / ref.norm()).item()


def _bound(shape=(16, 16)):
    """Of fewer than 16 rows or columns nothing averages out: every rounding counts with its whole half step, and they add up:
    three steps of 2^-11 (1 + 4.8 + 2.8), and the result's 2^-8."""
    return (OFF ** 2 + BF16_OFF ** 2) ** 0.5 if min(shape[-2:]) >= 16 else 3 * 2.0 ** -11 * 8.6 + 2.0 ** -8


# below one tile, at and across the tiles' edges, odd rows, wide, tall, one row, one column
SHAPES = [(1, 1), (1, 300), (300, 1), (3, 5), (16, 16), (63, 65), (64, 128), (127, 129), (128, 128), (257, 100), (130, 1000), (1000, 131), (384, 384), (512, 256),
          (250, 2000), (640, 1160), (1024, 1024)]


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("rows,cols", SHAPES)
def test_orthogonalize(rows, cols, dtype):
    say(f"case orthogonalize [{rows}, {cols}] {dtype}")
    G = (_randn(_gen(rows + cols), rows, cols) * 1e-4).to(dtype)
    O = sl.sl_orthogonalize(G)
    assert O.dtype is BF16 and O.shape == G.shape
    assert _off(O, _iterate(G)) <= _bound(G.shape)


@pytest.mark.gpu
@pytest.mark.parametrize("L,rows,cols", [(2, 5, 7), (3, 65, 130), (7, 200, 100), (33, 24, 40), (70, 10, 9), (5, 513, 515)])
def test_batches(L, rows, cols):
    say(f"case orthogonalize {L} x [{rows}, {cols}]")
    G = _randn(_gen(L), L, rows, cols) * torch.logspace(-8, 8, L, device="cuda")[:, None, None]     # each has its own norm
    O = sl.sl_orthogonalize(G)
    for l in range(L):
        assert _off(O[l], _iterate(G[l])) <= _bound(G.shape), l
    one = sl.sl_orthogonalize(G[L - 1].clone())
    assert _off(one, O[L - 1].double()) <= 2 * _bound(G.shape)


@pytest.mark.gpu
@pytest.mark.parametrize("rows,cols", [(2048, 2048), (4104, 300), (300, 4104), (1536, 2048), (2304, 2816)])
def test_large_tiles(rows, cols):
    say(f"case orthogonalize [{rows}, {cols}]")
    G = _randn(_gen(rows), 3, rows, cols)
    O = sl.sl_orthogonalize(G)
    for l in range(3):
        assert _off(O[l], _iterate(G[l])) <= _bound()
    assert torch.equal(sl.sl_orthogonalize(G), O)


@pytest.mark.gpu
@pytest.mark.parametrize("L,rows,cols", [(50, 640, 640), (60, 600, 520), (9, 1408, 1300), (1, 1800, 5000), (2, 4096, 2048)])
def test_rounds_of_tiles(L, rows, cols):
    """Products of whole rounds of the largest tiles with quarters for the rest, tiles half outside the matrix among them, and split
    sums of either."""
    say(f"case orthogonalize {L} x [{rows}, {cols}]")
    G = _randn(_gen(L), L, rows, cols)
    O = sl.sl_orthogonalize(G)
    for l in range(L):
        assert _off(O[l], _iterate(G[l])) <= _bound(), l
    assert torch.equal(sl.sl_orthogonalize(G), O)


@pytest.mark.gpu
def test_singular_values_over_decades():
    """Where singular values fall over four decades and over two steps of rank, the small ones are reached as the formula
    has it: a rounding of X would be multiplied by up to 3.4^5 there, but the first three steps carry what it left."""
    say("case orthogonalize falling singular values")
    g = _gen(4)
    m, n = 256, 640
    U = torch.linalg.qr(_randn(g, m, m).double())[0]
    V = torch.linalg.qr(_randn(g, n, m).double())[0]
    for s in (torch.logspace(0, -4, m, device="cuda").double(), torch.where(torch.arange(m, device="cuda") < m // 4, 1.0, 1e-3).double()):
        G = ((U * s) @ V.t()).float()
        for x in (G, G.t().contiguous()):
            assert _off(sl.sl_orthogonalize(x), _iterate(x)) <= _bound()


@pytest.mark.gpu
def test_steps_and_coefficients():
    say("case orthogonalize steps and coefficients")
    G = _randn(_gen(5), 200, 333)
    for steps in (0, 1, 2, 3, 4, 8):
        assert _off(sl.sl_orthogonalize(G, steps=steps), _iterate(G, steps)) <= _bound(), steps
    ks = [(3.4445, -4.7750, 2.0315)] * 3 + [(1.875, -1.25, 0.375)] * 2
    assert _off(sl.sl_orthogonalize(G, coefficients=ks), _iterate(G, 5, ks)) <= _bound()
    ks = [(1.5, -0.5, 0.0)] * 14                                               # the cubic iteration, to convergence
    O = sl.sl_orthogonalize(G, steps=14, coefficients=(1.5, -0.5, 0.0))
    assert _off(O, _iterate(G, 14, ks)) <= _bound()
    assert (O.double() @ O.double().t() - torch.eye(200, device="cuda", dtype=torch.float64)).norm() / 200 ** 0.5 <= 3 * _bound()


@pytest.mark.gpu
@pytest.mark.parametrize("power", [-100, -60, 60, 110])
def test_any_magnitude(power):
    """The norm is a sum in 64 bits: the scale of a gradient, a power of two, changes no bit of the result."""
    say(f"case orthogonalize 2^{power}")
    G = _randn(_gen(6), 70, 50)
    assert torch.equal(sl.sl_orthogonalize(G * 2.0 ** power), sl.sl_orthogonalize(G))


@pytest.mark.gpu
def test_zeros_and_other_than_numbers():
    say("case orthogonalize zeros, infinities and NaN")
    G = _randn(_gen(7), 4, 100, 150)
    want = sl.sl_orthogonalize(G)
    G[1], G[2, 5, 7], G[3, 99, 149] = 0, float("nan"), float("inf")
    O = sl.sl_orthogonalize(G)
    assert torch.equal(O[0], want[0]) and not O[1].any()
    assert torch.isnan(O[2]).all() and torch.isnan(O[3]).any()


def _muon(W, G, M, lr, mu, nesterov, wd, scale):
    """The step in float64: new momentum and new weight."""
    M = mu * M.double() + G.double()
    U = G.double() + mu * M if nesterov else M
    return M, (1 - lr * wd) * W.double() - lr * scale * _iterate(U)


@pytest.mark.gpu
@pytest.mark.parametrize("nesterov", [True, False])
@pytest.mark.parametrize("rows,cols,count", [(100, 60, 1), (61, 130, 3), (512, 256, 2), (24, 40, 40)])
def test_muon_step(rows, cols, count, nesterov):
    say(f"case muon {count} x [{rows}, {cols}] nesterov={nesterov}")
    g = _gen(rows)
    W = [(_randn(g, rows, cols) * 0.02).to(BF16) for _ in range(count)]
    masters = [w.float() + 1e-5 * _randn(g, rows, cols) for w in W]
    G = [_randn(g, rows, cols) * 1e-3 for _ in range(count)]
    M = [_randn(g, rows, cols) * 1e-2 for _ in range(count)]
    lr, mu, wd = 0.02, 0.9, 0.1
    scale = max(1.0, rows / cols) ** 0.5
    want = [_muon(w, x, m, lr, mu, nesterov, wd, scale) for w, x, m in zip(W, G, M)]
    kept = [_muon(w, x, m, lr, mu, nesterov, wd, 0.3) for w, x, m in zip(masters, G, M)]
    W2, M2, kept_g = [w.clone() for w in W], [m.clone() for m in M], [x.clone() for x in G]
    mass = [(mu * m.abs() + x.abs()).double() for m, x in zip(M, G)]
    assert sl.sl_muon_step(W, G, M, lr, momentum=mu, nesterov=nesterov, weight_decay=wd) is None
    for l in range(count):
        assert ((M[l].double() - want[l][0]).abs() <= 2 * 2.0 ** -24 * mass[l]).all()
        step = (lr * scale * _iterate(G[l].double() + mu * want[l][0] if nesterov else want[l][0])).norm()
        # half a bf16 step of every weight, and the iterate's error times lr scale
        assert (W[l].double() - want[l][1]).norm() <= 2.0 ** -8 * want[l][1].norm() + OFF * step
        assert torch.equal(G[l], kept_g[l])
    # fp32 masters take the step; the bf16 weights are their rounding
    sl.sl_muon_step(W2, G, M2, lr, momentum=mu, nesterov=nesterov, weight_decay=wd, scale=0.3, masters=masters)
    for l in range(count):
        assert torch.equal(M2[l], M[l]) and torch.equal(W2[l], masters[l].to(BF16))
        step = (lr * 0.3 * _iterate(G[l].double() + mu * want[l][0] if nesterov else want[l][0])).norm()
        assert (masters[l].double() - kept[l][1]).norm() <= 4 * 2.0 ** -24 * kept[l][1].norm() + OFF * step


@pytest.mark.gpu
def test_muon_on_the_buffer():
    """Weights of three shapes in one buffer, stepped from grad_data into param_data; what is not named stays."""
    say("case muon on the buffer")
    g = _gen(9)
    shapes = {"a": (136, 72), "b": (72, 136), "c": (136, 72), "norm": (136,), "d": (64, 64)}
    buf = sl.ParamAndGradBuffer(shapes, "cuda", bucket_size=None)
    buf.param_data.copy_((_randn(g, buf.numel) * 0.02).to(BF16))
    buf.grad_data.copy_(_randn(g, buf.numel) * 1e-3)
    momentum = torch.zeros_like(buf.grad_data)
    old, names = buf.param_data.clone(), ["a", "b", "c", "d"]
    want = {n: _muon(buf.param(n), buf.main_grad(n), torch.zeros(shapes[n], device="cuda"), 0.05, 0.95, True, 0.01,
                     max(1.0, shapes[n][0] / shapes[n][1]) ** 0.5) for n in names}
    buf.muon_step(names, momentum, 0.05, weight_decay=0.01)
    inside = torch.zeros(buf.numel, dtype=torch.bool, device="cuda")
    for n in names:
        s, e, _ = buf.index[n]
        inside[s:e] = True
        assert torch.equal(momentum[s:e], buf.grad_data[s:e])
        step = (want[n][1] - old[s:e].view(shapes[n]).double()).norm()
        assert (buf.param(n).double() - want[n][1]).norm() <= 2.0 ** -8 * want[n][1].norm() + OFF * step
    assert torch.equal(buf.param_data[~inside], old[~inside]) and not momentum[~inside].any()
    with pytest.raises(ValueError, match="momentum_data"):
        buf.muon_step(names, momentum[:-1], 0.05)


@pytest.mark.gpu
def test_empty_extents():
    say("case orthogonalize nothing")
    assert sl.sl_orthogonalize(torch.zeros((0, 5, 6), device="cuda")).shape == (0, 5, 6)
    assert sl.sl_orthogonalize(torch.zeros((2, 0, 6), device="cuda")).shape == (2, 0, 6)
    w, g, m = (torch.zeros((0, 6), device="cuda", dtype=t) for t in (BF16, torch.float32, torch.float32))
    sl.sl_muon_step([w, w], [g, g], [m, m], 0.1)


@pytest.mark.gpu
def test_captured_and_replayed():
    say("case muon graphs")
    g = _gen(10)
    G = _randn(g, 2, 300, 200)
    W, M = (_randn(g, 300, 200) * 0.02).to(BF16), torch.zeros((300, 200), device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sl.sl_orthogonalize(G)
        sl.sl_muon_step(W.clone(), G[0].clone(), M.clone(), 0.1)
    torch.cuda.current_stream().wait_stream(s)
    grad = G[0].clone()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    with torch.cuda.graph(graphs[0]):
        O = sl.sl_orthogonalize(G)
    with torch.cuda.graph(graphs[1]):
        sl.sl_muon_step(W, grad, M, 0.1)
    for r in range(3):
        G.copy_(_randn(g, 2, 300, 200))
        grad.copy_(G[1])
        W2, M2 = W.clone(), M.clone()
        graphs[r % 2].replay()
        graphs[1 - r % 2].replay()
        sl.sl_muon_step(W2, grad, M2, 0.1)
        want = sl.sl_orthogonalize(G)
        torch.cuda.synchronize()
        assert torch.equal(O, want) and torch.equal(W, W2) and torch.equal(M, M2)


# ---- the ways in which the tiled products are taken apart ------------------------------------------

# Ragged, so that padding is in every plan; as (L, rows, cols).
PLANS = [(1, 384, 380), (1, 512, 600), (1, 400, 760), (1, 850, 1000), (3, 3195, 890), (24, 1024, 1277), (12, 1400, 1390), (8, 2048, 2040), (4, 2680, 3570),
         (11, 1790, 1700), (4, 2944, 2900), (3, 1402, 3190), (4, 1024, 4090), (3, 1660, 3710), (3, 3330, 1790), (2, 2175, 4090), (2, 2040, 4200),
         (2, 2688, 3199)]


def _forms(L, rows, cols):
    """For each product of a step: its name, the tiles that it is taken apart into, and whether tiles of 256 lie half outside it."""
    m, n = (-(-min(rows, cols) // 128) * 128, -(-max(rows, cols) // 128) * 128)
    for name, (big, small, split, parts), wide in zip(("X X^T", "A A", "P X"), sl.sl_orthogonalize_tiles(L, rows, cols), (m, m, n)):
        assert (split > 0) == (parts > 1) and split <= small
        tiles = "128" if not big else "256" if not small else "both"
        yield name, tiles + (" split" if split else ""), bool(big and m % 256), bool(big and wide % 256)


def test_plans_cover_every_form():
    """The shapes that the GPU tests below run: a cost model that is fitted anew must not leave one of these without a test."""
    seen = {f for plan in PLANS for f in _forms(*plan)}
    tiles = {(name, t) for name, t, _, _ in seen}
    for name in ("X X^T", "A A", "P X"):
        for t in ("128", "128 split", "256", "both", "both split"):
            assert (name, t) in tiles, (name, t)
    for t in ("256", "both"):
        assert ("X X^T", t, True, True) in seen and ("A A", t, True, True) in seen, t
    assert ("X X^T", "both split", True, True) in seen
    for t in ("256", "both", "both split"):
        assert {(m, n) for name, u, m, n in seen if name == "P X" and u == t} >= {(True, True)}, t
    assert {(m, n) for name, _, m, n in seen if name == "P X"} == {(False, False), (False, True), (True, False), (True, True)}
    assert sl.sl_orthogonalize_tiles(1, 100, 60) is None and sl.sl_orthogonalize_tiles(0, 512, 512) is None
    with pytest.raises(RuntimeError):
        sl.sl_orthogonalize_tiles(1, 1 << 31, 5)


def _cosines(g, n, k):
    """k orthonormal columns of n elements: cosines under random signs (float64)."""
    i, j = torch.arange(n, device="cuda").double()[:, None], torch.arange(k, device="cuda").double()
    c = torch.cos(torch.pi / n * (i + 0.5) * j) * (2 / n) ** 0.5
    c[:, 0] = n ** -0.5
    signs = torch.randint(0, 2, (n, 1), generator=g, device="cuda").double() * 2 - 1
    return c * signs


def _falling(g, rows, cols, s):
    """A matrix with the singular values s."""
    k = min(rows, cols)
    return ((_cosines(g, rows, k) * s) @ _cosines(g, cols, k).t().contiguous()).float()


def _decades(k, how):
    at = torch.arange(k, device="cuda").double()
    return 10.0 ** (-4 * at / max(1, k - 1)) if how == "logarithmic" else torch.where(at < k // 4, 1.0, 1e-3).double()


@pytest.mark.gpu
@pytest.mark.parametrize("how", ["logarithmic", "two steps"])
@pytest.mark.parametrize("L,rows,cols", [(1, 384, 640), (3, 640, 384), (1, 100, 640), (3, 640, 100), (2, 33, 70), (3, 250, 500), (5, 128, 128),
                                         (2, 1000, 1160)])
def test_falling_singular_values(L, rows, cols, how):
    """As test_singular_values_over_decades, whose matrices have 256 rows: fewer rows, tiles, batches, tall and wide.  By the argument
    there the bound is the same; without what the roundings of X left, [384, 640] is 7.5e-3 off."""
    say(f"case orthogonalize falling singular values {L} x [{rows}, {cols}] {how}")
    g = _gen(L * rows + cols)
    G = torch.stack([_falling(g, rows, cols, _decades(min(rows, cols), how)) for _ in range(L)])
    O = sl.sl_orthogonalize(G)
    for l in range(L):
        assert _off(O[l], _iterate(G[l])) <= _bound(), l


@pytest.mark.gpu
@pytest.mark.parametrize("L,rows,cols", PLANS)
def test_every_form_of_tiles(L, rows, cols):
    """Matrices with falling singular values among normal ones."""
    say(f"case orthogonalize {L} x [{rows}, {cols}] {list(_forms(L, rows, cols))}")
    g = _gen(L + rows)
    G = torch.stack([_randn(g, rows, cols) if l % 2 else _falling(g, rows, cols, _decades(min(rows, cols), "logarithmic")) for l in range(L)])
    O = sl.sl_orthogonalize(G)
    for l in range(L):
        assert _off(O[l], _iterate(G[l])) <= _bound(), l
    assert torch.equal(sl.sl_orthogonalize(G), O)


# ---- a step on the buffer is refused as a whole ----------------------------------------------------

def _host_buffer(monkeypatch, shapes, **kw):
    """A buffer on the host, and the list of the calls that would be launched on it."""
    from sharded_linear_amd import ops
    calls = []
    monkeypatch.setattr(ops, "_device", lambda t: t.device)
    monkeypatch.setattr(ops, "_launch", lambda name, dev, *a: calls.append((name, *a)))
    monkeypatch.setattr(ops, "_scratch", lambda dev, need, ws: (ws, need if ws is None else ws.numel()))
    buf = sl.ParamAndGradBuffer(shapes, "cpu", bucket_size=None, **kw)
    return buf, torch.zeros_like(buf.grad_data), calls


SHAPES_OF_TWO = {"fc": (24, 16), "norm": (24,), "out": (16, 24), "fc2": (24, 16)}


@pytest.mark.parametrize("names,options,match", [
    (["fc", "norm"], {}, "matrix"),
    (["fc", "out", "fc"], {}, "twice"),
    (["fc", "out", "missing"], {}, "missing"),
    (["fc", "out"], {"momentum_data": torch.zeros(10)}, "momentum_data"),
    (["fc", "out"], {"momentum_data": "bf16"}, "momentum"),
    (["fc", "out"], {"masters": [torch.zeros(24, 16)]}, "1 masters of 2"),
    (["fc", "out"], {"masters": [torch.zeros(24, 16), torch.zeros(24, 16)]}, "shape"),
    (["fc", "out"], {"masters": torch.zeros(10)}, "masters"),
    (["fc", "out"], {"masters": "momenta"}, "twice"),
    (["fc", "out"], {"workspace": torch.zeros(16, dtype=torch.uint8)}, "EWORKSPACE"),
    (["fc", "out"], {"other": 1}, "other"),
])
def test_step_on_the_buffer_is_refused_before_anything_is_launched(names, options, match, monkeypatch):
    buf, momentum, calls = _host_buffer(monkeypatch, SHAPES_OF_TWO)
    options = dict(options)
    momentum = options.pop("momentum_data", momentum)
    if isinstance(momentum, str):
        momentum = torch.zeros_like(buf.param_data)
    if isinstance(options.get("masters"), str):
        options["masters"] = momentum
    with pytest.raises((ValueError, TypeError, KeyError, RuntimeError), match=match):
        buf.muon_step(names, momentum, 0.1, **options)
    assert not calls


def test_step_on_a_buffer_without_alignment_is_refused_as_a_whole(monkeypatch):
    buf, momentum, calls = _host_buffer(monkeypatch, {"b": (3, 5), "a": (16, 24)}, param_align=1)
    assert buf.main_grad("b").data_ptr() % 16 == 0 and buf.param("b").data_ptr() % 16 == 0
    buf, momentum, calls = _host_buffer(monkeypatch, {"c": (3, 4), "b": (3, 5), "a": (16, 24)}, param_align=1)
    with pytest.raises(RuntimeError, match="EALIGN"):
        buf.muon_step(["a", "c"], momentum, 0.1)
    assert not calls
    buf.muon_step(["a", "b"], momentum, 0.1)
    assert [c[0] for c in calls] == ["sl_muon_step"] * 2


def test_masters_go_with_their_names(monkeypatch):
    """As a buffer, as a list in the names' order, and one for one name; weights of two shapes in turn."""
    buf, momentum, calls = _host_buffer(monkeypatch, SHAPES_OF_TWO)
    flat = torch.zeros_like(buf.grad_data)
    at = lambda data, n: data[buf.index[n][0]:buf.index[n][1]].view(buf.shapes[n])  # noqa: E731
    names = ["fc", "out", "fc2"]
    want = [[at(flat, "fc").data_ptr(), at(flat, "fc2").data_ptr()], [at(flat, "out").data_ptr()]]
    for masters in (flat, [at(flat, n) for n in names]):
        calls.clear()
        buf.muon_step(names, momentum, 0.1, masters=masters)
        assert [list(c[2]) for c in calls] == want
        assert [list(c[1]) for c in calls] == [[buf.param("fc").data_ptr(), buf.param("fc2").data_ptr()], [buf.param("out").data_ptr()]]
    calls.clear()
    buf.muon_step(["out"], momentum, 0.1, masters=at(flat, "out"))
    assert [list(c[2]) for c in calls] == [want[1]]


@pytest.mark.gpu
def test_masters_on_the_buffer():
    say("case muon on the buffer with masters")
    g = _gen(13)
    shapes = {"a": (136, 72), "norm": (136,), "b": (72, 136), "c": (136, 72)}
    buf = sl.ParamAndGradBuffer(shapes, "cuda", bucket_size=None)
    buf.grad_data.copy_(_randn(g, buf.numel) * 1e-3)
    flat = _randn(g, buf.numel) * 0.02
    buf.param_data.copy_(flat)
    old, kept, names, momentum = buf.param_data.clone(), flat.clone(), ["a", "b", "c"], torch.zeros_like(buf.grad_data)
    buf.muon_step(names, momentum, 0.05, masters=flat, weight_decay=0.01)
    for n in names:
        s, e, _ = buf.index[n]
        w, p, m = (t[s:e].clone().view(shapes[n]) for t in (old, kept, torch.zeros_like(momentum)))
        sl.sl_muon_step(w, buf.main_grad(n), m, 0.05, masters=p, weight_decay=0.01)
        # alone a matrix takes other tiles than in its group: both are within the iterate's error of the formula
        step = (p.double() - kept[s:e].view(shapes[n]).double()).norm()
        assert (flat[s:e].view(shapes[n]).double() - p.double()).norm() <= 2 * OFF * step
        assert torch.equal(buf.param(n), flat[s:e].view(shapes[n]).to(BF16)) and torch.equal(momentum[s:e], m.view(-1))
    s, e, _ = buf.index["norm"]
    assert torch.equal(flat[s:e], kept[s:e]) and torch.equal(buf.param_data[s:e], old[s:e])


def test_a_graph_that_saved_a_weight_notices_its_step(monkeypatch):
    """The step writes through addresses; autograd has to learn of it all the same."""
    from sharded_linear_amd import ops
    monkeypatch.setattr(ops, "_device", lambda t: t.device)
    monkeypatch.setattr(ops, "_launch", lambda *a: None)
    monkeypatch.setattr(ops, "_scratch", lambda *a: (None, 0))
    w = torch.nn.Parameter(torch.ones((16, 24), dtype=BF16))
    x = torch.ones((4, 24), dtype=BF16, requires_grad=True)
    M, G, master = (torch.zeros((16, 24)) for _ in range(3))
    y = x @ w.t()
    before = [t._version for t in (M, G, master)]
    sl.sl_muon_step(w, G, M, 0.1, masters=master)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()
    assert [t._version for t in (M, G, master)] == [before[0] + 1, before[1], before[2] + 1]
    (x @ w.t()).sum().backward()                                          # a graph made after the step
    with torch.inference_mode():
        inside = torch.ones((16, 24), dtype=BF16)
        sl.sl_muon_step(inside, G, M, 0.1)
    buf, momentum, _ = _host_buffer(monkeypatch, SHAPES_OF_TWO)
    y = x @ buf.param("out").t()
    buf.muon_step(["out"], momentum, 0.1)
    with pytest.raises(RuntimeError, match="inplace"):
        y.sum().backward()


# ---- matrices at any address ----------------------------------------------------------------------

def test_alignment_of_matrices():
    """Rows of whole groups of four elements are loaded by groups, others element by element."""
    L = _lib.lib()
    f, k = L.sl_orthogonalize, _arr(*COEFFS * 5)
    for cols, g_bytes, at, ok in ((61, 4, 4, True), (61, 4, 2, False), (61, 2, 2, True), (61, 2, 1, False), (62, 4, 8, True), (60, 4, 8, False),
                                  (64, 2, 8, False)):
        assert f(None, A + at, g_bytes, A, 1, 100, cols, 5, k, None, 0) == (EWORKSPACE if ok else EALIGN), (cols, at)
    assert f(None, A, 4, A + 2, 1, 100, 61, 5, k, None, 0) == EWORKSPACE and f(None, A, 4, A + 1, 1, 100, 61, 5, k, None, 0) == EALIGN
    P = lambda *v: (ctypes.c_void_p * len(v))(*v)  # noqa: E731
    step = lambda cols, *at: L.sl_muon_step(None, P(A + at[0]), P(A + at[1]), P(A + at[2]), P(A + at[3]), 1, 100, cols, 0.1, 0.9, 1,  # noqa: E731
                                            0.0, 1.0, 5, k, None, 0)
    assert step(61, 2, 4, 12, 8) == EWORKSPACE and step(60, 16, 32, 0, 16) == EWORKSPACE
    odd = lambda w, g: L.sl_muon_step(None, P(A + w), None, P(A + g), P(A), 1, 33, 12, 0.1, 0.9, 1, 0.0, 1.0, 5, k, None, 0)  # noqa: E731
    assert odd(8, 0) == EWORKSPACE and odd(4, 0) == EALIGN and odd(0, 8) == EALIGN
    assert f(None, A + 8, 2, A + 8, 1, 33, 12, 5, k, None, 0) == EWORKSPACE and f(None, A + 8, 2, A, 1, 33, 16, 5, k, None, 0) == EALIGN
    for j in range(4):
        at = [0] * 4
        at[j] = 1 if j == 0 else 2
        assert step(61, *at) == EALIGN, j
        at[j] = 8
        assert step(60, *at) == EALIGN, j


@pytest.mark.gpu
@pytest.mark.parametrize("L,rows,cols", [(3, 5, 7), (5, 33, 35), (4, 101, 59), (3, 61, 130), (2, 301, 333), (2, 1, 3), (3, 33, 12), (2, 101, 300)])
def test_slices_of_batches(L, rows, cols):
    """Slices of a batch begin at any element; each is stepped as its copy at an address of its own, bit for bit."""
    say(f"case muon on slices {L} x [{rows}, {cols}]")
    g = _gen(L * rows)
    W, G, M, P = (_randn(g, L, rows, cols) * s for s in (0.02, 1e-3, 1e-2, 0.02))
    W = W.to(BF16)
    copies = [[t[l].clone() for l in range(L)] for t in (W, G, M, P)]
    assert any(t[l].data_ptr() % 16 for t in (W, G, M, P) for l in range(L))
    O = sl.sl_orthogonalize(G)
    for dtype in (F32, BF16):
        x = G.to(dtype)
        out = torch.zeros((L, rows, cols), dtype=BF16, device="cuda")
        sl.sl_orthogonalize(x[L - 1], out=out[L - 1])
        assert torch.equal(out[L - 1], sl.sl_orthogonalize(x[L - 1].clone())) and not out[:L - 1].any()
    sl.sl_muon_step(list(W.unbind(0)), list(G.unbind(0)), list(M.unbind(0)), 0.02, masters=list(P.unbind(0)), weight_decay=0.1)
    sl.sl_muon_step(*copies[:3], 0.02, masters=copies[3], weight_decay=0.1)
    for t, c in zip((W, G, M, P), copies):
        assert all(torch.equal(t[l], c[l]) for l in range(L))
    assert torch.isfinite(P).all() and O.shape == G.shape
