"""The vocabulary-parallel embedding: refusals on the CPU, lookups and gradients on the GPU against 64 bits."""
import pytest
import torch

import sharded_linear_amd as sl
from sharded_linear_amd import _lib
from tests.gpu_util import say

OK, EINVAL, EALIGN, ESHAPE, EWORKSPACE = 0, -1, -2, -3, -4
A = 1 << 20          # an aligned fake device address, never dereferenced
BF16, F32 = torch.bfloat16, torch.float32


def test_lookup_validation():
    f = _lib.lib().sl_embedding_fwd
    assert f(None, A, 4, A, A, 4, 10, 12, 0, 1.0) == ESHAPE                 # H % 8
    assert f(None, A, 4, A, A, 4, (1 << 24) + 1, 16, 0, 1.0) == ESHAPE
    assert f(None, A, 4, A, A, 1 << 31, 10, 16, 0, 1.0) == ESHAPE
    assert f(None, A, 2, A, A, 4, 10, 16, 0, 1.0) == EINVAL                 # ids of 2 bytes
    assert f(None, A, 4, A, A, -1, 10, 16, 0, 1.0) == EINVAL
    assert f(None, A, 4, A, A, 4, 10, 16, -1, 1.0) == EINVAL                # vocab_start
    assert f(None, A, 4, A, A, 4, 10, 16, 0, float("inf")) == EINVAL
    assert f(None, A, 4, A, A, 4, 10, 16, 0, float("nan")) == EINVAL
    assert f(None, None, 4, A, A, 4, 10, 16, 0, 1.0) == EINVAL
    assert f(None, A, 4, None, A, 4, 10, 16, 0, 1.0) == EINVAL
    assert f(None, A, 4, A, None, 4, 10, 16, 0, 1.0) == EINVAL
    assert f(None, A + 4, 8, A, A, 4, 10, 16, 0, 1.0) == EALIGN
    assert f(None, A, 4, A + 8, A, 4, 10, 16, 0, 1.0) == EALIGN
    assert f(None, A, 4, A, A + 2, 4, 10, 16, 0, 1.0) == EALIGN
    assert f(None, None, 4, None, None, 0, 10, 16, 0, 1.0) == OK
    assert f(None, A, 4, A, None, 4, 10, 0, 0, 1.0) == OK


def test_gradient_validation():
    L = _lib.lib()
    f, ws = L.sl_embedding_wgrad_accum, L.sl_embedding_wgrad_workspace_bytes
    need = ws(2000, 50, 64)
    assert need > 0 and ws(0, 50, 64) == 0 and ws(2000, 0, 64) == 0 and ws(2000, 50, 12) == 0 and ws(-1, 50, 64) == 0 and ws(1000, 50, 64) == 0
    ok = (2000, 50, 64, 0, 1.0)
    assert f(None, A, 4, A, A, 2000, 50, 60, 0, 1.0, A, need) == ESHAPE
    assert f(None, A, 4, A, A, (1 << 26) + 1, 50, 64, 0, 1.0, A, 1 << 60) == ESHAPE
    assert f(None, A, 4, A, A, 1 << 26, 50, 8192, 0, 1.0, A, 1 << 60) == ESHAPE     # more threads than a launch has
    assert f(None, A, 3, A, A, *ok, A, need) == EINVAL
    assert f(None, A, 4, None, A, *ok, A, need) == EINVAL
    assert f(None, A, 4, A, None, *ok, A, need) == EINVAL
    assert f(None, A + 2, 4, A, A, *ok, A, need) == EALIGN
    assert f(None, A, 4, A + 4, A, *ok, A, need) == EALIGN
    assert f(None, A, 4, A, A + 4, *ok, A, need) == EALIGN
    assert f(None, A, 4, A, A, *ok, None, 0) == EWORKSPACE
    assert f(None, A, 4, A, A, *ok, A, need - 1) == EWORKSPACE
    assert f(None, A, 4, A, A, *ok, A + 4, need) == EWORKSPACE
    assert f(None, None, 4, None, None, 0, 50, 64, 0, 1.0, None, 0) == OK
    assert f(None, A, 4, None, None, 2000, 0, 64, 0, 1.0, None, 0) == OK             # no rows in this shard


def test_binding_refusals(monkeypatch):
    from sharded_linear_amd import ops
    with pytest.raises(ValueError, match="GPU tensors"):
        sl.sl_embedding_fwd(torch.zeros(3, dtype=torch.int32), torch.zeros(4, 8, dtype=BF16))
    monkeypatch.setattr(ops, "_device", lambda t: t.device)
    ids, W = torch.zeros(3, dtype=torch.int32), torch.zeros(4, 8, dtype=BF16)
    with pytest.raises(TypeError, match="ids"):
        sl.sl_embedding_fwd(ids.float(), W)
    with pytest.raises(ValueError, match="matrix"):
        sl.sl_embedding_fwd(ids, W[0])
    with pytest.raises(TypeError, match="W"):
        sl.sl_embedding_fwd(ids, W.float())
    with pytest.raises(ValueError, match="Y"):
        sl.sl_embedding_fwd(ids, W, Y=torch.zeros(3, 9, dtype=BF16))
    with pytest.raises(ValueError, match="contiguous"):
        sl.sl_embedding_fwd(torch.zeros(6, dtype=torch.int32)[::2], W)
    with pytest.raises(ValueError, match="dY"):
        sl.sl_embedding_wgrad_accum(ids, torch.zeros(4, 8, dtype=BF16), torch.zeros(4, 8))
    with pytest.raises(TypeError, match="main_grad"):
        sl.sl_embedding_wgrad_accum(ids, torch.zeros(3, 8, dtype=BF16), W)
    with pytest.raises(ValueError, match="main_grad"):
        sl.embedding_with_grad_accumulation(ids, torch.nn.Parameter(W))


# ---- on the GPU -----------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(g, *shape):
    return torch.randn(shape, generator=g, device="cuda").to(BF16)


def _ids(g, T, lo, hi, dtype):
    return torch.randint(lo, hi, (T,), generator=g, device="cuda").to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,V,H,scale", [(1, 7, 8, 1.0), (5, 300, 64, 2.0), (33, 1000, 136, 0.3), (257, 129, 520, 45.25), (1030, 5000, 2056, 1.0)])
def test_lookup(T, V, H, scale, dtype):
    say(f"case lookup T={T} V={V} H={H} scale={scale} {dtype}")
    g = _gen(T)
    W, start = _bf16(g, V, H), 3 * V
    ids = _ids(g, T, start - V // 2, start + V + V // 2, dtype)
    ids[0] = start + V - 1
    if T > 4:
        ids[1], ids[2], ids[3], ids[4] = start, start - 1, start + V, -1
    Y = sl.sl_embedding_fwd(ids, W, vocab_start=start, scale=scale)
    at = ids.long() - start
    mine = (at >= 0) & (at < V)
    ref = torch.where(mine[:, None], W.double()[at.clamp(0, V - 1)] * scale, 0.0)
    # one fp32 rounding of the product, one to bf16 (half a step is 2^-8)
    assert ((Y.double() - ref).abs() <= ref.abs() * (2.0 ** -8 * (1 + 2.0 ** -23) + 2.0 ** -24)).all()
    if scale in (1.0, 2.0):
        assert torch.equal(Y.double(), ref)
    assert not Y[~mine].any()
    shaped = sl.sl_embedding_fwd(ids.view(1, T, 1), W, vocab_start=start, scale=scale)
    assert shaped.shape == (1, T, 1, H) and torch.equal(shaped.view(T, H), Y)


@pytest.mark.gpu
def test_lookup_keeps_infinities_and_ignores_rows_of_others():
    say("case lookup of infinities")
    W = torch.full((4, 16), float("nan"), dtype=BF16, device="cuda")
    W[2] = float("inf")
    Y = sl.sl_embedding_fwd(torch.tensor([2, 9, -2 ** 31, 2 ** 31 - 1], dtype=torch.int32, device="cuda"), W, scale=-1.0)
    assert (Y[0] == float("-inf")).all() and not Y[1:].any()
    far = torch.tensor([2 ** 62, -2 ** 63, 2 ** 63 - 1], device="cuda")
    assert not sl.sl_embedding_fwd(far, W, vocab_start=2 ** 40).any()


def _exact_case(ids, V, H, start, seed, scale=1.0):
    """Integers: every sum is exact in fp32, so main_grad has to be the right bits."""
    g = _gen(seed)
    dY = torch.randint(-8, 9, (ids.numel(), H), generator=g, device="cuda").to(BF16)
    grad = torch.randint(-8, 9, (V, H), generator=g, device="cuda").float()
    at = ids.long().view(-1)
    mine = (at >= start) & (at - max(start - 1, 0) <= V) if start else (at >= 0) & (at < V)
    at = at - start
    ref = grad.double().index_add_(0, at[mine], dY.double()[mine] * scale)
    got = sl.sl_embedding_wgrad_accum(ids, dY.view(*ids.shape, H), grad, vocab_start=start, scale=scale)
    assert got is grad
    assert torch.equal(got.double(), ref)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
@pytest.mark.parametrize("T,V,H", [(1, 1, 8), (2, 3, 8), (15, 4, 72), (16, 2, 64), (17, 1, 2048), (64, 5, 512), (100, 64128, 1032),
                                   (1013, 300, 520), (1025, 7, 2056), (4096, 100, 264), (8192, 64128, 128), (20011, 1000, 64)])
def test_gradient_of_integers(T, V, H, dtype):
    say(f"case embedding gradient T={T} V={V} H={H} {dtype}")
    _exact_case(_ids(_gen(T), T, V // 2, 2 * V + 1, dtype), V, H, V // 2 + V // 4, T, scale=0.5)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 16, 31, 32, 33, 1000, 8192, 40000])
def test_gradient_of_one_id(T):
    """All places hold one id: the longest run, across every border of chunks."""
    say(f"case embedding gradient of one id T={T}")
    _exact_case(torch.full((T,), 5, dtype=torch.int32, device="cuda"), 9, 136, 0, T)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [70000, 300000, 5000000])
def test_gradient_of_large_tables(V):
    """More ids than 256 buckets hold: buckets in the thousands; first and last rows met."""
    say(f"case embedding gradient V={V}")
    ids = _ids(_gen(3), 700, 0, V, torch.int64)
    ids[:3] = torch.tensor([0, V - 1, V - 1], device="cuda")
    _exact_case(ids, V, 8, 0, V)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [40, 3000])
def test_gradient_of_far_ids(T):
    """Ids and shards at the ends of 32 and 64 bits: differences that wrap name no row."""
    say(f"case embedding gradient of far ids T={T}")
    for dtype, start, ends in ((torch.int32, 2 ** 31 - 20, (-2 ** 31, -1, 0, 2 ** 31 - 21, 2 ** 31 - 1)),
                               (torch.int32, 2 ** 31 + 5, (-2 ** 31, 2 ** 31 - 1)), (torch.int32, 2 ** 32 + 3, (0, 3, 4)),
                               (torch.int64, 2 ** 62, (-2 ** 63, -2 ** 62, 2 ** 62 - 1, 2 ** 62 + 50, 2 ** 63 - 1)),
                               (torch.int64, 2 ** 63 - 20, (-2 ** 63, -1, 2 ** 63 - 1))):
        ids = torch.tensor([ends[k % len(ends)] for k in range(T)], dtype=dtype, device="cuda")
        _exact_case(ids, 30, 16, start, T)


@pytest.mark.gpu
def test_gradient_runs_of_all_lengths():
    """Runs of 1 .. 70 places in random order: each length begins and ends somewhere in a chunk."""
    say("case embedding gradient run lengths")
    g = _gen(11)
    ids = torch.repeat_interleave(torch.arange(70, device="cuda"), torch.arange(1, 71, device="cuda"))
    for seed in range(3):
        _exact_case(ids[torch.randperm(ids.numel(), generator=g, device="cuda")].to(torch.int32), 70, 72, 0, seed)


@pytest.mark.gpu
@pytest.mark.parametrize("T,V,H,scale", [(777, 50, 264, 22.625), (8192, 3000, 512, 0.37)])
def test_gradient_of_normal_values(T, V, H, scale):
    say(f"case embedding gradient, normal T={T} V={V} H={H}")
    g = _gen(T)
    ids, dY = _ids(g, T, 0, V, torch.int32), _bf16(g, T, H)
    grad = torch.randn((V, H), generator=g, device="cuda")
    old = grad.clone()
    ref = old.double().index_add_(0, ids.long(), dY.double() * scale)
    mass = old.double().abs().index_add_(0, ids.long(), dY.double().abs() * scale)
    count = torch.bincount(ids.long(), minlength=V).double()[:, None]
    sl.sl_embedding_wgrad_accum(ids, dY, grad, scale=scale)
    # count additions, the product with the scale and the addition to main_grad, half a step each
    assert ((grad.double() - ref).abs() <= (count + 3) * 2.0 ** -24 * mass).all()
    again = old.clone()
    sl.sl_embedding_wgrad_accum(ids, dY, again, scale=scale)
    assert torch.equal(again, grad)


@pytest.mark.gpu
def test_gradient_leaves_other_rows_alone():
    say("case embedding gradient, rows not met")
    whole = torch.full((3, 64, 16), float("nan"), device="cuda")       # the shard's rows between other data
    grad = whole[1]
    grad[::2] = 0
    dY = torch.ones((200, 16), dtype=BF16, device="cuda")
    ids = torch.arange(200, dtype=torch.int32, device="cuda") % 32 * 2
    ids[150:] = 1000
    dY[150:] = float("inf")                                            # another rank's places
    sl.sl_embedding_wgrad_accum(ids, dY, grad)
    assert torch.isfinite(grad[::2]).all() and grad[::2].sum() == 150 * 16
    assert torch.isnan(grad[1::2]).all() and torch.isnan(whole[0]).all() and torch.isnan(whole[2]).all()


@pytest.mark.gpu
def test_empty_extents():
    say("case embedding of no tokens")
    W = torch.ones((4, 8), dtype=BF16, device="cuda")
    grad = torch.ones((4, 8), device="cuda")
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    assert sl.sl_embedding_fwd(none, W).shape == (0, 8)
    sl.sl_embedding_wgrad_accum(none, W[:0], grad)
    assert (grad == 1).all()
    ids = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert not sl.sl_embedding_fwd(ids, W[:0]).any()                   # a shard without rows


@pytest.mark.gpu
def test_autograd_against_formula_and_differences():
    say("case embedding autograd")
    g = _gen(1)
    V, H, start, scale = 37, 24, 100, 2.0
    buf = sl.ParamAndGradBuffer({"table": (V, H)}, "cuda", bucket_size=None)
    w = buf.attach("table", torch.nn.Parameter(_bf16(g, V, H)))
    ids = _ids(g, 90, 90, 150, torch.int64).view(2, 45)
    c = _bf16(g, 2, 45, H)
    for k in range(2):                                                  # two micro-batches add up
        y = sl.embedding_with_grad_accumulation(ids, w, start, scale)
        assert y.shape == (2, 45, H)
        y.backward(c)
        assert w.grad is None and w.grad_added_to_main_grad
    loss = lambda t: (torch.nn.functional.embedding((ids - start).clamp(0, V - 1), t) * scale * c.double()  # noqa: E731
                      * ((ids >= start) & (ids < start + V))[..., None]).sum()
    t = w.detach().double()
    for v, h in ((0, 0), (V - 1, H - 1), (5, 7)):
        step = torch.zeros_like(t)
        step[v, h] = 1
        slope = (loss(t + step) - loss(t - step)) / 2                   # the loss is linear
        assert abs(w.main_grad[v, h].item() - 2 * slope.item()) <= 1e-5 * (1 + abs(slope.item()))
    with torch.no_grad():
        assert not sl.embedding_with_grad_accumulation(ids, w, start, scale).requires_grad
    assert torch.equal(sl.embedding_with_grad_accumulation(ids, w.detach(), start, scale), y)


@pytest.mark.gpu
def test_captured_and_replayed():
    """Two graphs over the same arrays, replayed in turn with other ids each time and eager work between."""
    say("case embedding graphs")
    g = _gen(8)
    V, H, T = 500, 256, 3000
    W, dY, ids = _bf16(g, V, H), _bf16(g, T, H), torch.zeros(T, dtype=torch.int32, device="cuda")
    grads = [torch.zeros((V, H), device="cuda") for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        sl.sl_embedding_wgrad_accum(ids, dY, torch.zeros((V, H), device="cuda"))
        sl.sl_embedding_fwd(ids, W)
    torch.cuda.current_stream().wait_stream(s)
    graphs, outs = [], []
    for k in range(2):
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs.append(sl.sl_embedding_fwd(ids, W, scale=1.0 + k))
            sl.sl_embedding_wgrad_accum(ids, dY, grads[k], scale=1.0 + k)
        graphs.append(graph)
    for r in range(4):
        ids.copy_(_ids(g, T, -5, V + 5 + 300 * r, torch.int32))
        k = r % 2
        before = grads[k].clone()
        graphs[k].replay()
        sl.sl_embedding_wgrad_accum(ids, dY, before, scale=1.0 + k)
        torch.cuda.synchronize()
        assert torch.equal(outs[k], sl.sl_embedding_fwd(ids, W, scale=1.0 + k))
        assert torch.equal(grads[k], before)


@pytest.mark.gpu
def test_on_a_side_stream():
    say("case embedding on a side stream")
    g = _gen(9)
    s = torch.cuda.Stream()
    V, H, T = 800, 512, 5000
    W, dY = _bf16(g, V, H), _bf16(g, T, H)
    ids = _ids(g, T, 0, V, torch.int32)
    want, grad = sl.sl_embedding_fwd(ids, W), sl.sl_embedding_wgrad_accum(ids, dY, torch.zeros((V, H), device="cuda"))
    torch.cuda.synchronize()
    with torch.cuda.stream(s):
        late = torch.zeros_like(ids)
        for _ in range(20):
            late.copy_(ids)                                             # work that the calls have to wait for
        y, got = sl.sl_embedding_fwd(late, W), sl.sl_embedding_wgrad_accum(late, dY, torch.zeros((V, H), device="cuda"))
    s.synchronize()
    assert torch.equal(y, want) and torch.equal(got, grad)


@pytest.mark.gpu
@pytest.mark.parametrize("V", [255000, 256001, 513000, 1100000, 2500000, 5000000, 9000000, 1 << 24])
def test_sorted_gradient_of_large_tables(V):
    """Tokens enough for the sort, and more ids than 256 buckets hold: 2^8 to 2^15 buckets; first and last rows met, repeated ids, and ids
    of one bucket (equal low bits)."""
    say(f"case embedding gradient, sorted, V={V}")
    g = _gen(V % 1000)
    ids = _ids(g, 1500, 0, V, torch.int64)
    ids[:4] = torch.tensor([0, V - 1, V - 1, 0], device="cuda")
    ids[100:400] = torch.arange(300, device="cuda") % 60 * 32768 % V
    ids[1000:1300] = ids[400:700]
    for dtype in (torch.int32, torch.int64):
        _exact_case(ids.to(dtype), V, 8, 0, V)
    _exact_case(ids + 12345, V, 8, 12345 + V // 3, V)
