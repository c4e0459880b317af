"""The embedding, the norm and the orthogonalised update where they meet: workspaces of their own for every call, offsets past 32
bits, captured gradients, and a training step of all of them on one buffer."""
import contextlib
import threading
import types

import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import sharded_linear_amd as sl
from sharded_linear_amd import ops
from tests.gpu_util import say

BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
HALF = 2.0 ** -8     # half a step of bf16


class _MeetingLibrary:
    """Stands for the C library: every call waits inside for the other thread's, and notes its workspace."""

    def __init__(self):
        self.inside, self.seen = threading.Barrier(2, timeout=30), []

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return lambda *a: 256

        def call(*a):
            self.seen.append((a[-2], int(a[-1])))
            self.inside.wait()
            return 0
        return call


def _z(dtype, *shape):
    return torch.zeros(shape, dtype=dtype)


CALLS = {
    "embedding": lambda: sl.sl_embedding_wgrad_accum(_z(I32, 2000), _z(BF16, 2000, 64), _z(F32, 10, 64)),
    "norm": lambda: sl.sl_rmsnorm_bwd(_z(BF16, 8, 64), _z(BF16, 8, 64), _z(BF16, 64), _z(F32, 8), _z(F32, 64)),
    "orthogonalize": lambda: sl.sl_orthogonalize(_z(F32, 8, 16)),
    "muon": lambda: sl.sl_muon_step(_z(BF16, 8, 16), _z(F32, 8, 16), _z(F32, 8, 16), 0.1),
}


@pytest.mark.parametrize("name", CALLS)
def test_calls_of_two_threads_on_one_stream_have_workspaces_of_their_own(name, monkeypatch):
    fake = _MeetingLibrary()
    monkeypatch.setattr(ops, "lib", lambda: fake)
    monkeypatch.setattr(ops, "_device", lambda t: t.device)
    monkeypatch.setattr(ops, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: types.SimpleNamespace(cuda_stream=0))
    errors = []

    def run():
        try:
            CALLS[name]()
        except BaseException as e:  # noqa: BLE001
            errors.append(e)

    threads = [threading.Thread(target=run) for _ in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not errors
    (a, n), (b, m) = fake.seen
    assert a and b and n >= 256 and m >= 256
    assert a + n <= b or b + m <= a, "two calls under way share a workspace"


# ---- on the GPU -----------------------------------------------------------------------------------

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _bf16(g, *shape, std=1.0):
    return (torch.randn(shape, generator=g, device="cuda") * std).to(BF16)


def _work(seed):
    """A closure that runs the four calls with a workspace, on operands of its own."""
    g = _gen(seed)
    ids = torch.randint(0, 500, (3000,), generator=g, device="cuda").to(I32)
    dY, W = _bf16(g, 3000, 256), (1 + 0.1 * torch.randn(256, generator=g, device="cuda")).to(BF16)
    h, G, wide = _bf16(g, 3000, 256), torch.randn((400, 700), generator=g, device="cuda"), torch.randn((3, 60, 200), generator=g, device="cuda")
    start = _bf16(g, 400, 700, std=0.02)

    def run():
        table, grad = torch.zeros((500, 256), device="cuda"), torch.zeros(256, device="cuda")
        sl.sl_embedding_wgrad_accum(ids, dY, table)
        rstd = sl.sl_rmsnorm_fwd(h, W, 1e-5)[2]
        dx = sl.sl_rmsnorm_bwd(dY, h, W, rstd, grad)
        w, m = start.clone(), torch.zeros((400, 700), device="cuda")
        sl.sl_muon_step(w, G, m, 0.1)
        return table, grad, dx, w, m, sl.sl_orthogonalize(G), sl.sl_orthogonalize(wide)
    return run


@pytest.mark.gpu
def test_two_threads_on_one_stream():
    say("case step operators, two threads on one stream")
    runs = [_work(k) for k in range(2)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    got, start = [[], []], threading.Barrier(2, timeout=60)

    def work(k):
        start.wait()
        for _ in range(15):
            got[k].append(runs[k]())

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for k in range(2):
        assert len(got[k]) == 15
        for outs in got[k]:
            assert all(torch.equal(o, w) for o, w in zip(outs, want[k]))


@pytest.mark.gpu
def test_two_graphs_side_by_side():
    say("case step operators, two graphs side by side")
    runs = [_work(k) for k in range(2)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    cases = []
    for run in runs:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = run()
        cases.append((graph, outs))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        torch.cuda.synchronize()
        for (graph, _outs), s in zip(cases, streams):
            with torch.cuda.stream(s):
                graph.replay()
        eager = runs[0]()
        torch.cuda.synchronize()
        assert all(torch.equal(e, w) for e, w in zip(eager, want[0]))
        for (_graph, outs), w in zip(cases, want):
            assert all(torch.equal(o, x) for o, x in zip(outs, w))


@pytest.mark.gpu
def test_embedding_past_32_bits():
    """A table and a gradient of more than 2^31 elements, and more than 2^31 elements of results."""
    say("case embedding past 32 bits")
    V, H = (1 << 19) + 100, 4096 + 8
    assert V * H > 1 << 31
    W = torch.zeros((V, H), dtype=BF16, device="cuda")
    W[-3:] = torch.arange(1, 4, device="cuda")[:, None].to(BF16)
    T = (1 << 19) + 50
    ids = torch.full((T,), V - 2, dtype=I32, device="cuda")
    ids[-1] = V - 1
    Y = sl.sl_embedding_fwd(ids, W)
    assert (Y[T - 2] == 2).all() and (Y[T - 1] == 3).all() and (Y[0] == 2).all()
    del W
    grad = torch.zeros((V, H), device="cuda")
    few = ids[-2000:].contiguous()
    sl.sl_embedding_wgrad_accum(few, Y[-2000:].contiguous(), grad)
    assert (grad[V - 2] == 2 * 1999).all() and (grad[V - 1] == 3).all() and not grad[:V - 2].any()
    Y.fill_(1)
    grad[-2:] = 0
    sl.sl_embedding_wgrad_accum(ids, Y, grad)                       # the longest run, and offsets of dY past 2^31
    assert (grad[V - 2] == T - 1).all() and (grad[V - 1] == 1).all() and not grad[:V - 2].any()


@pytest.mark.gpu
def test_norm_past_32_bits():
    say("case norm past 32 bits")
    T, H = (1 << 19) + 32, 4096 + 32
    assert T * H > 1 << 31
    g = _gen(1)
    tail = _bf16(g, 64, H)
    x = torch.ones((T, H), dtype=BF16, device="cuda")
    x[-64:] = tail
    w = (1 + 0.1 * torch.randn(H, generator=g, device="cuda")).to(BF16)
    qr, sr, qc, sc, h, rstd = sl.sl_rmsnorm_fwd_mxfp8(x, w, 1e-5, residual=x)
    want = sl.sl_rmsnorm_fwd_mxfp8(tail, w, 1e-5, residual=tail)
    assert torch.equal(qr[-64:], want[0]) and torch.equal(sr[-64:], want[1]) and torch.equal(h[-64:], want[4])
    assert torch.equal(qc[:, -64:], want[2]) and torch.equal(sc[:, -2:], want[3])
    del qr, sr, qc, sc
    grad = torch.zeros(H, device="cuda")
    dX = sl.sl_rmsnorm_bwd(x, h, w, rstd, grad, dresidual=x)
    alone = sl.sl_rmsnorm_bwd(tail, want[4], w, want[5], None, dresidual=tail)
    # a row's threads and so its sums' order depend on the number of rows: the same values up to a step of bf16
    assert ((dX[-64:].float() - alone.float()).abs() <= 2 * HALF * alone.float().abs() + 1e-4).all()


@pytest.mark.gpu
@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
def test_captured_gradients():
    """Forward and gradients of all three autograd functions in a captured graph.  While an eager graph of the same leaves
    lives, whose accumulators belong to its stream, the capture is refused."""
    say("case step operators, captured gradients")
    g = _gen(3)
    T, H, O, V = 128, 256, 384, 300
    buf = sl.ParamAndGradBuffer({"table": (V, H), "norm0": (H,), "norm": (H,), "fc": (O, H)}, "cuda", bucket_size=None)
    p = {n: buf.attach(n, torch.nn.Parameter(_bf16(g, *s, std=0.1))) for n, s in buf.shapes.items()}
    r = _bf16(g, T, H).requires_grad_()
    ids = torch.randint(0, V, (T,), generator=g, device="cuda")
    cy, ch = _bf16(g, T, O), _bf16(g, T, H)
    calls = {
        "embedding": lambda: sl.embedding_with_grad_accumulation(ids, p["table"], scale=4.0),
        "norm": lambda: sl.rmsnorm_with_grad_accumulation(r, p["norm0"]),
        "residual": lambda: sl.rmsnorm_with_grad_accumulation(cy[:, :H], p["norm0"], r)[0],
        "norm linear": lambda: sl.norm_linear_mxfp8_with_grad_accumulation(r, p["norm"], p["fc"]),
    }

    def both():
        x = sl.rmsnorm_with_grad_accumulation(calls["embedding"](), p["norm0"])
        y, h = sl.norm_linear_mxfp8_with_grad_accumulation(x, p["norm"], p["fc"], r)
        dr, _ = torch.autograd.grad((y, h), (r, p["table"]), (cy, ch), allow_unused=True)
        return y.detach(), h.detach(), dr

    for call in calls.values():
        eager = call()
        with pytest.raises(RuntimeError, match="drop its results"):
            with torch.cuda.graph(torch.cuda.CUDAGraph()):
                call()
        torch.autograd.grad(eager.sum(), [q for q in (r, *p.values())], allow_unused=True)
        del eager
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = both()
    for k in range(3):
        ids.copy_(torch.randint(0, V, (T,), generator=g, device="cuda"))
        buf.zero_grad_buffer()
        graph.replay()
        got = buf.grad_data.clone()
        buf.zero_grad_buffer()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want)) and torch.equal(got, buf.grad_data)


@pytest.mark.gpu
def test_a_training_step_of_one_rank():
    """Two vocabulary shards, a block of norm and linear layers with its residual stream, gradients of two micro-batches in one
    buffer, and the optimiser's step on it, against the same step in 64 bits."""
    say("case training step of one rank")
    g = _gen(5)
    V, H, F, T = 200, 128, 256, 192
    shapes = {"table0": (V // 2, H), "table1": (V // 2, H), "norm1": (H,), "fc1": (F, H), "fc2": (H, F), "norm2": (H,)}
    buf = sl.ParamAndGradBuffer(shapes, "cuda", bucket_size=None)
    std = {"table0": 1.0, "table1": 1.0, "fc1": 0.1, "fc2": 0.1}
    p = {n: buf.attach(n, torch.nn.Parameter(_bf16(g, *s, std=std[n]) if n in std else (1 + _bf16(g, *s, std=0.1).float()).to(BF16)))
         for n, s in shapes.items()}
    batches = [(torch.randint(0, V, (2, T // 2), generator=g, device="cuda"), _bf16(g, 2, T // 2, H, std=0.1)) for _ in range(2)]

    def model(ids):
        x = sum(sl.embedding_with_grad_accumulation(ids, p[f"table{k}"], vocab_start=k * V // 2) for k in range(2))
        n = sl.rmsnorm_with_grad_accumulation(x, p["norm1"])
        a = sl.linear_with_grad_accumulation(torch.tanh(sl.linear_with_grad_accumulation(n, p["fc1"])), p["fc2"])
        return sl.rmsnorm_with_grad_accumulation(a, p["norm2"], x)

    def exact(ids, q):
        x = torch.cat([q["table0"], q["table1"]])[ids]
        norm = lambda v, w: v / torch.sqrt(v.square().mean(-1, keepdim=True) + 1e-5) * w  # noqa: E731
        h = x + torch.tanh(norm(x, q["norm1"]) @ q["fc1"].t()) @ q["fc2"].t()
        return norm(h, q["norm2"]), h

    q = {n: w.detach().double().requires_grad_() for n, w in p.items()}
    buf.zero_grad_buffer()
    for ids, c in batches:
        y, h = model(ids)
        ((y + h) * c).sum().backward()
        ye, he = exact(ids, q)
        # ten roundings to bf16 on the way, of a step's half each, in values that add up: 10 half steps of the largest
        assert (y.double() - ye).abs().max() <= 10 * HALF * ye.abs().max()
        ((ye + he) * c.double()).sum().backward()
    for n in shapes:
        # as many roundings again in the gradient, each seen through both layers: 20 half steps of the gradient's norm
        off = (buf.main_grad(n).double() - q[n].grad).norm()
        assert off <= 20 * HALF * q[n].grad.norm(), n
    momentum, old = torch.zeros_like(buf.grad_data), buf.param_data.clone()
    buf.muon_step(["fc1", "fc2"], momentum, 0.02)
    for n in ("fc1", "fc2"):
        s, e, _ = buf.index[n]
        assert torch.equal(momentum[s:e], buf.grad_data[s:e]) and not torch.equal(buf.param_data[s:e], old[s:e])
        step = (old[s:e].double() - buf.param_data[s:e].double()).view(shapes[n]) / (0.02 * max(1.0, shapes[n][0] / shapes[n][1]) ** 0.5)
        sv = torch.linalg.svdvals(step)
        assert sv.max() <= 1.3 and sv[: len(sv) // 2].min() >= 0.5         # orthogonalised: singular values near 1


def _linear_calls(g):
    """Both linear functions with one weight and its gradient buffer, an input that is no leaf, and a gradient of the results."""
    T, H, O = 128, 256, 384
    buf = sl.ParamAndGradBuffer({"fc": (O, H)}, "cuda", bucket_size=None)
    w = buf.attach("fc", torch.nn.Parameter(_bf16(g, O, H, std=0.1)))
    x = _bf16(g, T, H)
    return buf, w, x, _bf16(g, T, O), {"linear": lambda: sl.linear_with_grad_accumulation(x, w),
                                       "mxfp4": lambda: sl.linear_mxfp4_with_grad_accumulation(x, w)}


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["linear", "mxfp4"])
def test_captured_linear_gradients(name):
    """The linear functions leave a weight's gradient in main_grad as the others do: a captured backward pass that comes to the weight's
    accumulator, beside a living eager graph, is refused.  A captured forward pass is not, and without such a graph the captured
    gradients are the eager ones."""
    say(f"case captured gradients of {name}")
    buf, w, x, c, calls = _linear_calls(_gen(4))
    call = calls[name]

    def both():
        y = call()
        y.backward(c)
        return y.detach()

    eager, graph = call(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = call()
        with pytest.raises(RuntimeError, match="drop its results"):
            y.backward(c)
    y = y.detach()
    for k in range(2):
        x.copy_(_bf16(_gen(20 + k), *x.shape))
        graph.replay()
        want = call()
        torch.cuda.synchronize()
        assert torch.equal(y, want.detach()) and not buf.grad_data.any()
    del eager, want
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        both()
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for k in range(3):
        x.copy_(_bf16(_gen(10 + k), *x.shape))
        buf.zero_grad_buffer()
        graph.replay()
        got = buf.grad_data.clone()
        buf.zero_grad_buffer()
        want = both()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(got, buf.grad_data) and got.any()


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["linear", "mxfp4"])
def test_captured_linear_gradients_of_the_input_alone(name):
    """torch.autograd.grad for the input comes to no accumulator of the weight: it is captured beside a living eager graph of the weight."""
    say(f"case captured input gradients of {name}")
    buf, w, x, c, _ = _linear_calls(_gen(5))
    call = {"linear": sl.linear_with_grad_accumulation, "mxfp4": sl.linear_mxfp4_with_grad_accumulation}[name]

    def both():
        leaf = x.detach().requires_grad_()
        y = call(leaf, w)
        return y.detach(), torch.autograd.grad(y, leaf, c)[0]

    eager, graph = call(x, w), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = both()
    for k in range(3):
        x.copy_(_bf16(_gen(30 + k), *x.shape))
        buf.zero_grad_buffer()
        graph.replay()
        got = buf.grad_data.clone()
        buf.zero_grad_buffer()
        want = both()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want)) and torch.equal(got, buf.grad_data) and got.any()
    assert eager.requires_grad


@pytest.mark.gpu
@pytest.mark.filterwarnings("ignore:The CUDA Graph is empty")
def test_capture_beside_a_graph_of_another_function():
    """The accumulator is the leaf's, whichever function met it first; one that a hook's owner holds is refused by a message that names it."""
    say("case captures beside graphs of other functions")
    g = _gen(6)
    buf = sl.ParamAndGradBuffer({"table": (304, 256)}, "cuda", bucket_size=None)
    w = buf.attach("table", torch.nn.Parameter(_bf16(g, 304, 256)))
    ids, x, c = torch.randint(0, 304, (64,), generator=g, device="cuda"), _bf16(g, 32, 256), _bf16(g, 32, 304)
    lookup = lambda: sl.embedding_with_grad_accumulation(ids, w)  # noqa: E731
    product = lambda: sl.linear_with_grad_accumulation(x, w).backward(c)  # noqa: E731
    for first, second in ((lookup, product), (lambda: sl.linear_with_grad_accumulation(x, w), lookup)):          # a tied table
        eager = first()
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            with pytest.raises(RuntimeError, match="drop its results"):
                second()
        del eager
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            second()
    node = torch.autograd.graph.get_gradient_edge(w).node
    lookup()
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        with pytest.raises(RuntimeError, match="hook"):
            lookup()
    del node
    with torch.cuda.graph(torch.cuda.CUDAGraph()):
        lookup()
    # results made on the capture's own stream may live
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        eager = lookup()
        s.synchronize()
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
            lookup()
            product()
    assert eager.requires_grad


class _Made(TorchDispatchMode):
    """Notes the storages of what the dispatcher's operations return."""

    def __init__(self):
        super().__init__()
        self.storages = set()

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if isinstance(out, torch.Tensor):
            self.storages.add(out.untyped_storage().data_ptr())
        return out


@pytest.mark.gpu
def test_results_are_seen_by_the_dispatcher():
    """Modes that follow or fill new tensors see every result."""
    say("case step operators under a dispatch mode")
    g = _gen(7)
    x, w, ids = _bf16(g, 64, 64), _bf16(g, 64), torch.zeros(64, dtype=I32, device="cuda")
    rstd = sl.sl_rmsnorm_fwd(x, w, 1e-5)[2]
    q, s, _, _ = sl.sl_mxfp8_quantize(x)
    calls = {
        "embedding": lambda: (sl.sl_embedding_fwd(ids, x),),
        "norm": lambda: sl.sl_rmsnorm_fwd(x, w, 1e-5, residual=x),
        "norm mxfp8": lambda: sl.sl_rmsnorm_fwd_mxfp8(x, w, 1e-5, residual=x),
        "norm gradient": lambda: (sl.sl_rmsnorm_bwd(x, x, w, rstd, None),),
        "orthogonalize": lambda: (sl.sl_orthogonalize(x),),
        "dequantize": lambda: (sl.sl_mxfp8_dequantize(q, s),),
    }
    for name, call in calls.items():
        with _Made() as made:
            outs = call()
        for out in outs:
            assert out.untyped_storage().data_ptr() in made.storages, name


@pytest.mark.gpu
def test_results_are_modified_in_place():
    """No result of the embedding and the norms is a view made inside the function.  The residual stream h is read again by backward, which refuses a modified one; the
    other results are not."""
    say("case results modified in place")
    g = _gen(8)
    shapes = {"table": (64, 256), "norm": (256,), "fc": (128, 256)}
    buf = sl.ParamAndGradBuffer(shapes, "cuda", bucket_size=None)
    p = {n: buf.attach(n, torch.nn.Parameter(_bf16(g, *s, std=0.1))) for n, s in shapes.items()}
    x, r = _bf16(g, 2, 64, 256).requires_grad_(), _bf16(g, 2, 64, 256).requires_grad_()
    ids = torch.randint(0, 64, (2, 64), generator=g, device="cuda")
    calls = {
        "embedding": lambda: sl.embedding_with_grad_accumulation(ids, p["table"]),
        "norm": lambda: sl.rmsnorm_with_grad_accumulation(x, p["norm"]),
        "norm residual": lambda: sl.rmsnorm_with_grad_accumulation(x, p["norm"], r),
        "norm linear": lambda: sl.norm_linear_mxfp8_with_grad_accumulation(x, p["norm"], p["fc"]),
        "norm linear residual": lambda: sl.norm_linear_mxfp8_with_grad_accumulation(x, p["norm"], p["fc"], r),
    }
    for name, call in calls.items():
        say(f"case {name}")
        grads = []
        for inplace in (True, False):
            buf.zero_grad_buffer()
            out = call()
            y = out[0] if isinstance(out, tuple) else out
            assert y.shape[:2] == (2, 64) and not y._is_view()
            y = y.mul_(2.0) if inplace else y * 2.0
            dx = torch.autograd.grad(y, [x, p["table"]], torch.ones_like(y), allow_unused=True)[0]
            grads.append((dx, buf.grad_data.clone()))
        assert torch.equal(grads[0][1], grads[1][1]) and grads[0][1].any(), name
        assert (grads[0][0] is None) == (name == "embedding") and (grads[0][0] is None or torch.equal(grads[0][0], grads[1][0])), name
        if isinstance(out, tuple):
            y, h = call()
            assert h.shape == x.shape and not h._is_view()
            kept = h.detach().clone()
            h += y.detach()[..., :1]
            assert torch.equal(h.detach(), kept + y.detach()[..., :1])
            with pytest.raises(RuntimeError, match="inplace"):
                torch.autograd.grad(y, x, torch.ones_like(y))
            with torch.no_grad():
                y, h = call()
                h += 1
