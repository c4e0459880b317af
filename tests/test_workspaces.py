"""Workspaces that the binding takes by itself: each call's own.

A call with a workspace is two launches (partial sums and their join, or a weight's bf16 copy and the
product), and the interpreter runs other threads during a call into the library: a buffer shared by two
callers on one stream would be filled by the second between the first one's launches.
"""
import contextlib
import threading
import types

import numpy as np
import pytest
import torch

import sharded_linear_amd as sl
from oracle import mxfp4
from sharded_linear_amd import ops
from tests.gpu_util import dev_u8, say

U8, BF16 = torch.uint8, torch.bfloat16


class _MeetingLibrary:
    """Stands for the C library: every call waits inside for the other thread's, and notes its workspace."""

    def __init__(self):
        self.inside, self.seen = threading.Barrier(2, timeout=30), []

    def __getattr__(self, name):
        if name.endswith("_workspace_bytes"):
            return lambda *a: 256

        def call(*a):
            ws = a[-2]
            self.seen.append((getattr(ws, "value", ws), int(a[-1])))
            self.inside.wait()
            return 0
        return call


def _zeros(dtype, *shape):
    return torch.zeros(shape, dtype=dtype)


# 1024 tokens, 64 inputs, 64 outputs
CALLS = {
    "wgrad": lambda: sl.sl_linear_wgrad_accum(_zeros(BF16, 1024, 64), _zeros(BF16, 1024, 64), _zeros(torch.float32, 64, 64)),
    "dgrad_mxfp8w": lambda: sl.sl_linear_dgrad_mxfp8w(_zeros(BF16, 1024, 64), _zeros(U8, 64, 64), _zeros(U8, 64, 2)),
    "wgrad_mxfp8x": lambda: sl.sl_linear_wgrad_accum_mxfp8x(_zeros(U8, 1024, 64), _zeros(U8, 1024, 2), _zeros(BF16, 1024, 64),
                                                            _zeros(torch.float32, 64, 64)),
    "wgrad_mxfp8": lambda: sl.sl_linear_wgrad_accum_mxfp8(_zeros(U8, 64, 1024), _zeros(U8, 64, 32), _zeros(U8, 64, 1024),
                                                          _zeros(U8, 64, 32), _zeros(torch.float32, 64, 64)),
    "fwd_mxfp4": lambda: sl.sl_linear_fwd_mxfp4(_zeros(U8, 1024, 32), _zeros(U8, 1024, 2), _zeros(U8, 64, 32), _zeros(U8, 64, 2)),
    "dgrad_mxfp4": lambda: sl.sl_linear_dgrad_mxfp4(_zeros(U8, 1024, 32), _zeros(U8, 1024, 2), _zeros(U8, 64, 32), _zeros(U8, 64, 2)),
    "wgrad_mxfp4": lambda: sl.sl_linear_wgrad_accum_mxfp4(_zeros(U8, 64, 512), _zeros(U8, 64, 32), _zeros(U8, 64, 512),
                                                          _zeros(U8, 64, 32), _zeros(torch.float32, 64, 64)),
    "fwd_mxfp4w": lambda: sl.sl_linear_fwd_mxfp4w(_zeros(BF16, 1024, 64), _zeros(U8, 64, 32), _zeros(U8, 64, 2)),
    "dgrad_mxfp4w": lambda: sl.sl_linear_dgrad_mxfp4w(_zeros(BF16, 1024, 64), _zeros(U8, 64, 32), _zeros(U8, 64, 2)),
}


@pytest.mark.parametrize("name", CALLS)
def test_calls_of_two_threads_on_one_stream_have_workspaces_of_their_own(name, monkeypatch):
    fake = _MeetingLibrary()
    monkeypatch.setattr(ops, "lib", lambda: fake)
    monkeypatch.setattr(ops, "_device", lambda t: t.device)
    monkeypatch.setattr(ops, "_stream", lambda dev: None)
    monkeypatch.setattr(ops, "_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: None)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: types.SimpleNamespace(cuda_stream=0))
    monkeypatch.setattr(torch.cuda, "device", lambda dev: contextlib.nullcontext())
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
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

def _operand(rows, k, seed):
    g = np.random.default_rng(seed)
    return tuple(dev_u8(t) for t in mxfp4.quantize(g.standard_normal((rows, k))))


@pytest.mark.gpu
def test_two_threads_on_one_stream():
    """Two host threads on the default stream, each with operands of its own: split sums, a bf16 copy of the weight, and a
    split weight gradient give every thread the bits that it gets alone."""
    say("case two threads on one stream")

    def make(k):
        a, b, w = _operand(200, 8192, 10 + k), _operand(64, 8192, 20 + k), _operand(520, 512, 30 + k)
        x, many = torch.randn((100, 8192), device="cuda").bfloat16(), torch.randn((1100, 512), device="cuda").bfloat16()
        ta, tb = _operand(136, 8192, 40 + k), _operand(72, 8192, 50 + k)

        def run():
            g = torch.zeros((136, 72), device="cuda")
            sl.sl_linear_wgrad_accum_mxfp4(*ta, *tb, g)
            return sl.sl_linear_fwd_mxfp4(*a, *b), sl.sl_linear_fwd_mxfp4w(x, *b), sl.sl_linear_fwd_mxfp4w(many, *w), g
        return run

    assert sl.sl_mxfp4_fwd_workspace_bytes(200, 8192, 64) and sl.sl_mxfp4w_fwd_workspace_bytes(100, 8192, 64)
    assert sl.sl_mxfp4w_fwd_workspace_bytes(1100, 512, 520) == 512 * 520 * 2 and sl.sl_mxfp4_wgrad_workspace_bytes(8192, 72, 136)
    runs = [make(k) for k in range(2)]
    want = [run() for run in runs]
    torch.cuda.synchronize()
    got, start = [[], []], threading.Barrier(2, timeout=60)

    def work(k):
        start.wait()
        for _ in range(25):
            got[k].append(runs[k]())

    threads = [threading.Thread(target=work, args=(k,)) for k in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for k in range(2):
        assert len(got[k]) == 25
        for outs in got[k]:
            for o, w in zip(outs, want[k]):
                assert torch.equal(o, w), k


@pytest.mark.gpu
def test_a_call_keeps_no_memory():
    """The bf16 copy of a 4-bit weight that a product of many tokens takes goes back to the allocator with the call."""
    say("case workspace given back")
    w, X = _operand(4096, 1024, 1), torch.ones((1024, 1024), dtype=BF16, device="cuda")
    Y = torch.empty((1024, 4096), dtype=BF16, device="cuda")
    assert sl.sl_mxfp4w_fwd_workspace_bytes(1024, 1024, 4096) == 4096 * 1024 * 2
    torch.cuda.synchronize()
    with torch.cuda.stream(torch.cuda.Stream()):
        before = torch.cuda.memory_allocated()
        sl.sl_linear_fwd_mxfp4w(X, *w, Y)
        assert torch.cuda.memory_allocated() == before
    torch.cuda.synchronize()


@pytest.mark.gpu
def test_two_graphs_of_split_bf16_weight_gradients():
    """Two captured graphs, replayed side by side on two streams: neither uses the other's planes, nor an eager call's."""
    say("case two graphs of bf16 weight gradients")
    T, n_in, n_out = 4096, 264, 520
    assert sl.sl_wgrad_workspace_bytes(T, n_in, n_out)
    cases = []
    for k in range(2):
        g = torch.Generator(device="cuda")
        g.manual_seed(k)
        X, dY = (torch.randn((T, n), device="cuda", generator=g).bfloat16() for n in (n_in, n_out))
        grad = torch.zeros((n_out, n_in), device="cuda")
        want = sl.sl_linear_wgrad_accum(X, dY, torch.zeros_like(grad))
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            grad.zero_()
            sl.sl_linear_wgrad_accum(X, dY, grad)
        cases.append((graph, X, dY, grad, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        torch.cuda.synchronize()
        for (graph, *_rest), s in zip(cases, streams):
            with torch.cuda.stream(s):
                graph.replay()
        eager = sl.sl_linear_wgrad_accum(*cases[0][1:3], torch.zeros((n_out, n_in), device="cuda"))
        torch.cuda.synchronize()
        assert torch.equal(eager, cases[0][4])
        for _graph, _x, _dy, grad, want in cases:
            assert torch.equal(grad, want)
