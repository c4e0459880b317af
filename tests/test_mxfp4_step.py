"""The MXFP4 step's calls that compute no gradient, and its refusals."""
import pytest
import torch

import sharded_linear_amd as sl
from sharded_linear_amd import autograd
from tests.gpu_util import say

BF16 = torch.bfloat16


@pytest.fixture
def casts(monkeypatch):
    """The step without a GPU: its casts and its forward product are noted, not computed."""
    asked = []

    def quantize(x, rows=True, cols=True, seed=None):
        asked.append((tuple(x.shape), rows, cols))
        r, c = x.shape
        new = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
        up = lambda n: (n + 31) // 32 * 32  # noqa: E731
        return ((new(r, up(c) // 2), new(r, up(c) // 32)) if rows else (None, None)) + \
               ((new(c, up(r) // 2), new(c, up(r) // 32)) if cols else (None, None))

    monkeypatch.setattr(autograd, "sl_mxfp4_quantize", quantize)
    monkeypatch.setattr(autograd, "sl_linear_fwd_mxfp4", lambda xq, xs, wq, ws: torch.zeros((xq.shape[0], wq.shape[0]), dtype=BF16))
    return asked


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_evaluation_needs_no_main_grad_and_casts_rows_only(casts, mode):
    w = torch.nn.Parameter(torch.zeros(16, 64, dtype=BF16))               # no main_grad
    x = torch.zeros(4, 64, dtype=BF16, requires_grad=True)
    with mode():
        for call in (sl.linear_mxfp4_with_grad_accumulation, sl.LinearMXFP4WithGradAccumulation.apply):
            y = call(x, w, None, None)
            assert y.shape == (4, 16) and not y.requires_grad
    assert casts == [((4, 64), True, False), ((16, 64), True, False)] * 2
    w.main_grad = torch.zeros(16, 64)
    del casts[:]
    y = sl.linear_mxfp4_with_grad_accumulation(x, w)                       # with gradients both copies are taken
    assert y.requires_grad and casts == [((4, 64), True, True), ((16, 64), True, True)]


@pytest.mark.gpu
def test_evaluation_gives_the_forward_of_training():
    say("case mxfp4 step without gradients")
    g = torch.Generator(device="cuda")
    g.manual_seed(3)
    x = torch.randn((37, 72), device="cuda", generator=g).to(BF16).requires_grad_()
    w = torch.nn.Parameter(torch.randn((40, 72), device="cuda", generator=g).to(BF16))
    with torch.no_grad():
        bare = sl.linear_mxfp4_with_grad_accumulation(x, w)
        kept = sl.linear_mxfp4_with_grad_accumulation(x, w, weight_mxfp4=sl.sl_mxfp4_quantize(w, cols=False))
    w.main_grad = torch.zeros((40, 72), device="cuda")
    y = sl.linear_mxfp4_with_grad_accumulation(x, w)
    assert y.requires_grad and not bare.requires_grad
    assert torch.equal(bare, y) and torch.equal(kept, y)


@pytest.mark.parametrize("features", [40, 72])
def test_an_input_of_other_features_than_the_weight_is_refused(casts, features):
    """Both pad to the same whole blocks of 32, so the products alone would not tell 40 from 64 or 72 from 96."""
    w = torch.zeros((16, features // 32 * 32 + 32), dtype=BF16)
    with pytest.raises(ValueError, match="features"):
        sl.linear_mxfp4_with_grad_accumulation(torch.zeros((4, features), dtype=BF16), w)
    assert not casts


def _copies(out, n_in, out_p, in_p):
    """Shapes of a weight's four MXFP4 tensors: rowwise [out, in_p], columnwise [n_in, out_p]."""
    u = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    return [u(out, in_p // 2), u(out, in_p // 32), u(n_in, out_p // 2), u(n_in, out_p // 32)]


@pytest.mark.parametrize("other", [(24, 72, 32, 96), (40, 64, 64, 64), (40, 104, 64, 128)], ids=["out", "in", "wider"])
def test_copies_of_another_weight_are_refused(casts, other):
    w = torch.nn.Parameter(torch.zeros((40, 72), dtype=BF16))
    w.main_grad = torch.zeros((40, 72))
    x = torch.zeros((4, 72), dtype=BF16, requires_grad=True)
    good = _copies(40, 72, 64, 96)
    assert sl.linear_mxfp4_with_grad_accumulation(x, w, weight_mxfp4=good).shape == (4, 40)
    bad = _copies(*other)
    del casts[:]
    for mixed in (bad, good[:2] + bad[2:], bad[:2] + good[2:], good[:1] + bad[1:2] + good[2:], good[:3]):
        if all(a.shape == b.shape for a, b in zip(mixed, good)) and len(mixed) == 4:
            continue
        with pytest.raises(ValueError, match="weight_mxfp4"):
            sl.linear_mxfp4_with_grad_accumulation(x, w, weight_mxfp4=mixed)
    with pytest.raises(ValueError, match="weight_mxfp4"):
        sl.linear_mxfp4_with_grad_accumulation(x, w, weight_mxfp4=[None, None] + good[2:])
    with pytest.raises(ValueError, match="columnwise"):
        sl.linear_mxfp4_with_grad_accumulation(x, w, weight_mxfp4=good[:2] + [None, None])
    assert not casts
