"""MXFP4 products where addresses, scales and streams are at their limits.

Every sum here is of integers or halves small enough to be exact in fp32 (or compared with the same
call's bits), so results have to be the correctly rounded ones.
"""
import numpy as np
import pytest
import torch

import sharded_linear_amd as sl
import synth
from oracle import mxfp4
from oracle.numerics import bf16_bits_to_f64
from sharded_linear_amd import ops
from tests.gpu_util import dev_bf16, dev_u8, host_f64, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    yield
    torch.cuda.synchronize()


def _dev(m):
    return dev_u8(m[0]), dev_u8(m[1])


def _codes(rows, k, seed, scale=127, small=False):
    """Random codes under one scale; small: magnitudes up to 1.5."""
    g = np.random.default_rng(seed)
    q = g.integers(0, 256, (rows, k // 2), dtype=np.uint8)
    return (q & 0xBB if small else q), np.full((rows, k // 32), scale, np.uint8)


def _ints(rows, cols, seed, power=0):
    """bf16 integers of -8 .. 8 times 2^power: patterns and values."""
    v = np.random.default_rng(seed).integers(-8, 9, (rows, cols)).astype(np.float64) * 2.0 ** power
    return synth.f32_to_bf16_bits(v.astype(np.float32)), v


def _rounded(ref):
    return bf16_bits_to_f64(synth.f32_to_bf16_bits(ref.astype(np.float32)))


def _moved(s, off):
    """The scales at an address off bytes behind an aligned one, NaN scales all around."""
    buf = torch.full((s.numel() + 8,), 255, dtype=torch.uint8, device="cuda")
    buf[off:off + s.numel()] = s.view(-1)
    return buf[off:off + s.numel()].view(s.shape)


# odd numbers of blocks to a row; several splits, one, and a bf16 copy of the weight
@pytest.mark.parametrize("T,n_in,n_out", [(1, 96, 2056), (5, 544, 4104), (70, 288, 1032), (200, 544, 136), (1100, 96, 264)])
def test_frozen_weight_gradient_with_scales_at_any_address(T, n_in, n_out):
    say(f"case mxfp4w gradient scale offsets T={T} in={n_in} out={n_out}")
    q, s = _dev(mxfp4.quantize(np.random.default_rng(T).standard_normal((n_out, n_in))))
    dY = torch.randn((T, n_out), device="cuda").bfloat16()
    want = sl.sl_linear_dgrad_mxfp4w(dY, q, s)
    assert torch.isfinite(want).all() and want.any()
    for off in (1, 2, 3):
        assert torch.equal(sl.sl_linear_dgrad_mxfp4w(dY, q, _moved(s, off)), want), off


@pytest.mark.parametrize("n_out,n_in,T", [(136, 72, 8224), (264, 264, 544), (8, 8, 32)])
def test_weight_gradient_with_scales_at_any_address(n_out, n_in, T):
    say(f"case mxfp4 wgrad scale offsets out={n_out} in={n_in} T={T}")
    assert bool(sl.sl_mxfp4_wgrad_workspace_bytes(T, n_in, n_out)) == (T == 8224)
    (aq, as_), (bq, bs) = (_dev(mxfp4.quantize(np.random.default_rng(r).standard_normal((r, T)))) for r in (n_out, n_in))
    want = torch.ones((n_out, n_in), device="cuda")
    sl.sl_linear_wgrad_accum_mxfp4(aq, as_, bq, bs, want)
    assert torch.isfinite(want).all()
    for off in (1, 2, 3):
        g = torch.ones((n_out, n_in), device="cuda")
        sl.sl_linear_wgrad_accum_mxfp4(aq, _moved(as_, off), bq, _moved(bs, 4 - off), g)
        assert torch.equal(g, want), off


@pytest.mark.parametrize("T,n_out", [(1, 72), (40, 72), (130, 4104), (600, 72), (1100, 72)])
def test_nan_block_of_a_frozen_weight_reaches_its_columns_only(T, n_out):
    """In the last block of a row, past which a tile holds the next row's scales, and in the first of the row after."""
    say(f"case mxfp4w gradient NaN block T={T} out={n_out}")
    w = _codes(n_out, 544, T)
    bits, dy = _ints(T, n_out, T + 1)
    ref = dy @ mxfp4.dequantize(*w)
    for blocks in ([(n_out - 1, 16)], [(3, 16), (4, 0)], [(0, 5)]):
        s = w[1].copy()
        bad = np.zeros(544, bool)
        for r, b in blocks:
            s[r, b] = 255
            bad[32 * b:32 * b + 32] = True
        dX = host_f64(sl.sl_linear_dgrad_mxfp4w(dev_bf16(bits), dev_u8(w[0]), dev_u8(s)))
        assert np.isnan(dX[:, bad]).all(), blocks
        assert np.array_equal(dX[:, ~bad], _rounded(ref)[:, ~bad]), blocks


# scale 0 with activations of 2^120, scale 254 with 2^-120 (there the larger codes pass bf16's range)
@pytest.mark.parametrize("T", [1, 3, 16, 20, 40, 200, 1100])
@pytest.mark.parametrize("scale,power", [(0, 120), (1, 119), (254, -120)])
def test_smallest_and_largest_scales_of_a_weight(T, scale, power):
    say(f"case mxfp4w scale {scale} T={T}")
    n_in, n_out = 288, 264
    w = _codes(n_out, n_in, T, scale, small=scale == 254)
    one = mxfp4.dequantize(w[0], np.full_like(w[1], 127))
    unit = 2.0 ** (scale - 127 + power)
    bits, _ = _ints(T, n_in, T + 1, power)
    _, x = _ints(T, n_in, T + 1)
    Y = host_f64(sl.sl_linear_fwd_mxfp4w(dev_bf16(bits), *_dev(w)))
    assert np.array_equal(Y, _rounded(x @ one.T) * unit)
    bits, _ = _ints(T, n_out, T + 2, power)
    _, y = _ints(T, n_out, T + 2)
    dX = host_f64(sl.sl_linear_dgrad_mxfp4w(dev_bf16(bits), *_dev(w)))
    assert np.array_equal(dX, _rounded(y @ one) * unit)


@pytest.mark.parametrize("M", [3, 48, 300])
@pytest.mark.parametrize("sa,sb", [(0, 247), (247, 0), (254, 7), (7, 254)])
def test_smallest_and_largest_scales_of_both_operands(M, sa, sb):
    say(f"case mxfp4 scales {sa} and {sb} M={M}")
    a, b = _codes(M, 288, 1, sa), _codes(264, 288, 2, sb)
    ref = mxfp4.dequantize(a[0], np.full_like(a[1], 127)) @ mxfp4.dequantize(b[0], np.full_like(b[1], 127)).T
    Y = host_f64(sl.sl_linear_fwd_mxfp4(*_dev(a), *_dev(b)))
    assert np.array_equal(Y, _rounded(ref) * 2.0 ** (sa + sb - 254))


def test_two_side_streams_with_operands_of_their_own(monkeypatch):
    """Split sums on two streams at a time, each on inputs that its own stream writes late, the default stream busy: a
    launch on another stream would read stale inputs or leave its result too late, and shared planes would mix."""
    say("case mxfp4 two side streams")
    taken = []
    plain = ops.wgrad_workspace

    def noted(dev, nbytes):
        t = plain(dev, nbytes)
        taken.append((torch.cuda.current_stream(dev).cuda_stream, t.data_ptr(), nbytes))
        return t

    cases = []
    for k in range(2):
        g = np.random.default_rng(k)
        a, b, w = (mxfp4.quantize(g.standard_normal(s)) for s in ((200, 8192), (64, 8192), (4096, 96)))
        real = [*_dev(a), *_dev(b), *_dev(w), torch.randn((100, 8192), device="cuda").bfloat16(),
                torch.randn((100, 4096), device="cuda").bfloat16()]
        held = [torch.zeros_like(t) for t in real]

        def run(t, fill):
            outs = [torch.full(s, float("nan"), dtype=torch.bfloat16, device="cuda") for s in ((200, 64), (100, 64), (100, 96))]
            grad = torch.zeros((200, 64), device="cuda")
            fill()
            sl.sl_linear_fwd_mxfp4(*t[:4], outs[0])
            sl.sl_linear_fwd_mxfp4w(t[6], *t[2:4], outs[1])
            sl.sl_linear_dgrad_mxfp4w(t[7], *t[4:6], outs[2])
            sl.sl_linear_wgrad_accum_mxfp4(*t[:4], grad)
            return [o.clone() for o in (*outs, grad)]

        want = run(real, lambda: None)
        cases.append((real, held, run, want))
    assert sl.sl_mxfp4_fwd_workspace_bytes(200, 8192, 64) and sl.sl_mxfp4w_fwd_workspace_bytes(100, 8192, 64)
    assert sl.sl_mxfp4w_dgrad_workspace_bytes(100, 96, 4096) and sl.sl_mxfp4_wgrad_workspace_bytes(8192, 64, 200)
    big = torch.ones((4096, 4096), device="cuda")
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    monkeypatch.setattr(ops, "wgrad_workspace", noted)
    for _ in range(10):
        big @ big                                                  # the default stream, some milliseconds
    got = []
    for s, (real, held, run, _want) in zip(streams, cases):
        with torch.cuda.stream(s):
            own = torch.ones((4096, 4096), device="cuda")

            def late(held=held, real=real, own=own):
                for _ in range(3):
                    own @ own
                for h, r in zip(held, real):
                    h.copy_(r)
            got.append(run(held, late))
    torch.cuda.synchronize()
    for outs, (_real, _held, _run, want) in zip(got, cases):
        for o, w in zip(outs, want):
            assert torch.equal(o, w)
    assert {t[0] for t in taken} == {s.cuda_stream for s in streams} and len(taken) == 8
    for s, p, n in taken:
        for t, q, m in taken:
            assert s == t or p + n <= q or q + m <= p
