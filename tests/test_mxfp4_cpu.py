"""The MXFP4 oracle's pins and the entry points' argument checks (no GPU).

No call here reaches a kernel launch: each fails validation, or is a zero-extent no-op.
"""
import numpy as np
import pytest
import torch

import sharded_linear_amd as sl
import synth
from oracle import mxfp4
from oracle.numerics import bf16_bits_to_f64
from sharded_linear_amd import _lib

OK, EINVAL, EALIGN, ESHAPE, EWORKSPACE = 0, -1, -2, -3, -4
A = 1 << 20          # an aligned fake device address, never dereferenced
MIS = A + 2


def test_philox_published_answers():
    """Known answers of the generator's authors for a zero counter and key, 10 and 7 rounds."""
    zero = np.zeros(1, np.uint64)
    assert [hex(v) for v in mxfp4.philox4x32(zero, 0, 10)[0]] == ["0x6627e8d5", "0xe169c58d", "0xbc57ac4c", "0x9b00dbd8"]
    assert [hex(v) for v in mxfp4.philox4x32(zero, 0, 7)[0]] == ["0x5f6fb709", "0xd893f64", "0x4f121f81", "0x4f730a48"]


def test_draws_are_uniform_and_keyed():
    r = mxfp4.draws(64, 256, 12345)
    assert r.min() >= 0 and r.max() < 65536
    # mean of n uniform draws: 6 standard errors of 65536 / sqrt(12 n)
    assert abs(r.mean() - 32767.5) < 6 * 65536 / np.sqrt(12 * r.size)
    assert not np.array_equal(r, mxfp4.draws(64, 256, 12346))
    assert np.array_equal(r[:8], mxfp4.draws(8, 256, 12345))              # a draw depends on its place alone


def test_nearest_against_a_scalar_rule():
    """Every finite bf16 below a block maximum of 5.0 (X = 0), by distance to the grid."""
    grid = [0, .5, 1, 1.5, 2, 3, 4, 6]
    bits = np.arange(0, 0x40A0, 37, dtype=np.uint16)
    x = bf16_bits_to_f64(bits)
    for v in x:
        row = np.zeros((1, 32))
        row[0, 0], row[0, 1], row[0, 2] = 5.0, v, -v
        q, s = mxfp4.quantize(row)
        assert s[0, 0] == 127
        d = [abs(v - g) for g in grid]
        best = [i for i in range(8) if d[i] == min(d)]
        want = best[0] if len(best) == 1 else [i for i in best if i % 2 == 0][0]
        assert q[0, 0] >> 4 == want and q[0, 1] & 15 == want + 8, v


def test_nearest_hand_worked():
    row = np.array([[7.9, 6.0, 5.0, 2.5, 0.25, 0.75, -0.1, -7.0] + [0.0] * 24])
    q, s = mxfp4.quantize(row)
    assert s[0, 0] == 127
    assert list(q[0, :4]) == [7 | 7 << 4, 6 | 4 << 4, 0 | 2 << 4, 8 | 15 << 4]
    q, s = mxfp4.quantize(row * 2.0 ** -20)
    assert s[0, 0] == 107 and list(q[0, :2]) == [7 | 7 << 4, 6 | 4 << 4]


def test_stochastic_never_saturates_and_is_unbiased():
    x = bf16_bits_to_f64(synth.normal_bf16((4, 64), 5))
    total = np.zeros_like(x)
    n = 500
    for k in range(n):
        q, s = mxfp4.quantize(x, mxfp4.draws(4, 64, k))
        v = mxfp4.dequantize(q, s)
        unit = np.exp2(s.astype(float) - 127).repeat(32, 1)
        assert (np.abs(x) <= 6 * unit).all()
        assert (np.abs(v - x) <= 2 * unit).all()
        total += v
    # one rounding's standard deviation is at most half a step, 1.0 units; 6 standard errors
    assert (np.abs(total / n - x) <= 6 * unit / np.sqrt(n)).all()


def test_special_blocks_and_padding():
    x = np.zeros((3, 40))
    x[0, 3], x[1, 35], x[2, 0] = np.inf, np.nan, 2.0 ** -133          # the smallest bf16 subnormal
    q, s = mxfp4.quantize(x)
    assert q.shape == (3, 32) and s.shape == (3, 2)
    assert list(s[0]) == [255, 0] and list(s[1]) == [0, 255] and list(s[2]) == [0, 0]
    assert not q.any()
    assert np.isnan(mxfp4.dequantize(q, s)[0, :32]).all()


def test_quantize_validation():
    q = _lib.lib().sl_mxfp4_quantize
    tail = (0, 0, None)
    assert q(None, A, 64, 44, A, A, None, None, *tail) == ESHAPE                  # cols % 8
    assert q(None, A, -1, 64, A, A, None, None, *tail) == EINVAL
    assert q(None, A, 1 << 31, 64, A, A, None, None, *tail) == ESHAPE
    assert q(None, A, 64, 64, A, None, None, None, *tail) == EINVAL               # codes without scales
    assert q(None, A, 64, 64, None, None, None, A, *tail) == EINVAL
    assert q(None, None, 64, 64, A, A, None, None, *tail) == EINVAL
    assert q(None, MIS, 64, 64, A, A, None, None, *tail) == EALIGN
    assert q(None, A, 64, 64, MIS, A, None, None, *tail) == EALIGN
    assert q(None, A, 64, 64, None, None, MIS, A, *tail) == EALIGN
    assert q(None, A, 64, 64, A, A, None, None, 2, 0, None) == EINVAL             # no such rounding
    assert q(None, A, 64, 64, A, A, None, None, 1, 0, MIS) == EALIGN              # seed offset
    assert q(None, None, 0, 64, None, None, None, None, *tail) == OK
    assert q(None, None, 64, 64, None, None, None, None, *tail) == OK


def test_dequantize_validation():
    d = _lib.lib().sl_mxfp4_dequantize
    assert d(None, A, A, A, 64, 48) == ESHAPE
    assert d(None, A, A, A, -1, 64) == EINVAL
    assert d(None, None, A, A, 64, 64) == EINVAL
    assert d(None, A, A, None, 64, 64) == EINVAL
    assert d(None, MIS, A, A, 64, 64) == EALIGN
    assert d(None, A, A, MIS, 64, 64) == EALIGN
    assert d(None, None, None, None, 0, 64) == OK


@pytest.mark.parametrize("name,dims", [("sl_linear_fwd_mxfp4", lambda k, n: (k, n)), ("sl_linear_dgrad_mxfp4", lambda k, n: (n, k))])
def test_product_validation(name, dims):
    """dims(contracted, other) -> (in, out)"""
    L = _lib.lib()
    f, ws = getattr(L, name), getattr(L, f"sl_mxfp4_{name.split('_')[2]}_workspace_bytes")
    assert f(None, A, A, A, A, A, 16, *dims(48, 64), None, 0) == ESHAPE                    # contracted % 32
    assert f(None, A, A, A, A, A, 16, *dims(64, 12), None, 0) == ESHAPE                    # other % 8
    assert f(None, A, A, A, A, A, 16, *dims(1 << 24, 64), None, 0) == ESHAPE
    assert f(None, A, A, A, A, A, 16, *dims(64, 1 << 24), None, 0) == ESHAPE
    assert f(None, A, A, A, A, A, -1, *dims(64, 64), None, 0) == EINVAL
    assert f(None, A, A, A, A, A, 1 << 31, *dims(64, 64), None, 0) == ESHAPE
    assert f(None, A, A, A, A, A, (1 << 31) - 1, *dims(64, 1 << 23), None, 0) == ESHAPE        # too many tiles
    assert f(None, A, A, A, None, A, 16, *dims(64, 64), None, 0) == EINVAL
    assert f(None, MIS, A, A, A, A, 16, *dims(64, 64), None, 0) == EALIGN
    assert f(None, A, A, MIS, A, A, 16, *dims(64, 64), None, 0) == EALIGN
    assert f(None, A, A, A, A, MIS, 16, *dims(64, 64), None, 0) == EALIGN
    assert f(None, A, A, A, A, None, 16, *dims(0, 64), None, 0) == EINVAL
    assert f(None, None, None, None, None, None, 0, *dims(64, 64), None, 0) == OK
    assert f(None, None, None, None, None, None, 16, *dims(64, 0), None, 0) == OK
    assert ws(16, *dims(48, 64)) == 0 and ws(0, *dims(64, 64)) == 0 and ws(1, *dims(8192, 64)) == 0
    need = ws(200, *dims(8192, 64))                                               # few tiles, a long sum: split
    assert need and need % (200 * 64 * 4) == 0
    assert f(None, A, A, A, A, A, 200, *dims(8192, 64), None, 0) == EWORKSPACE
    assert f(None, A, A, A, A, A, 200, *dims(8192, 64), A, need - 1) == EWORKSPACE
    assert f(None, A, A, A, A, A, 200, *dims(8192, 64), MIS, need) == EWORKSPACE


@pytest.mark.parametrize("cfg", [-1, 0, 1])
def test_few_tokens_need_no_workspace(cfg):
    L = _lib.lib()
    with sl.tuning(f8=cfg):
        for T in (1, 16):
            assert L.sl_mxfp4_fwd_workspace_bytes(T, 16384, 64) == 0 and L.sl_mxfp4_dgrad_workspace_bytes(T, 64, 16384) == 0
            assert L.sl_mxfp4w_fwd_workspace_bytes(T, 16384, 64) == 0 and L.sl_mxfp4w_fwd_workspace_bytes(T, 64, 1 << 18) == 0


def test_workspaces_of_another_device_are_refused():
    for ws in (torch.zeros(64, dtype=torch.uint8), torch.zeros((8, 8), dtype=torch.uint8)[:, :4]):
        with pytest.raises(ValueError, match="workspace"):
            sl.ops._scratch(torch.device("cuda", 0) if ws.is_contiguous() else ws.device, 32, ws)


def test_wgrad_validation():
    L = _lib.lib()
    w = L.sl_linear_wgrad_accum_mxfp4
    assert w(None, A, A, A, A, A, 48, 64, 64, None, 0) == ESHAPE                  # T % 32
    assert w(None, A, A, A, A, A, 64, 60, 64, None, 0) == ESHAPE
    assert w(None, A, A, A, A, A, -32, 64, 64, None, 0) == EINVAL
    assert w(None, A, A, A, None, A, 64, 64, 64, None, 0) == EINVAL
    assert w(None, A, A, A, A, MIS, 64, 64, 64, None, 0) == EALIGN
    assert w(None, A, A, MIS, A, A, 64, 64, 64, None, 0) == EALIGN
    assert w(None, None, None, None, None, None, 0, 64, 64, None, 0) == OK
    assert L.sl_mxfp4_wgrad_workspace_bytes(48, 64, 64) == 0 and L.sl_mxfp4_wgrad_workspace_bytes(0, 64, 64) == 0
    for T, n_in, n_out in [(8192, 2048, 1536), (4096, 256, 256), (64, 64, 64)]:
        need = L.sl_mxfp4_wgrad_workspace_bytes(T, n_in, n_out)
        assert need or T != 4096
        assert need % (n_in * n_out * 4) == 0
        if need:
            assert w(None, A, A, A, A, A, T, n_in, n_out, None, 0) == EWORKSPACE
            assert w(None, A, A, A, A, A, T, n_in, n_out, A, need - 1) == EWORKSPACE
            assert w(None, A, A, A, A, A, T, n_in, n_out, MIS, need) == EWORKSPACE


@pytest.mark.parametrize("which", ["fwd", "dgrad"])
def test_mxfp4w_validation(which):
    L = _lib.lib()
    f, ws = getattr(L, f"sl_linear_{which}_mxfp4w"), getattr(L, f"sl_mxfp4w_{which}_workspace_bytes")
    assert f(None, A, A, A, A, 16, 48, 64, A, 1 << 40) == ESHAPE                  # in % 32
    assert f(None, A, A, A, A, 16, 64, 12, A, 1 << 40) == ESHAPE
    assert f(None, A, A, A, A, -1, 64, 64, A, 1 << 40) == EINVAL
    assert f(None, None, A, A, A, 16, 64, 64, A, 1 << 40) == EINVAL
    assert f(None, A, A, None, A, 16, 64, 64, A, 1 << 40) == EINVAL
    assert f(None, MIS, A, A, A, 16, 64, 64, A, 1 << 40) == EALIGN
    assert f(None, A, MIS, A, A, 16, 64, 64, A, 1 << 40) == EALIGN
    assert f(None, None, None, None, None, 0, 64, 64, None, 0) == OK
    assert ws(16, 48, 64) == 0 and ws(0, 64, 64) == 0
    for T, n_in, n_out, unit in [(8192, 2048, 8192, 2048 * 8192 * 2), (100, 4096, 4096, 100 * 4096 * 4)]:
        need = ws(T, n_in, n_out)                                                 # a bf16 weight; planes of a split sum
        assert need and need % unit == 0
        assert f(None, A, A, A, A, T, n_in, n_out, None, 0) == EWORKSPACE
        assert f(None, A, A, A, A, T, n_in, n_out, A, need - 1) == EWORKSPACE
        assert f(None, A, A, A, A, T, n_in, n_out, MIS, need) == EWORKSPACE


def test_python_refuses_cpu_tensors():
    b, u = torch.zeros(32, 32, dtype=torch.bfloat16), torch.zeros(32, 16, dtype=torch.uint8)
    s = torch.zeros(32, 1, dtype=torch.uint8)
    for call in (lambda: sl.sl_mxfp4_quantize(b), lambda: sl.sl_mxfp4_dequantize(u, s),
                 lambda: sl.sl_linear_fwd_mxfp4(u, s, u, s), lambda: sl.sl_linear_dgrad_mxfp4(u, s, u, s),
                 lambda: sl.sl_linear_wgrad_accum_mxfp4(u, s, u, s, torch.zeros(32, 32)),
                 lambda: sl.sl_linear_fwd_mxfp4w(b, u, s), lambda: sl.sl_linear_dgrad_mxfp4w(b, u, s)):
        with pytest.raises(ValueError):
            call()


def test_autograd_refuses_a_weight_without_main_grad():
    w = torch.nn.Parameter(torch.zeros(32, 32, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="main_grad"):
        sl.linear_mxfp4_with_grad_accumulation(torch.zeros(4, 32, dtype=torch.bfloat16), w)


def test_cast_of_more_tiles_than_a_launch_takes_is_refused():
    q = _lib.lib().sl_mxfp4_quantize
    for rows, cols in (((1 << 31) - 1, 8), ((1 << 31) - 127, 128), (1 << 30, 136)):
        assert q(None, A, rows, cols, A, A, A, A, 0, 0, None) == ESHAPE
