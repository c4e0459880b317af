"""The MXFP4 operators on the GPU against their definition in float64.

Casts are compared code for code.  Products: every sum's error is at most K fp32 roundings of partial
sums no larger than S = sum |a||b|, 2^-24 each (counted as 2^-23, one unit, in case the matrix unit cuts
instead of rounding), and a bf16 result adds half a bf16 step, 2^-8 of its value:
    |got - ref| <= K 2^-23 S + 2^-8 |ref| (1 + K 2^-23)
Where every partial sum is exact in fp32 the result has to be the correctly rounded one.
"""
import numpy as np
import pytest
import torch

import sharded_linear_amd as sl
import synth
from oracle import mxfp4
from oracle.numerics import bf16_bits_to_f64
from tests.gpu_util import dev_bf16, dev_u8, host_bits, host_f64, say

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    assert torch.cuda.is_available(), "GPU tests need a HIP device"
    yield
    torch.cuda.synchronize()


def _host(t):
    return t.cpu().numpy()


def _bits(rows, cols, seed, std=1.0):
    """bf16 patterns whose rows and columns differ in size by powers of two."""
    g = np.random.default_rng(seed)
    x = g.standard_normal((rows, cols)) * std * np.exp2(g.integers(-6, 7, (rows, 1)) + g.integers(-6, 7, (1, cols)))
    return synth.f32_to_bf16_bits(x.astype(np.float32))


def _f64(bits):
    with np.errstate(invalid="ignore"):                     # signalling NaN patterns among the inputs
        return bf16_bits_to_f64(bits)


def _check_cast(bits, seed=None, key=None):
    x = _f64(bits)
    r = None if seed is None else mxfp4.draws(*x.shape, seed if key is None else key)
    got = [_host(t) for t in sl.sl_mxfp4_quantize(dev_bf16(bits), seed=seed)]
    want = [*mxfp4.quantize(x, r), *mxfp4.quantize(x.T, None if r is None else r.T)]
    for g, w, name in zip(got, want, ("q_rows", "s_rows", "q_cols", "s_cols")):
        assert g.shape == w.shape
        assert np.array_equal(g, w), (name, int((g != w).sum()))
    return got


# ---- casts --------------------------------------------------------------------------------------

@pytest.mark.parametrize("seed", [None, 99])
def test_cast_every_bf16_pattern(seed):
    """Every pattern, subnormals, infinities and NaNs among them: in blocks of neighbours (rows) and in blocks
    of all sizes (columns), and next to block maxima 2^0 .. 2^3 and 2^-125 above them."""
    say(f"case cast every pattern seed={seed}")
    p = np.arange(65536, dtype=np.uint32).astype(np.uint16)
    _check_cast(p.reshape(512, 128), seed)
    finite = p[(p & 0x7F80) != 0x7F80]
    m = finite.reshape(-1, 16)                                   # 65024 = 4064 x 16
    lead = np.zeros((m.shape[0], 16), np.uint16)
    top = (m & 0x7FFF).max(1).astype(np.int64)
    lead[:, 0] = np.minimum(top + 128 * (np.arange(m.shape[0]) % 4), 0x7F7F)
    _check_cast(np.concatenate([lead, m], 1), seed)
    small = np.tile(p[:0x0400].reshape(-1, 32), (1, 1))           # subnormal blocks and just above: X clamps
    _check_cast(small, seed)


@pytest.mark.parametrize("rows,cols", [(1, 8), (1, 32), (31, 40), (33, 64), (128, 128), (129, 136), (300, 1040), (257, 2064), (1000, 72)])
@pytest.mark.parametrize("seed", [None, 0, (1 << 63) + 12345])
def test_cast_shapes(rows, cols, seed):
    say(f"case cast {rows}x{cols} seed={seed}")
    _check_cast(_bits(rows, cols, rows + cols), seed)


@pytest.mark.parametrize("scale", [1.0, 2.0 ** 100, 2.0 ** -60, 2.0 ** -123])
def test_cast_largest_draws_on_the_smallest_values(scale):
    """Where the draw is 2^16 - 1 a value of one draw's unit rounds up and anything less does not: values on both sides of
    it, down to what only a cut, not a rounding, of v keeps apart."""
    say(f"case cast largest draws scale={scale}")
    rows, cols, key = 1024, 1024, 7
    at = np.argwhere(mxfp4.draws(rows, cols, key) == 65535)
    at = at[(at % 32 != 0).all(1)]
    assert len(at) > 8
    x = np.zeros((rows, cols), np.float32)
    x[::32, :], x[:, ::32] = 6, 6                                # v = x in every block, by rows and by columns
    unit = 2.0 ** -17                                             # of the draw where the step is 0.5
    for k, (i, j) in enumerate(at):
        x[i, j] = unit * (255 / 256, 1, 129 / 128, 2.0 ** -9, 127 / 128, 255 / 128, 255 / 1024, -255 / 256)[k % 8]
    _check_cast(synth.f32_to_bf16_bits((x * np.float32(scale)).astype(np.float32)), key)


def test_cast_zero_and_non_finite_blocks():
    say("case cast zero / non-finite blocks")
    b = _bits(96, 96, 3)
    b[:32, :32] = 0
    b[32:64, 32:64] = 0x8000                                     # negative zeros
    b[70, 5], b[71, 40], b[3, 90] = 0x7F80, 0xFF80, 0x7FC1
    for seed in (None, 5):
        q, s, qc, sc = _check_cast(b, seed)
        assert s[70, 0] == 255 and s[71, 1] == 255 and s[3, 2] == 255 and sc[5, 2] == 255
        v = host_f64(sl.sl_mxfp4_dequantize(dev_u8(q), dev_u8(s)))
        assert np.isnan(v[70, :32]).all() and not np.isnan(v[70, 32:]).any()


def test_cast_one_copy_and_given_outputs():
    say("case cast one copy / outputs with guard bytes")
    b = _bits(129, 136, 8)
    x = dev_bf16(b)
    both = sl.sl_mxfp4_quantize(x)
    r = sl.sl_mxfp4_quantize(x, cols=False)
    c = sl.sl_mxfp4_quantize(x, rows=False)
    assert r[2] is None and r[3] is None and c[0] is None and c[1] is None
    for a, g in ((both[0], r[0]), (both[1], r[1]), (both[2], c[2]), (both[3], c[3])):
        assert torch.equal(a, g)
    out, guards = [], []
    for t in both:
        full = torch.full((t.numel() + 512,), 0xA5, dtype=torch.uint8, device="cuda")
        out.append(full[256:256 + t.numel()].view(t.shape))
        guards.append((full, t.numel()))
    got = sl.sl_mxfp4_quantize(x, out=tuple(out))
    for g, t, (full, n) in zip(got, both, guards):
        assert torch.equal(g, t)
        assert (full[:256] == 0xA5).all() and (full[256 + n:] == 0xA5).all()


def test_stochastic_seeds():
    say("case stochastic seeds")
    x = dev_bf16(_bits(256, 256, 4))
    a, b = sl.sl_mxfp4_quantize(x, seed=7), sl.sl_mxfp4_quantize(x, seed=7)
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    assert not torch.equal(a[0], sl.sl_mxfp4_quantize(x, seed=8)[0])
    t = torch.tensor([7], dtype=torch.int64, device="cuda")
    assert all(torch.equal(p, q) for p, q in zip(a, sl.sl_mxfp4_quantize(x, seed=t)))
    neg = torch.tensor([-3], dtype=torch.int64, device="cuda")
    assert torch.equal(sl.sl_mxfp4_quantize(x, seed=neg)[0], sl.sl_mxfp4_quantize(x, seed=-3)[0])


def test_cast_large_index():
    """More than 2^32 bytes of input: the last rows of a long matrix, by element."""
    rows, cols = (1 << 21) + 3, 1040
    say(f"case cast {rows}x{cols}")
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    b = _bits(67, cols, 5)
    x[-67:] = dev_bf16(b)
    r = mxfp4.philox4x32(np.arange((rows - 67) * cols // 8, rows * cols // 8), 11, 7)
    d = np.stack([r & np.uint64(0xFFFF), r >> np.uint64(16)], -1).astype(np.int64).reshape(67, cols)
    q, s, qc, sc = sl.sl_mxfp4_quantize(x, seed=11)
    wq, ws = mxfp4.quantize(_f64(b), d)
    assert np.array_equal(_host(q[-67:]), wq) and np.array_equal(_host(s[-67:]), ws)
    assert not q[:-67].any() and not s[:-67].any()
    # columns: the last 67 rows are rows 0..2 of the last block, and two whole blocks before it
    wq, ws = mxfp4.quantize(_f64(b).T[:, :64], d.T[:, :64])
    assert np.array_equal(_host(qc[:, -48:-16]), wq) and np.array_equal(_host(sc[:, -3:-1]), ws)
    wq, ws = mxfp4.quantize(_f64(b).T[:, 64:], d.T[:, 64:])
    assert np.array_equal(_host(qc[:, -16:]), wq) and np.array_equal(_host(sc[:, -1:]), ws)


def test_dequantize_every_code_with_every_scale():
    say("case dequantise every code x every scale")
    pairs = np.arange(256, dtype=np.uint8)
    q = np.tile(pairs, (256, 1))                                  # 512 elements: 16 blocks to a row
    s = np.repeat(np.arange(256, dtype=np.uint8)[:, None], 16, 1)
    got = host_f64(sl.sl_mxfp4_dequantize(dev_u8(q), dev_u8(s)))
    want = mxfp4.dequantize(q, s)
    want[np.abs(want) >= 2.0 ** 128] *= np.inf
    assert np.array_equal(got, want, equal_nan=True)


@pytest.mark.parametrize("rows,cols", [(1, 32), (7, 96), (300, 1056), (4097, 288)])
def test_dequantize_shapes(rows, cols):
    say(f"case dequantise {rows}x{cols}")
    g = np.random.default_rng(rows)
    q, s = g.integers(0, 256, (rows, cols // 2), dtype=np.uint8), g.integers(0, 250, (rows, cols // 32), dtype=np.uint8)
    assert np.array_equal(host_f64(sl.sl_mxfp4_dequantize(dev_u8(q), dev_u8(s))), mxfp4.dequantize(q, s))


# ---- products -----------------------------------------------------------------------------------

def _operand(rows, k, seed):
    return mxfp4.quantize(_f64(_bits(rows, k, seed)))


def _exact_operand(rows, k, seed):
    """Codes of 0, +-0.5 .. +-6 under scales of 1 and 2: with k < 2^14 every partial sum of products is a multiple
    of 1/4 below 2^22, exact in fp32."""
    g = np.random.default_rng(seed)
    return g.integers(0, 256, (rows, k // 2), dtype=np.uint8), g.integers(127, 129, (rows, k // 32), dtype=np.uint8)


def _dev(m):
    return dev_u8(m[0]), dev_u8(m[1])


def _close(got, ref, S, K, bf16=True):
    got = host_f64(got)
    tol = K * 2.0 ** -23 * S + (2.0 ** -8 * np.abs(ref) * (1 + K * 2.0 ** -23) if bf16 else 0)
    over = np.abs(got - ref) - tol
    assert np.isfinite(got).all() and (over <= 0).all(), (float(over.max()), int((over > 0).sum()))


def _bf16_exact(ref):
    return synth.f32_to_bf16_bits(ref.astype(np.float32))


# (M, N, K): one row to many, extents that fill no tile, contracted extents with whole and part groups of scales
PRODUCTS = [(1, 8, 32), (1, 256, 2048), (2, 40, 96), (5, 1000, 1056), (16, 264, 4096), (17, 520, 544), (33, 72, 5504),
            (64, 256, 512), (65, 776, 288), (100, 1544, 1024), (128, 128, 32), (129, 136, 160), (200, 4096, 160),
            (256, 256, 512), (257, 264, 544), (300, 2056, 1056), (72, 136, 4128), (130, 264, 5504), (65, 1160, 2336), (1000, 776, 1056), (513, 1032, 2080), (2048, 1536, 96)]


@pytest.mark.parametrize("M,N,K", PRODUCTS)
def test_fwd_and_dgrad(M, N, K):
    say(f"case mxfp4 product {M}x{N}x{K}")
    a, b = _operand(M, K, M + K), _operand(N, K, N + 2 * K)
    ref, S = mxfp4.product(a, b)
    Y = sl.sl_linear_fwd_mxfp4(*_dev(a), *_dev(b))
    dX = sl.sl_linear_dgrad_mxfp4(*_dev(a), *_dev(b))
    _close(Y, ref, S, K)
    assert torch.equal(Y.view(torch.int16), dX.view(torch.int16))
    a, b = _exact_operand(M, K, M), _exact_operand(N, K, N + 1)
    Y = sl.sl_linear_fwd_mxfp4(*_dev(a), *_dev(b))
    assert np.array_equal(host_bits(Y) & 0x7FFF, _bf16_exact(mxfp4.product(a, b)[0]) & 0x7FFF)
    assert np.array_equal(host_f64(Y), bf16_bits_to_f64(_bf16_exact(mxfp4.product(a, b)[0])))


@pytest.mark.parametrize("n_out,n_in,T", [(m + -m % 8, n, k) for m, n, k in PRODUCTS] + [(256, 256, 8192), (1536, 2048, 4096)])
def test_wgrad(n_out, n_in, T):
    say(f"case mxfp4 wgrad out={n_out} in={n_in} T={T}")
    a, b = _operand(n_out, T, T + 1), _operand(n_in, T, T + 2)
    ref, S = mxfp4.product(a, b)
    g0 = np.random.default_rng(T).standard_normal(ref.shape).astype(np.float32) * np.float32(np.sqrt((ref ** 2).mean()))
    pad = torch.full((n_out * n_in + 128,), 7.0, device="cuda")
    g = pad[64:-64].view(n_out, n_in)
    g.copy_(torch.from_numpy(g0))
    for k in (1, 2):
        sl.sl_linear_wgrad_accum_mxfp4(*_dev(a), *_dev(b), g)
        # each call adds one rounding of the running gradient, and one for each partial plane (16 at most)
        tot = np.abs(g0) + k * S
        _close(g, g0 + k * ref, tot, k * (T + 17), bf16=False)
    assert (pad[:64] == 7.0).all() and (pad[-64:] == 7.0).all()
    a, b = _exact_operand(n_out, T, 1), _exact_operand(n_in, T, 2)
    g.zero_()
    sl.sl_linear_wgrad_accum_mxfp4(*_dev(a), *_dev(b), g)
    assert np.array_equal(host_f64(g), mxfp4.product(a, b)[0])


@pytest.mark.parametrize("M,N,K", [(1, 64, 544), (20, 72, 1056), (300, 264, 512), (513, 520, 160)])
def test_scales_at_any_address(M, N, K):
    """Scale arrays 1, 2 and 3 bytes behind an aligned address give the same bits."""
    say(f"case mxfp4 scale offsets {M}x{N}x{K}")
    (aq, as_), (bq, bs) = _dev(_operand(M, K, 1)), _dev(_operand(N, K, 2))
    X = torch.randn((M, K), device="cuda").bfloat16()
    want = sl.sl_linear_fwd_mxfp4(aq, as_, bq, bs)
    want_w = sl.sl_linear_fwd_mxfp4w(X, bq, bs)
    for o in (1, 2, 3):
        moved = []
        for s, off in ((as_, o), (bs, 4 - o)):
            buf = torch.full((s.numel() + 8,), 255, dtype=torch.uint8, device="cuda")     # NaN scales all around
            buf[off:off + s.numel()] = s.view(-1)
            moved.append(buf[off:off + s.numel()].view(s.shape))
        got = sl.sl_linear_fwd_mxfp4(aq, moved[0], bq, moved[1])
        assert torch.equal(got.view(torch.int16), want.view(torch.int16)), o
        got = sl.sl_linear_fwd_mxfp4w(X, bq, moved[1])
        assert torch.equal(got.view(torch.int16), want_w.view(torch.int16)), o


@pytest.mark.parametrize("M,N,K", [(3, 64, 544), (40, 72, 1056), (300, 264, 512)])
def test_nan_blocks_reach_their_rows_only(M, N, K):
    say(f"case mxfp4 NaN scales {M}x{N}x{K}")
    a, b = _exact_operand(M, K, 1), _exact_operand(N, K, 2)
    ref = mxfp4.product(a, b)[0]
    a[1][M - 1, K // 32 - 1] = 255
    b[1][7, 0] = 255
    Y = host_f64(sl.sl_linear_fwd_mxfp4(*_dev(a), *_dev(b)))
    bad = np.zeros((M, N), bool)
    bad[M - 1], bad[:, 7] = True, True
    assert np.isnan(Y[bad]).all()
    assert np.array_equal(Y[~bad], bf16_bits_to_f64(_bf16_exact(ref))[~bad])


def test_extreme_scales():
    """Products of scales at both ends of their range, whose result is a normal number."""
    say("case mxfp4 extreme scales")
    a, b = _exact_operand(48, 256, 1), _exact_operand(40, 256, 2)
    want = mxfp4.product(a, b)[0]
    for sa, sb in ((-126, 120), (120, -126), (60, -60)):
        x = (a[0], (a[1].astype(int) + sa).astype(np.uint8)), (b[0], (b[1].astype(int) + sb).astype(np.uint8))
        got = host_f64(sl.sl_linear_fwd_mxfp4(*_dev(x[0]), *_dev(x[1])))
        assert np.array_equal(got, bf16_bits_to_f64(_bf16_exact(want)) * 2.0 ** (sa + sb))


def test_empty_extents():
    say("case mxfp4 empty extents")
    u = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    assert sl.sl_linear_fwd_mxfp4(u(0, 32), u(0, 2), u(8, 32), u(8, 2)).shape == (0, 8)
    Y = torch.full((4, 8), 3.0, dtype=torch.bfloat16, device="cuda")
    assert not sl.sl_linear_fwd_mxfp4(u(4, 0), u(4, 0), u(8, 0), u(8, 0), Y).any()        # an empty sum is 0
    Y.fill_(3.0)
    assert not sl.sl_linear_fwd_mxfp4w(bf(4, 0), u(8, 0), u(8, 0), Y).any()
    assert sl.sl_linear_fwd_mxfp4w(bf(0, 64), u(8, 32), u(8, 2)).shape == (0, 8)
    dX = torch.full((4, 64), 3.0, dtype=torch.bfloat16, device="cuda")
    assert not sl.sl_linear_dgrad_mxfp4w(bf(4, 0), u(0, 32), u(0, 2), dX).any()
    for T in (100, 1100):
        Y = torch.full((T, 8), 3.0, dtype=torch.bfloat16, device="cuda")
        assert not sl.sl_linear_fwd_mxfp4w(bf(T, 0), u(8, 0), u(8, 0), Y).any()
        Y.fill_(3.0)
        assert not sl.sl_linear_fwd_mxfp4(u(T, 0), u(T, 0), u(8, 0), u(8, 0), Y).any()
        dX = torch.full((T, 64), 3.0, dtype=torch.bfloat16, device="cuda")
        assert not sl.sl_linear_dgrad_mxfp4w(bf(T, 0), u(0, 32), u(0, 2), dX).any()
    g = torch.ones((8, 16), device="cuda")
    sl.sl_linear_wgrad_accum_mxfp4(u(8, 0), u(8, 0), u(16, 0), u(16, 0), g)
    assert (g == 1).all()
    q, s, qc, sc = sl.sl_mxfp4_quantize(bf(0, 64))
    assert q.shape == (0, 32) and qc.shape == (64, 0)


# ---- bf16 activations, 4-bit weights --------------------------------------------------------------

@pytest.mark.parametrize("T,n_in,n_out", [(1, 32, 8), (1, 2048, 512), (2, 96, 40), (3, 1056, 1000), (8, 4096, 264),
                                          (15, 544, 520), (16, 5504, 72), (17, 160, 136), (32, 1024, 776), (33, 288, 2056),
                                          (48, 2048, 128), (64, 512, 264), (65, 544, 136), (200, 1056, 4096),
                                          (256, 256, 256), (257, 2080, 520), (3, 96, 9000), (40, 8192, 136), (4, 5504, 264), (32, 6176, 72), (17, 8192, 40), (100, 5504, 72),
                                          (300, 96, 5504), (1000, 1056, 776), (1023, 2080, 2056), (2049, 512, 1032)])
def test_fwd_and_dgrad_mxfp4w(T, n_in, n_out):
    say(f"case mxfp4w T={T} in={n_in} out={n_out}")
    w = _operand(n_out, n_in, n_in)
    xb, yb = _bits(T, n_in, T), _bits(T, n_out, T + 1)
    ref, S = mxfp4.product(_f64(xb), w)
    _close(sl.sl_linear_fwd_mxfp4w(dev_bf16(xb), *_dev(w)), ref, S, n_in)
    ref, S = mxfp4.product(_f64(yb), mxfp4.dequantize(*w).T)
    _close(sl.sl_linear_dgrad_mxfp4w(dev_bf16(yb), *_dev(w)), ref, S, n_out)
    # small integers: every partial sum exact
    g = np.random.default_rng(T)
    w = _exact_operand(n_out, n_in, 1)
    xb = synth.f32_to_bf16_bits(g.integers(-8, 9, (T, n_in)).astype(np.float32))
    yb = synth.f32_to_bf16_bits(g.integers(-8, 9, (T, n_out)).astype(np.float32))
    Y = sl.sl_linear_fwd_mxfp4w(dev_bf16(xb), *_dev(w))
    assert np.array_equal(host_f64(Y), bf16_bits_to_f64(_bf16_exact(mxfp4.product(_f64(xb), w)[0])))
    dX = sl.sl_linear_dgrad_mxfp4w(dev_bf16(yb), *_dev(w))
    assert np.array_equal(host_f64(dX), bf16_bits_to_f64(_bf16_exact(mxfp4.product(_f64(yb), mxfp4.dequantize(*w).T)[0])))


@pytest.mark.parametrize("T", [1, 5, 16, 40, 130, 600])
def test_mxfp4w_non_finite(T):
    """An infinity or NaN in a token reaches that token alone; a NaN block its output column alone."""
    say(f"case mxfp4w non-finite T={T}")
    w = _exact_operand(72, 544, 1)
    x = np.ones((T, 544), np.float32)
    x[T - 1, 543] = np.nan
    w[1][5, 16] = 255
    Y = host_f64(sl.sl_linear_fwd_mxfp4w(dev_bf16(synth.f32_to_bf16_bits(x)), *_dev(w)))
    assert np.isnan(Y[T - 1]).all() and np.isnan(Y[:, 5]).all()
    Y[T - 1], Y[:, 5] = 0, 0
    assert np.isfinite(Y).all()
    w[1][5, 16] = 128
    dy = np.ones((T, 72), np.float32)
    dy[0, 3] = np.inf
    w[0][3, 0], w[0][3, 1] = 0x22, 0xAA                            # +1 +1 -1 -1: infinities of known sign
    dX = host_f64(sl.sl_linear_dgrad_mxfp4w(dev_bf16(synth.f32_to_bf16_bits(dy)), *_dev(w)))
    assert (dX[0, :2] == np.inf).all() and (dX[0, 2:4] == -np.inf).all()
    assert np.isfinite(dX[1:]).all()


@pytest.mark.parametrize("cfg,M,N,K", [(0, 1, 8, 32), (0, 4104, 4104, 544), (0, 264, 520, 8224), (1, 3, 1000, 96), (1, 2824, 2952, 288),
                                       (1, 136, 72, 16416), (2, 1, 8, 32), (2, 264, 264, 800), (2, 2056, 2184, 288),
                                       (2, 2056, 2184, 1056), (2, 136, 72, 16416), (2, 2824, 2952, 1312)])
def test_forced_tiles(cfg, M, N, K):
    """Either tile size on any shape: more tiles than workgroups, odd numbers of stages, split sums."""
    say(f"case mxfp4 tiles {cfg} {M}x{N}x{K}")
    a, b = _exact_operand(M, K, M), _exact_operand(N, K, N + 1)
    ref = mxfp4.product(a, b)[0]
    a, b = _dev(a), _dev(b)
    with sl.tuning(f8=cfg):
        Y = sl.sl_linear_fwd_mxfp4(*a, *b)
        assert np.array_equal(host_f64(Y), bf16_bits_to_f64(_bf16_exact(ref)))
        g = torch.ones(((M + 7) // 8 * 8, N), device="cuda")
        pad = [torch.zeros((g.shape[0], t.shape[1]), dtype=torch.uint8, device="cuda") for t in a]
        for p, t in zip(pad, a):
            p[:M] = t
        sl.sl_linear_wgrad_accum_mxfp4(*pad, *b, g)
    assert np.array_equal(host_f64(g)[:M], ref + 1) and (g[M:] == 1).all()


def test_results_repeat():
    """The same call gives the same bits, with poisoned outputs and workspaces in between."""
    say("case mxfp4 repeat")
    for M, N, K in ((1, 512, 2048), (200, 264, 1056), (700, 1000, 2080)):
        a, b = _dev(_operand(M, K, 1)), _dev(_operand(N, K, 2))
        X = torch.randn((M, K), device="cuda").bfloat16()
        first = sl.sl_linear_fwd_mxfp4(*a, *b), sl.sl_linear_fwd_mxfp4w(X, *b)
        for _ in range(3):
            Y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device="cuda")
            assert torch.equal(sl.sl_linear_fwd_mxfp4(*a, *b, Y), first[0])
            Y.fill_(float("nan"))
            assert torch.equal(sl.sl_linear_fwd_mxfp4w(X, *b, Y), first[1])
    a, b = _dev(_operand(264, 4096, 1)), _dev(_operand(256, 4096, 2))
    need = max(sl.sl_mxfp4_wgrad_workspace_bytes(4096, 256, 264), 16)
    got = []
    for fill in (0, 255, 127):
        g = torch.zeros((264, 256), device="cuda")
        sl.sl_linear_wgrad_accum_mxfp4(*a, *b, g, workspace=torch.full((need,), fill, dtype=torch.uint8, device="cuda"))
        got.append(g)
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_refusals_in_python():
    say("case mxfp4 refusals")
    u = lambda *s: torch.zeros(s, dtype=torch.uint8, device="cuda")  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16, device="cuda")  # noqa: E731
    bad = [
        (ValueError, lambda: sl.sl_mxfp4_quantize(bf(32, 36))),
        (ValueError, lambda: sl.sl_mxfp4_quantize(bf(4, 32, 32))),
        (TypeError, lambda: sl.sl_mxfp4_quantize(torch.zeros((32, 32), device="cuda"))),
        (ValueError, lambda: sl.sl_mxfp4_quantize(bf(64, 64).t()[:, :32])),
        (ValueError, lambda: sl.sl_mxfp4_quantize(bf(32, 32), seed=torch.zeros(2, dtype=torch.int64, device="cuda"))),
        (ValueError, lambda: sl.sl_mxfp4_quantize(bf(32, 32), seed=torch.zeros(1, dtype=torch.int64))),
        (TypeError, lambda: sl.sl_mxfp4_quantize(bf(32, 32), seed=torch.zeros(1, device="cuda"))),
        (ValueError, lambda: sl.sl_mxfp4_dequantize(u(4, 24), u(4, 1))),
        (ValueError, lambda: sl.sl_linear_fwd_mxfp4(u(4, 32), u(4, 2), u(8, 16), u(8, 1))),
        (ValueError, lambda: sl.sl_linear_fwd_mxfp4(u(4, 32), u(4, 1), u(8, 32), u(8, 2))),
        (ValueError, lambda: sl.sl_linear_dgrad_mxfp4(u(4, 32), u(4, 2), u(8, 16), u(8, 1))),
        (ValueError, lambda: sl.sl_linear_wgrad_accum_mxfp4(u(8, 32), u(8, 2), u(16, 32), u(16, 2), torch.zeros((16, 8), device="cuda"))),
        (TypeError, lambda: sl.sl_linear_wgrad_accum_mxfp4(u(8, 32), u(8, 2), u(16, 32), u(16, 2), bf(8, 16))),
        (ValueError, lambda: sl.sl_linear_fwd_mxfp4w(bf(4, 32), u(8, 32), u(8, 2))),
        (TypeError, lambda: sl.sl_linear_fwd_mxfp4w(torch.zeros((4, 64), device="cuda", dtype=torch.float16), u(8, 32), u(8, 2))),
        (sl._lib.SLError, lambda: sl.sl_linear_fwd_mxfp4w(bf(4, 64), u(12, 32), u(12, 2))),        # out % 8
        (ValueError, lambda: sl.sl_linear_dgrad_mxfp4w(bf(4, 16), u(8, 32), u(8, 2))),
    ]
    for err, call in bad:
        with pytest.raises(err):
            call()


# ---- the operators together -----------------------------------------------------------------------

def _layer(T, n_in, n_out, seed):
    xb, wb, yb = _bits(T, n_in, seed), _bits(n_out, n_in, seed + 1), _bits(T, n_out, seed + 2)
    w = torch.nn.Parameter(dev_bf16(wb))
    w.main_grad = torch.zeros((n_out, n_in), device="cuda")
    return xb, wb, yb, w


def _step_ref(xb, wb, yb, key):
    x, w, y = _f64(xb), _f64(wb), _f64(yb)
    r = None if key is None else mxfp4.draws(*y.shape, key)
    Y = mxfp4.product(mxfp4.quantize(x), mxfp4.quantize(w))
    dX = mxfp4.product(mxfp4.quantize(y, r), mxfp4.quantize(w.T))
    G = mxfp4.product(mxfp4.quantize(y.T, None if r is None else r.T), mxfp4.quantize(x.T))
    return Y, dX, G


@pytest.mark.parametrize("T,n_in,n_out", [(1, 32, 8), (37, 72, 40), (128, 256, 512), (300, 1040, 776)])
@pytest.mark.parametrize("seed", [None, 21])
def test_training_step(T, n_in, n_out, seed):
    """Cast, forward, input gradient and accumulated weight gradient against the definition, two micro-batches."""
    say(f"case mxfp4 step T={T} in={n_in} out={n_out} seed={seed}")
    total, S_total = 0, 0
    xb, wb, yb, w = _layer(T, n_in, n_out, 50)
    wq = sl.sl_mxfp4_quantize(w.detach())
    for mb in range(2):
        xb, yb = _bits(T, n_in, 60 + mb), _bits(T, n_out, 70 + mb)
        x = dev_bf16(xb).requires_grad_()
        y = sl.linear_mxfp4_with_grad_accumulation(x, w, seed, weight_mxfp4=wq if mb else None)
        y.backward(dev_bf16(yb))
        (Y, SY), (dX, SX), (G, SG) = _step_ref(xb, wb, yb, seed)
        _close(y, Y, SY, n_in + 32)
        _close(x.grad, dX, SX, n_out + 32)
        total, S_total = total + G, S_total + SG
        _close(w.main_grad, total, S_total, (mb + 1) * (T + 49), bf16=False)
    assert w.grad is None and w.grad_added_to_main_grad


def test_training_step_is_the_gradient_of_its_products():
    """The product is linear in each operand: with operands that the cast leaves as they are (few bits, one size), the
    step's gradients are those of sum(Y dY), taken by central differences of the layer itself, whose values are exact."""
    say("case mxfp4 step differences")
    g = np.random.default_rng(3)
    T, n_in, n_out = 32, 64, 32
    grid = np.array([-6, -4, -3, -2, -1, 0, 1, 2, 3, 4, 6], np.float32)
    pick = lambda *s: grid[g.integers(0, grid.size, s)]  # noqa: E731
    x, wt, dy = pick(T, n_in), pick(n_out, n_in), pick(T, n_out)
    for m in (x, wt, dy):
        m[::32, :], m[:, ::32] = 6, 6                             # every block's largest value
    dev = lambda a: torch.from_numpy(a).bfloat16().cuda()  # noqa: E731
    w = torch.nn.Parameter(dev(wt))
    w.main_grad = torch.zeros((n_out, n_in), device="cuda")
    xd = dev(x).requires_grad_()
    sl.linear_mxfp4_with_grad_accumulation(xd, w).backward(dev(dy))
    # dY / dx_j by the central difference of the layer at x = 0 along entry j
    for t, j in ((0, 1), (5, 33), (31, 63)):
        up = np.zeros((1, n_in), np.float32)
        up[0, j] = 1
        Yp = host_f64(sl.linear_mxfp4_with_grad_accumulation(dev(up), w.detach(), weight_mxfp4=sl.sl_mxfp4_quantize(w.detach())))
        Ym = host_f64(sl.linear_mxfp4_with_grad_accumulation(dev(-up), w.detach(), weight_mxfp4=sl.sl_mxfp4_quantize(w.detach())))
        slope = (Yp - Ym)[0] / 2                                   # dY / dx_j
        want = float((slope * dy[t]).sum())
        assert host_f64(xd.grad)[t, j] == float(torch.tensor(want).bfloat16())
        assert host_f64(w.main_grad)[:, j].tolist() == (dy.astype(np.float64).T @ x[:, j].astype(np.float64)).tolist()


def test_training_step_partial_gradients():
    say("case mxfp4 step partial gradients")
    xb, wb, yb, w = _layer(64, 64, 32, 5)
    y = sl.linear_mxfp4_with_grad_accumulation(dev_bf16(xb), w)            # input needs none
    y.backward(dev_bf16(yb))
    assert w.main_grad.any()
    w.requires_grad_(False)
    before = w.main_grad.clone()
    x = dev_bf16(xb).requires_grad_()
    sl.linear_mxfp4_with_grad_accumulation(x, w).backward(dev_bf16(yb))       # a frozen weight
    assert x.grad.any() and torch.equal(before, w.main_grad)
    x3 = dev_bf16(xb).view(2, 32, 64).requires_grad_()                       # [s, b, h]
    y3 = sl.linear_mxfp4_with_grad_accumulation(x3, w)
    assert y3.shape == (2, 32, 32)
    y3.backward(dev_bf16(yb).view(2, 32, 32))
    assert torch.equal(x3.grad.view(64, 64), x.grad)
    with pytest.raises(ValueError, match="columnwise"):
        sl.linear_mxfp4_with_grad_accumulation(x, w, weight_mxfp4=sl.sl_mxfp4_quantize(w.detach(), cols=False))


def test_other_stream():
    """On a side stream, with the default stream busy, results are those of the default stream."""
    say("case mxfp4 side stream")
    a, b = _dev(_operand(300, 4096, 1)), _dev(_operand(264, 4096, 2))
    want = torch.zeros((300 + 4, 264), device="cuda")
    qa = _dev(_operand(304, 4096, 1))
    sl.sl_linear_wgrad_accum_mxfp4(*qa, *b, want)
    Y = sl.sl_linear_fwd_mxfp4(*a, *b)
    torch.cuda.synchronize()
    got, outs = [torch.zeros_like(want) for _ in range(2)], []
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for s, g in zip(streams, got):
        with torch.cuda.stream(s):
            sl.sl_linear_wgrad_accum_mxfp4(*qa, *b, g)
            outs.append(sl.sl_linear_fwd_mxfp4(*a, *b))
    torch.cuda.synchronize()
    for g, o in zip(got, outs):
        assert torch.equal(g, want) and torch.equal(o, Y)


def test_graph_replay():
    """The training step and a token's forward, captured: replays follow their inputs and the seed tensor, and equal
    the eager results, with eager work on the same kernels in between."""
    say("case mxfp4 graph replay")
    T, n_in, n_out = 256, 1056, 264
    _, wb, _, w = _layer(T, n_in, n_out, 5)
    x, dy = torch.zeros((T, n_in), dtype=torch.bfloat16, device="cuda"), torch.zeros((T, n_out), dtype=torch.bfloat16, device="cuda")
    seed = torch.zeros(1, dtype=torch.int64, device="cuda")
    grad = w.main_grad

    def step(main_grad, seed):
        xr, xrs, xc, xcs = sl.sl_mxfp4_quantize(x)
        wr, wrs, wc, wcs = sl.sl_mxfp4_quantize(w.detach())
        dr, drs, dc, dcs = sl.sl_mxfp4_quantize(dy, seed=seed)
        y = sl.sl_linear_fwd_mxfp4(xr, xrs, wr, wrs)
        dx = sl.sl_linear_dgrad_mxfp4(dr, drs, wc, wcs)
        sl.sl_linear_wgrad_accum_mxfp4(dc, dcs, xc, xcs, main_grad)
        one = sl.sl_linear_fwd_mxfp4w(x[:1], wr, wrs)
        back = sl.sl_linear_dgrad_mxfp4w(dy, wr, wrs)
        return y, dx, one, back

    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        step(grad, seed)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = step(grad, seed)
    for k in range(3):
        x.copy_(dev_bf16(_bits(T, n_in, 100 + k)))
        dy.copy_(dev_bf16(_bits(T, n_out, 200 + k)))
        seed.fill_(k + 5)
        grad.zero_()
        graph.replay()
        torch.cuda.synchronize()
        got = [o.clone() for o in outs] + [grad.clone()]
        g = torch.zeros_like(grad)
        want = [*step(g, k + 5), g]
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b), k


def test_two_graphs_of_split_products():
    """Two captured graphs, each with split sums, replayed side by side on two streams: neither uses the other's planes."""
    say("case mxfp4 two graphs")
    cases = []
    for k in range(2):
        a, b, x = _dev(_operand(104, 8192, 10 + k)), _dev(_operand(72, 8192, 20 + k)), dev_bf16(_bits(100, 8192, k))
        dy, wt, g = dev_bf16(_bits(100, 4096, 5 + k)), _dev(_operand(4096, 96, 30 + k)), torch.zeros((104, 72), device="cuda")

        def run(a=a, b=b, x=x, dy=dy, wt=wt, g=g):
            g.zero_()
            sl.sl_linear_wgrad_accum_mxfp4(*a, *b, g)
            return (sl.sl_linear_fwd_mxfp4(*a, *b), sl.sl_linear_fwd_mxfp4w(x, *b), sl.sl_linear_dgrad_mxfp4w(dy, *wt), g)

        want = [t.clone() for t in run()]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outs = run()
        cases.append((graph, outs, want))
    assert sl.sl_mxfp4_fwd_workspace_bytes(104, 8192, 72) and sl.sl_mxfp4w_fwd_workspace_bytes(100, 8192, 72)
    assert sl.sl_mxfp4w_dgrad_workspace_bytes(100, 96, 4096) and sl.sl_mxfp4_wgrad_workspace_bytes(8192, 72, 104)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(3):
        torch.cuda.synchronize()
        for (graph, outs, _want), s in zip(cases, streams):
            with torch.cuda.stream(s):
                for o in outs[:3]:
                    o.fill_(float("nan"))
                graph.replay()
        torch.cuda.synchronize()
        for _graph, outs, want in cases:
            for o, w in zip(outs, want):
                assert torch.equal(o, w)


@pytest.mark.parametrize("T", [1, 5, 70])
def test_many_features(T):
    """More features than the chip has room for tiles at a time, as of a vocabulary, by few tokens."""
    say(f"case mxfp4 vocabulary T={T}")
    n_in, n_out = 64, 131080
    w, xb = _exact_operand(n_out, n_in, 1), _bits(T, n_in, T)
    _close(sl.sl_linear_fwd_mxfp4w(dev_bf16(xb), *_dev(w)), *mxfp4.product(_f64(xb), w), n_in)
    a = _exact_operand(T, n_in, 2)
    assert np.array_equal(host_f64(sl.sl_linear_fwd_mxfp4(*_dev(a), *_dev(w))), bf16_bits_to_f64(_bf16_exact(mxfp4.product(a, w)[0])))


def _device_operand(rows, k, seed):
    """Random codes under scale 1, made on the device."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randint(0, 256, (rows, k // 2), dtype=torch.uint8, device="cuda", generator=g),
            torch.full((rows, k // 32), 127, dtype=torch.uint8, device="cuda"))


def test_products_large_index():
    """Results, weights and gradients past 2^31 elements: their ends are those of the same product of the last rows alone.
    Sums of multiples of 1/4 below 2^22 are exact, so the kernels that the sizes choose agree to the bit."""
    say("case mxfp4 large products")
    a, b = _device_operand(300008, 64, 1), _device_operand(7304, 64, 2)
    Y = sl.sl_linear_fwd_mxfp4(*a, *b)
    assert Y.numel() > 2**31
    assert torch.equal(Y[-50:], sl.sl_linear_fwd_mxfp4(a[0][-50:], a[1][-50:], *b))
    assert torch.equal(Y[:50], sl.sl_linear_fwd_mxfp4(a[0][:50], a[1][:50], *b))
    del Y
    X = torch.randint(-1, 2, (300008, 64), device="cuda").bfloat16()
    Y = sl.sl_linear_fwd_mxfp4w(X, *b)
    assert torch.equal(Y[-50:], sl.sl_linear_fwd_mxfp4w(X[-50:], *b))
    del Y, X
    a, b = _device_operand(32776, 32, 3), _device_operand(65544, 32, 4)
    g = torch.ones((32776, 65544), device="cuda")
    sl.sl_linear_wgrad_accum_mxfp4(*a, *b, g)
    end = torch.ones((264, 65544), device="cuda")
    sl.sl_linear_wgrad_accum_mxfp4(a[0][-264:], a[1][-264:], *b, end)
    assert torch.equal(g[-264:], end)
    del g, end
    n_out, n_in = 131080, 65568                                    # more than 2^32 bytes of codes
    w = _device_operand(n_out, n_in, 5)
    assert w[0].numel() > 2**32
    last = w[0][-256:], w[1][-256:]
    for T in (2, 70):
        X = torch.randint(-1, 2, (T, n_in), device="cuda").bfloat16()
        assert torch.equal(sl.sl_linear_fwd_mxfp4w(X, *w)[:, -256:], sl.sl_linear_fwd_mxfp4w(X, *last)), T
        a = _device_operand(T, n_in, 6)
        assert torch.equal(sl.sl_linear_fwd_mxfp4(*a, *w)[:, -256:], sl.sl_linear_fwd_mxfp4(*a, *last)), T
        dY = torch.randint(-1, 2, (T, n_out), device="cuda").bfloat16()
        cols = w[0][:, -32:].contiguous(), w[1][:, -2:].contiguous()
        assert torch.equal(sl.sl_linear_dgrad_mxfp4w(dY, *w)[:, -64:], sl.sl_linear_dgrad_mxfp4w(dY, *cols)), T


def test_second_derivatives_are_refused():
    say("case mxfp4 second derivative")
    xb, wb, yb, w = _layer(32, 64, 32, 5)
    x = dev_bf16(xb).requires_grad_()
    y = sl.linear_mxfp4_with_grad_accumulation(x, w)
    (dx,) = torch.autograd.grad(y, x, dev_bf16(yb).requires_grad_(), create_graph=True)
    with pytest.raises(RuntimeError, match="once_differentiable"):
        dx.sum().backward()


def test_backward_capture():
    """The autograd function captured as a whole, on leaves of its own."""
    say("case mxfp4 autograd capture")
    T, n_in, n_out = 64, 96, 72
    xb, wb, yb, w = _layer(T, n_in, n_out, 9)
    dy = dev_bf16(yb)
    x = dev_bf16(xb).requires_grad_()

    def step():
        y = sl.linear_mxfp4_with_grad_accumulation(x, w, 3)
        return y, torch.autograd.grad(y, x, dy)[0]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y, dx = step()
        y, dx = y.detach().clone(), dx.clone()
    torch.cuda.synchronize()
    once = w.main_grad.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy, gdx = step()
    for _ in range(3):
        w.main_grad.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(gy, y) and torch.equal(gdx, dx) and torch.equal(w.main_grad, once)
