"""GPU parity of the microscaled 4-bit matrices against the fp64 oracle.

Codes, scales and read-back values are bit-exact.  A product's terms are exact in
binary32 and its sum has K terms: with operands from a grid on which every
partial sum fits 24 bits the result is exact in any order, and for other
operands it is off by at most K 2^-23 times the sum of the terms' magnitudes
(each of K additions off by 2^-24 of a partial sum that is at most that, twice
over for an addition that truncates), plus the output type's half step."""
import numpy as np
import pytest

from oracle import mx4 as ref
from tests.gpu_util import dev, sync

pytestmark = pytest.mark.gpu

HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8, "float16": 2.0 ** -11}
DTYPES = sorted(HALF)


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


def _t(name):
    import torch
    return getattr(torch, name)


def _f64(t):
    import torch
    return t.detach().to(torch.float64).cpu().numpy()


def _float(a, dtype, lead=0, pad=0):
    """Device copy of a [r, c] array as dtype, `lead` elements into its buffer
    and with rows `pad` elements apart; NaN around it."""
    import torch
    r, c = a.shape
    buf = torch.full((lead + r * (c + pad),), float("nan"), dtype=_t(dtype), device=dev())
    v = buf[lead:].view(r, c + pad)[:, :c]
    v.copy_(torch.from_numpy(np.ascontiguousarray(a)).to(dev()).to(_t(dtype)))
    return v


def _wide(seed, r, c):
    g = np.random.default_rng(seed)
    x = g.standard_normal((r, c)) * np.exp2(g.integers(-12, 12, (r, c)) * (g.random((r, c)) < 0.2))
    x[g.random((r, c)) < 0.05] = 0.0
    return x


SIZES = [(1, 1), (1, 31), (3, 32), (2, 33), (5, 64), (17, 100), (64, 128), (70, 777), (257, 8), (1, 4097), (1000, 1),
         (20011, 1), (5000, 2), (16500, 3), (700, 5), (9000, 17), (333, 63), (40, 66)]


@pytest.mark.parametrize("lead,pad", [(0, 0), (1, 0), (0, 3), (8, 8)])
@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", SIZES)
def test_quantize_both_axes_bit_exact(m, size, dtype, lead, pad):
    import torch
    r, c = size
    x = _float(_wide(r * 1000 + c, r, c), dtype, lead, pad)
    for axis in (1, 0):
        q = m.mx4_empty(r, c, axis)
        q.codes.fill_(0xA5)
        q.scales.fill_(0xA5)
        m.mx4_quantize(x, q, axis=axis)
        sync()
        h = _f64(x) if axis == 1 else _f64(x).T
        codes, scales = ref.quantize(h)
        assert np.array_equal(q.scales.cpu().numpy(), scales.astype(np.uint8)), (axis, "scales")
        assert np.array_equal(q.codes.cpu().numpy(), ref.pack(codes)), (axis, "codes")
        for od in DTYPES:
            want = ref.values(codes, scales, h.shape[1])
            out = _float(np.zeros(h.shape), od, lead, pad)
            m.mx4_dequantize(q, out)
            sync()
            assert torch.equal(out, torch.from_numpy(want).to(dev()).to(_t(od))), (axis, od)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("size", [(1, 1), (1023, 1), (1024, 2), (2050, 3), (5001, 7), (3000, 8), (4099, 9), (1500, 15),
                                  (9000, 16), (70001, 1)])
def test_quantize_narrow_matrices_along_their_rows(m, size, dtype):
    """One block a row, with and without a gap between rows, non-finite rows
    among them; and of one column the column too."""
    import torch
    r, c = size
    x = _float(_wide(r + c, r, c), dtype)
    x[r // 2, c - 1] = float("nan")
    x[r // 3, 0] = float("-inf")
    gap = torch.full((r, c + 3), 7.0, dtype=x.dtype, device=dev())
    gap[:, 1:c + 1] = x
    for y, axis in ((x, 1), (gap[:, 1:c + 1], 1)) + (((x, 0), (gap[:, 1:2], 0)) if c == 1 else ()):
        q = m.mx4_empty(r, c, axis)
        q.codes.fill_(0xA5)
        q.scales.fill_(0xA5)
        m.mx4_quantize(y, q, axis=axis)
        sync()
        codes, scales = ref.quantize(_f64(x) if axis else _f64(x).T)
        assert np.array_equal(q.scales.cpu().numpy(), scales.astype(np.uint8))
        assert np.array_equal(q.codes.cpu().numpy(), ref.pack(codes))


@pytest.mark.parametrize("size", [(140_000, 20), (270_003, 9), (1_100_007, 3), (4_200_005, 1)])
def test_quantize_narrow_matrices_along_their_columns(m, size):
    """Few columns and many rows, where a wave takes several blocks of one."""
    r, c = size
    x = _float(_wide(r, r, c), "bfloat16", pad=2)
    q = m.mx4_empty(r, c, 0)
    q.codes.fill_(0xA5)
    q.scales.fill_(0xA5)
    m.mx4_quantize(x, q, axis=0)
    sync()
    codes, scales = ref.quantize(_f64(x).T)
    assert np.array_equal(q.scales.cpu().numpy(), scales.astype(np.uint8))
    assert np.array_equal(q.codes.cpu().numpy(), ref.pack(codes))


def test_quantize_every_rounding_border(m):
    """Each block: the largest magnitude sets the scale to 1 (or a power of
    two), the others sit on and next to the borders between codes."""
    borders = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, 7.0]
    ys = []
    for b in borders:
        f = np.float32(b)
        ys += [f, np.nextafter(f, np.float32(0)), np.nextafter(f, np.float32(9))]
    rows = []
    for e in (0, -100, 100, -125):
        for i in range(0, len(ys), 31):
            blk = np.zeros(32, np.float32)
            part = np.array(ys[i:i + 31], np.float32)
            blk[1:1 + len(part)] = part
            blk[0] = 4.0
            blk = np.concatenate([blk, -blk])
            rows.append((blk.astype(np.float64) * 2.0 ** e).astype(np.float32))
    x = _float(np.array(rows, np.float64), "float32")
    q = m.mx4_empty(*x.shape)
    m.mx4_quantize(x, q)
    sync()
    codes, scales = ref.quantize(_f64(x))
    assert np.array_equal(q.scales.cpu().numpy(), scales) and np.array_equal(q.codes.cpu().numpy(), ref.pack(codes))


def test_quantize_extremes(m):
    """Largest and subnormal magnitudes, zeros, negative zeros, NaN and
    infinities at each place of a block."""
    import torch
    rows = [[3.4e38] * 32, [1e-45] * 32, [1e-38, 1e-40, 1e-45] + [0.0] * 29, [0.0] * 32, [-0.0] * 32,
            [1.1754944e-38] + [0.0] * 31, [2.0 ** -125, 2.0 ** -127, 1e-42] + [0.0] * 29,
            [2.0 ** -124, 2.0 ** -127] + [0.0] * 30, [-3.4e38, 3e38, 1.0] + [0.0] * 29]
    for bad in (np.nan, np.inf, -np.inf):
        for at in (0, 7, 8, 31):
            v = [1.0] * 32
            v[at] = bad
            rows.append(v)
    a = np.array(rows, np.float64).astype(np.float32).astype(np.float64)
    a = np.concatenate([a, np.ones_like(a)], 1)  # a clean block beside each
    for axis in (1, 0):
        x = _float(a if axis == 1 else a.T, "float32")
        q = m.mx4_empty(*x.shape, axis)
        m.mx4_quantize(x, q, axis=axis)
        v = torch.zeros(a.shape, device=dev())
        m.mx4_dequantize(q, v)
        sync()
        codes, scales = ref.quantize(a)
        assert np.array_equal(q.scales.cpu().numpy(), scales) and np.array_equal(q.codes.cpu().numpy(), ref.pack(codes))
        assert np.array_equal(_f64(v), ref.values(codes, scales, 64), equal_nan=True)


# ----------------------------------------------------------------- products
def _grid(g, rows, cols):
    """Values whose quantisation is exact and whose products' sums are:
    multiples of 0.5 up to 6 with a 4 or a 6 in every block of scale 1, half of
    the blocks at scale 1/2."""
    x = g.choice(ref.LEVELS, (rows, cols)) * g.choice([-1.0, 1.0], (rows, cols))
    x[:, ::32] = g.choice([4.0, 6.0], x[:, ::32].shape)
    half = np.repeat(g.random((rows, -(-cols // 32))) < 0.5, 32, 1)[:, :cols]
    return np.where(half, x * 0.5, x)


def _operand(m, a):
    x = _float(a, "float32")
    q = m.mx4_empty(*a.shape)
    m.mx4_quantize(x, q)
    return q


PRODUCTS = [(1, 1, 1), (1, 16, 32), (2, 3, 33), (1, 512, 256), (1, 4096, 1024), (5, 100, 64), (16, 129, 96), (17, 16, 128),
            (33, 257, 160), (64, 64, 512), (127, 130, 1000), (129, 128, 31), (200, 333, 777), (256, 512, 2048),
            (300, 17, 4100), (1024, 1, 200), (1000, 513, 256), (515, 777, 130), (16, 8, 8192), (40, 40, 6500),
            (1030, 1031, 400), (1500, 1411, 600), (500, 1040, 700), (20, 3000, 2000), (32, 500, 288), (129, 700, 4000),
            (16, 24, 9000), (500, 1040, 900), (1030, 1031, 300),
            (1700, 1300, 70), (1601, 1333, 256), (2001, 1500, 300), (600, 40, 513),
            (40, 40, 50_000), (300, 330, 50_001), (700, 760, 9000), (1000, 1000, 8200), (20, 4000, 400), (513, 500, 600)]


@pytest.mark.parametrize("mnk", PRODUCTS)
def test_product_exact_on_the_grid(m, mnk):
    """Every form of the product on operands for which any order of the sum
    is exact: equality, for each type, with and without bias and relu, rows
    of the output further apart than N, nothing written between them."""
    import torch
    M, N, K = mnk
    g = np.random.default_rng(M + 10 * N + 100 * K)
    a, b = _grid(g, M, K), _grid(g, N, K)
    aq, bq = _operand(m, a), _operand(m, b)
    bias = g.integers(-40, 40, N) * 0.25
    tb = torch.from_numpy(bias.astype(np.float32)).to(dev())
    y = a @ b.T
    ws = m.mx4_matmul_workspace(M, N, K)
    for od in DTYPES:
        for use_bias, relu, pad in ((False, False, 0), (True, True, 5), (True, False, 4)):
            want = y + (bias if use_bias else 0.0)
            want = np.maximum(want, 0.0) if relu else want
            want = torch.from_numpy(want).float().to(_t(od)).to(dev())  # exact in f32, then one rounding
            buf = torch.full((M, N + pad), 77.0, dtype=_t(od), device=dev())
            ws.fill_(0xFF)
            m.mx4_matmul(aq, bq, buf[:, :N], ws, bias=tb if use_bias else None, relu=relu)
            sync()
            assert torch.equal(buf[:, :N], want), ("matmul", od, use_bias, relu)
            assert torch.all(buf[:, N:] == 77.0)
            for xd in DTYPES:
                x = _float(a, xd, lead=3, pad=1) if pad == 5 else _float(a, xd)
                buf.fill_(77.0)
                ws.fill_(0xFF)
                m.mx4_linear(x, bq, buf[:, :N], ws, bias=tb if use_bias else None, relu=relu)
                sync()
                assert torch.equal(buf[:, :N], want), ("linear", xd, od, use_bias, relu)
                assert torch.all(buf[:, N:] == 77.0)


@pytest.mark.parametrize("mnk", [(2900, 2950, 1056), (2817, 3000, 1500), (8200, 1030, 1024), (1000, 9000, 2100),
                                 (33000, 250, 1024), (4096, 4096, 4096), (8192, 512, 256), (9001, 77, 33), (12345, 513, 130),
                                 (16384, 512, 256), (17001, 77, 33), (16399, 513, 130), (16384, 16, 1000),
                                 (65536, 128, 128), (8200, 450, 1000), (4000, 3300, 260), (1409, 1500, 3000), (700, 2500, 1111)])
def test_large_products_exact_on_the_grid(m, mnk):
    """Products of many tiles, ragged in each size: equality with the oracle
    at the matrix's corners, edges and a sample of rows, and of all rows with a
    second product (sums of each row against a vector of ones)."""
    import torch
    M, N, K = mnk
    g = np.random.default_rng(M + N + K)
    a, b = _grid(g, M, K), _grid(g, N, K)
    aq, bq = _operand(m, a), _operand(m, b)
    bias = g.integers(-40, 40, N) * 0.25
    tb = torch.from_numpy(bias.astype(np.float32)).to(dev())
    ws = m.mx4_matmul_workspace(M, N, K)
    rows = np.unique(np.concatenate([[0, 1, 127, 128, 255, 256, M - 257, M - 2, M - 1], g.integers(0, M, 200)]))
    want = torch.from_numpy(a[rows] @ b.T).to(dev())
    total = torch.from_numpy(a @ b.sum(0)).to(dev())
    tr = torch.from_numpy(rows).to(dev())
    for od, use_bias, relu, pad in (("float32", False, False, 0), ("bfloat16", True, True, 4), ("float16", False, True, 7),
                                    ("float32", True, False, 1)):
        buf = torch.full((M, N + pad), 77.0, dtype=_t(od), device=dev())
        ws.fill_(0xFF)
        m.mx4_matmul(aq, bq, buf[:, :N], ws, bias=tb if use_bias else None, relu=relu)
        w = want + (tb.double() if use_bias else 0.0)
        w = w.clamp(min=0) if relu else w
        sync()
        assert torch.equal(buf[tr, :N], w.float().to(_t(od))), (od, use_bias, relu)
        assert torch.all(buf[:, N:] == 77.0)
        if od == "float32" and not use_bias:
            assert torch.equal(buf[:, :N].double().sum(1), total)
        x = _float(a, "bfloat16", lead=1, pad=1)
        other = torch.full_like(buf, 77.0)
        ws.fill_(0xFF)
        m.mx4_linear(x, bq, other[:, :N], ws, bias=tb if use_bias else None, relu=relu)
        sync()
        assert torch.equal(other, buf)


@pytest.mark.parametrize("mnk", [(3, 50, 100), (17, 40, 300), (70, 300, 200), (257, 900, 700), (1500, 1411, 600),
                                 (2900, 2950, 300), (9000, 60, 100)])
def test_rows_behind_the_last_stay_as_they_were(m, mnk):
    """Operands and outputs as the first rows of larger buffers: NaN behind the
    operands' last rows, and nothing written behind the output's."""
    import torch
    M, N, K = mnk
    g = np.random.default_rng(M * N)
    a, b = _grid(g, M, K), _grid(g, N, K)
    want = torch.from_numpy(a @ b.T).float().to(dev())
    kb = -(-K // 32)

    def padded(x, rows):
        codes = torch.full((rows + 40, kb * 16), 0x77, dtype=torch.uint8, device=dev())
        scales = torch.full((rows + 40, kb), 255, dtype=torch.uint8, device=dev())
        q = m.Mx4(codes[:rows], scales[:rows], rows, K)
        m.mx4_quantize(_float(x, "float32"), q)
        sync()
        assert torch.all(codes[rows:] == 0x77) and torch.all(scales[rows:] == 255)
        return q

    aq, bq = padded(a, M), padded(b, N)
    ws = m.mx4_matmul_workspace(M, N, K)
    guard = torch.full((ws.numel() + 256,), 0x5A, dtype=torch.uint8, device=dev())
    ws = guard[:ws.numel()]
    for x in (None, _float(np.concatenate([a, np.full((40, K), np.nan)]), "bfloat16")[:M]):
        buf = torch.full((M + 40, N), 77.0, device=dev())
        if x is None:
            m.mx4_matmul(aq, bq, buf[:M], ws)
        else:
            m.mx4_linear(x, bq, buf[:M], ws)
        sync()
        assert torch.equal(buf[:M], want)
        assert torch.all(buf[M:] == 77.0)
        assert torch.all(guard[ws.numel():] == 0x5A)
    back = torch.full((M + 3, K), 77.0, device=dev())
    m.mx4_dequantize(aq, back[:M])
    sync()
    assert torch.all(back[M:] == 77.0) and np.array_equal(_f64(back[:M]), a)


def test_products_on_several_streams_at_once(m):
    import torch
    g = np.random.default_rng(5)
    streams = [torch.cuda.Stream() for _ in range(4)]
    jobs = []
    for M, N, K in ((1, 500, 900), (200, 333, 777), (3000, 2500, 1100), (9000, 100, 200)):
        a, b = _grid(g, M, K), _grid(g, N, K)
        jobs.append((_float(a, "bfloat16"), _operand(m, b), torch.zeros((M, N), device=dev()),
                     m.mx4_matmul_workspace(M, N, K), torch.from_numpy(a @ b.T).float().to(dev())))
    sync()
    for rep in range(4):
        for x, b, y, ws, _ in jobs:
            y.zero_()
        sync()
        for _ in range(3):
            for st, (x, b, y, ws, _) in zip(streams, jobs):
                m.mx4_linear(x, b, y, ws, stream=st)
        sync()
        for x, b, y, ws, want in jobs:
            assert torch.equal(y, want)


@pytest.mark.parametrize("od", DTYPES)
@pytest.mark.parametrize("mnk", [(1, 1000, 1000), (9, 300, 2000), (200, 130, 555), (600, 512, 256)])
def test_product_of_wide_ranging_values(m, mnk, od):
    import torch
    M, N, K = mnk
    a, b = _wide(M + K, M, K), _wide(N + K, N, K)
    aq, bq = _operand(m, a), _operand(m, b)
    av = ref.round_trip(a.astype(np.float32).astype(np.float64))
    bv = ref.round_trip(b.astype(np.float32).astype(np.float64))
    scale = 2.0 ** -8 if od == "float16" else 1.0  # keeps binary16 results in range
    av = av * scale
    aq2 = _operand(m, a * scale)
    out = torch.zeros((M, N), dtype=_t(od), device=dev())
    m.mx4_matmul(aq2 if od == "float16" else aq, bq, out, m.mx4_matmul_workspace(M, N, K))
    sync()
    want, mag = av @ bv.T, np.abs(av) @ np.abs(bv).T
    tiny = 2.0 ** -25 if od == "float16" else 0.0
    got, slack = _f64(out), K * 2.0 ** -23 * mag
    # binary16 ends at 65504 = 2^16 - 2^5; its next step would be 2^16, and what
    # lies at or above the middle, 65520, rounds to infinity of its sign
    top = 65520.0 if od == "float16" else np.inf
    over = np.isinf(got)
    assert np.all(np.abs(want[over]) + slack[over] >= top) and np.all(np.sign(want[over]) == np.sign(got[over]))
    assert np.all(over[np.abs(want) - slack >= top])
    err = np.abs(np.where(over, 0.0, got - want))
    assert np.all(err <= slack + HALF[od] * 1.01 * np.abs(want) + tiny), np.max(err / (mag + 1e-300))
    # the sum itself is far inside that bound; its error is a few roundings
    if od == "float32":
        assert np.median(err / (mag + 1e-300)) <= 2.0 ** -23


def test_linear_equals_quantize_then_matmul(m):
    import torch
    for M, N, K in ((1, 300, 500), (7, 512, 256), (16, 64, 33), (130, 200, 700), (1500, 256, 256)):
        x = _float(_wide(M, M, K), "bfloat16", lead=1, pad=3)
        bq = _operand(m, _wide(N, N, K))
        aq = m.mx4_empty(M, K)
        m.mx4_quantize(x, aq)
        ws = m.mx4_matmul_workspace(M, N, K)
        y1, y2 = torch.zeros((M, N), device=dev()), torch.ones((M, N), device=dev())
        m.mx4_matmul(aq, bq, y1, ws)
        m.mx4_linear(x, bq, y2, ws)
        sync()
        assert torch.equal(y1, y2), (M, N, K)


def test_non_finite_blocks_reach_their_outputs_only(m):
    import torch
    for M, N, K in ((5, 40, 100), (150, 200, 300), (1, 64, 2048)):
        g = np.random.default_rng(K)
        a, b = _grid(g, M, K), _grid(g, N, K)
        a[M // 2, K - 1] = np.inf
        b[3, 0] = np.nan
        bq = _operand(m, b)
        x = _float(a, "float32")
        y = torch.zeros((M, N), device=dev())
        ws = m.mx4_matmul_workspace(M, N, K)
        m.mx4_linear(x, bq, y, ws, relu=True)
        sync()
        bad = torch.zeros((M, N), dtype=torch.bool, device=dev())
        bad[M // 2, :] = True
        bad[:, 3] = True
        assert torch.equal(torch.isnan(y), bad)


@pytest.mark.parametrize("mnk", [(12, 90, 700), (20, 40, 100), (60, 300, 100), (17, 300, 500), (300, 500, 1000), (700, 760, 1500),
                                 (700, 760, 8300), (1500, 1411, 300), (1500, 1411, 600), (1400, 1500, 2100), (4096, 3700, 520),
                                 (4096, 3700, 2100), (16400, 96, 100), (40, 50, 44_000)])
def test_non_finite_rows_of_every_kernel(m, mnk):
    """NaN and infinities in the first, a middle and the last block of rows at
    tile edges: their outputs and no others are NaN."""
    import torch
    M, N, K = mnk
    gen = torch.Generator(device=dev()).manual_seed(M + N + K)
    a = torch.randn((M, K), generator=gen, device=dev())
    b = torch.randn((N, K), generator=gen, device=dev())
    bad = torch.zeros((M, N), dtype=torch.bool, device=dev())
    for row, k, v in ((0, K - 1, "nan"), (M // 2, K // 2, "inf"), (M - 1, 0, "-inf")):
        a[row, k] = float(v)
        bad[row] = True
    for row, k, v in ((1, K - 1, "inf"), (N // 2, K // 3, "nan"), (N - 1, K - 1, "nan")):
        b[row, k] = float(v)
        bad[:, row] = True
    aq, bq = m.mx4_empty(M, K), m.mx4_empty(N, K)
    m.mx4_quantize(a, aq)
    m.mx4_quantize(b, bq)
    ws = m.mx4_matmul_workspace(M, N, K)
    y, z = torch.zeros((M, N), device=dev()), torch.zeros((M, N), device=dev())
    ws.fill_(0xFF)
    m.mx4_matmul(aq, bq, y, ws)
    ws.fill_(0xFF)
    m.mx4_linear(a, bq, z, ws, relu=True)
    sync()
    assert torch.equal(torch.isnan(y), bad) and torch.equal(torch.isnan(z), bad)
    assert bool(torch.isfinite(y[~bad]).all()) and bool((z[~bad] >= 0).all())


def test_products_captured_with_a_shared_workspace(m):
    import torch
    g = np.random.default_rng(0)
    jobs = []
    ws = m.mx4_matmul_workspace(300, 512, 6000)
    for M, N, K in ((1, 512, 6000), (300, 200, 700), (12, 64, 4096)):
        x = torch.zeros((M, K), device=dev())
        y = torch.zeros((M, N), device=dev())
        jobs.append((x, _operand(m, _grid(g, N, K)), y))
    graphs = []
    for x, b, y in jobs:
        m.mx4_linear(x, b, y, ws)
        sync()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            m.mx4_linear(x, b, y, ws)
        graphs.append(gr)
    for k in range(3):
        for x, _, _ in jobs:
            x.copy_(torch.randn(x.shape, device=dev()))
        for gr in graphs:
            gr.replay()
        sync()
        got = [y.clone() for _, _, y in jobs]
        for (x, b, y), r in zip(jobs, got):
            y.fill_(-1.0)
            m.mx4_linear(x, b, y, ws)
            sync()
            assert torch.equal(y, r)


def test_offsets_behind_32_bits(m):
    """Rows whose byte offsets pass 2^32 in x, codes and out."""
    import torch
    if torch.cuda.mem_get_info()[0] < 60 << 30:
        pytest.skip("needs 60 GB of free device memory")
    rows, cols = 70_000, 65_536  # x: 9.2 GB, codes 2.3 GB
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device=dev())
    g = torch.Generator(device=dev()).manual_seed(3)
    last = torch.randn((3, cols), generator=g, device=dev()).to(torch.bfloat16)
    x[-3:] = last
    q = m.mx4_empty(rows, cols)
    m.mx4_quantize(x, q)
    small = m.mx4_empty(3, cols)
    m.mx4_quantize(last, small)
    qt = m.mx4_empty(rows, cols, 0)
    m.mx4_quantize(x, qt, axis=0)
    back = torch.zeros((cols, rows), dtype=torch.bfloat16, device=dev())
    m.mx4_dequantize(qt, back)
    sync()
    assert torch.equal(q.codes[-3:], small.codes) and torch.equal(q.scales[-3:], small.scales)
    assert int(q.codes[:-3].count_nonzero()) == 0
    kb0 = rows // 32 * 32
    want = ref.round_trip(_f64(x[kb0:, -100:]).T)
    assert np.array_equal(_f64(back[-100:, kb0:]), want)
    b = m.mx4_empty(2, cols)
    m.mx4_quantize(torch.ones((2, cols), device=dev()), b)
    y = torch.full((rows, 2), 5.0, device=dev())
    m.mx4_matmul(q, b, y, m.mx4_matmul_workspace(rows, 2, cols))
    sync()
    assert int(y[:-3].count_nonzero()) == 0
    want = ref.round_trip(_f64(last)).sum(1)
    mag = np.abs(ref.round_trip(_f64(last))).sum(1)
    assert np.all(np.abs(_f64(y[-3:, 0]) - want) <= cols * 2.0 ** -23 * mag)


# ---------------------------------------------------- value network in 4 bits
def _trainer(m, S, H, H2, B, groups, params, dtype=0):
    cfg = m.make_config(S, H, B, num_groups=groups, compute_dtype=dtype, hidden2=H2)
    return m.IqlTrainer(cfg, np.concatenate(params).astype(np.float32))


NETS = [(16, 32, 0, 1), (128, 128, 0, 2), (42, 128, 0, 1), (256, 512, 0, 1), (100, 96, 160, 2), (1, 32, 0, 1),
        (65, 72, 40, 2), (700, 64, 0, 1), (1000, 1024, 512, 1), (1100, 96, 0, 2), (40, 1056, 64, 1)]


@pytest.mark.parametrize("B", [1, 67, 1000])
@pytest.mark.parametrize("net", NETS)
def test_value_network_exact_on_a_grid(m, net, B):
    """Parameters and states from a grid of which every sum is exact: V and the
    bootstrap target equal the oracle's."""
    import torch
    S, H, H2, G = net
    H2v = H2 or H
    g = np.random.default_rng(S + H)
    params = []
    for _ in range(G):
        # sparse small weights: hidden values stay small multiples of 1/4
        w1 = g.choice([0.0, 0.0, 0.0, 0.5, -0.5, 1.0], (H, S))
        w2 = g.choice([0.0] * 20 + [0.5, -0.5, 1.0], (H2v, H))
        params.append(np.concatenate([w1.ravel(), g.integers(-4, 5, H) * 0.5, w2.ravel(), g.integers(-4, 5, H2v) * 0.5,
                                      g.choice([0.0, 0.25, -0.25], H2v), [0.5]]))
    x = g.choice([0.0, 0.5, 1.0, -1.0, 2.0], (B, S))
    r = g.choice([1.0, -0.5], B).astype(np.float32)
    d = (g.random(B) < 0.3).astype(np.float32)
    tr = _trainer(m, S, H, H2, B, G, params)
    v = torch.zeros((G, B), device=dev())
    t = torch.zeros((G, B), device=dev())
    ws = tr.forward_values_mx4_workspace(B)
    for xd in ("float32", "bfloat16"):
        for pad in (0, 5):
            ws.fill_(0xFF)
            v.zero_()
            tr.forward_values_mx4(_float(x, xd, pad=pad), B, v, ws, rewards=torch.from_numpy(r).to(dev()),
                                  dones=torch.from_numpy(d).to(dev()), gamma=0.5, out_target=t)
            sync()
            for k in range(G):
                want = ref.value_network(params[k], S, H, H2v, x)
                assert np.array_equal(_f64(v[k]), want), (xd, pad, k)
                assert np.array_equal(_f64(t[k]), r + 0.5 * (1 - d) * want)
    tr.close()


@pytest.mark.parametrize("net", [(256, 512, 0, 1), (33, 288, 257, 2), (1024, 1024, 0, 1)])
def test_value_network_of_many_rows_exact_on_a_grid(m, net):
    """The same on a batch large enough for the 128-row workgroups, ragged."""
    import torch
    S, H, H2, G = net
    H2v, B = H2 or H, 32768 + 77
    g = np.random.default_rng(S + H + 1)
    params = []
    for _ in range(G):
        w1 = g.choice([0.0, 0.0, 0.0, 0.5, -0.5, 1.0], (H, S)) * (g.random((H, S)) < 32 / S)
        w2 = g.choice([0.0] * 20 + [0.5, -0.5, 1.0], (H2v, H))
        params.append(np.concatenate([w1.ravel(), g.integers(-4, 5, H) * 0.5, w2.ravel(), g.integers(-4, 5, H2v) * 0.5,
                                      g.choice([0.0, 0.25, -0.25], H2v), [0.5]]))
    x = g.choice([0.0, 0.5, 1.0, -1.0, 2.0], (B, S))
    tr = _trainer(m, S, H, H2, B, G, params, m.BF16)
    v = torch.zeros((G, B), device=dev())
    ws = tr.forward_values_mx4_workspace(B)
    ws.fill_(0xFF)
    tr.forward_values_mx4(_float(x, "bfloat16", pad=1), B, v, ws)
    sync()
    rows = np.unique(np.concatenate([np.arange(200), g.integers(0, B, 300), np.arange(B - 200, B)]))
    for k in range(G):
        want = ref.value_network(params[k], S, H, H2v, x[rows])
        assert np.array_equal(_f64(v[k])[rows], want)
    tr.close()


@pytest.mark.parametrize("net", [(128, 128, 0, 2), (256, 512, 0, 1), (100, 96, 160, 2), (1500, 200, 96, 1)])
def test_value_network_with_trained_like_weights(m, net):
    """Kaiming-sized weights: V within the oracle's bound for hidden sums
    that are off by K 2^-23 of their terms (a hidden value next to a border may
    then take the neighbouring code), and near the unquantised V."""
    import torch
    S, H, H2, G = net
    H2v = H2 or H
    B = 1500
    g = np.random.default_rng(7)
    params = [np.concatenate([g.uniform(-1, 1, H * S) / np.sqrt(S), g.uniform(-1, 1, H) / np.sqrt(S),
                              g.uniform(-1, 1, H2v * H) / np.sqrt(H), g.uniform(-1, 1, H2v) / np.sqrt(H),
                              g.uniform(-1, 1, H2v) / np.sqrt(H2v), [0.1]]).astype(np.float32) for _ in range(G)]
    x = g.standard_normal((B, S)).astype(np.float32)
    tr = _trainer(m, S, H, H2, B, G, params)
    v = torch.zeros((G, B), device=dev())
    tx = torch.from_numpy(x).to(dev())
    tr.forward_values_mx4(tx, B, v, tr.forward_values_mx4_workspace(B))
    full = torch.zeros((G, B), device=dev())
    tr.forward_values(tx, B, full)
    sync()
    for k in range(G):
        want, bound = ref.value_network(params[k], S, H, H2v, x, eps_scale=(max(S, H, H2v) + 2) * 2.0 ** -23)
        err = np.abs(_f64(v[k]) - want)
        assert np.all(err <= bound), (k, np.max(err / bound))
        # most rows have no hidden value next to a border
        assert np.median(err) <= 1e-5 * np.std(want)
        diff = _f64(v[k]) - _f64(full[k])
        print(net, "4-bit against full precision:", np.std(diff) / np.std(_f64(full[k])), flush=True)
    tr.close()


def test_step_clip_and_quantised_values_together(m):
    """A small value network trained outside the handle (autograd), its
    gradients clipped in place over the list, its weights read by the 4-bit
    product: the products' gradients and the clipped step follow the oracle."""
    import torch
    from oracle import tensors
    torch.manual_seed(0)
    S, H, B = 48, 80, 300
    ws_ = [torch.randn(H, S) / 7, torch.randn(H) / 7, torch.randn(1, H) / 9, torch.zeros(1)]
    ps = [w.to(dev()).requires_grad_(True) for w in ws_]
    x = torch.randn(B, S, device=dev())
    q = torch.randn(B, 1, device=dev())
    s = None
    out = torch.zeros(2, device=dev())
    for step in range(3):
        for p in ps:
            p.grad = torch.zeros_like(p) if p.grad is None else p.grad.zero_()
        v = torch.relu(x @ ps[0].t() + ps[1]) @ ps[2].t() + ps[3]
        (50.0 * (v - q).square().mean()).backward()
        if s is None:
            s = m.TensorSet([p.grad for p in ps])
            cws = m.grad_norm_workspace(s)
        h = [_f64(p.grad) for p in ps]
        m.grad_clip(s, 1.0, out, cws)
        sync()
        n, c, want = tensors.clip(h, 1.0)
        assert n > 1.0 and abs(float(out[0]) - n) <= 2.0 ** -23 * n
        for p, w in zip(ps, want):
            assert np.all(np.abs(_f64(p.grad) - w) <= 2.0 ** -23 * 1.01 * np.abs(w) + 2.0 ** -149)
        with torch.no_grad():
            for p in ps:
                p -= 0.1 * p.grad
    w1 = m.mx4_empty(H, S)
    m.mx4_quantize(ps[0].detach(), w1)
    h1 = torch.zeros((B, H), device=dev())
    m.mx4_linear(x, w1, h1, m.mx4_matmul_workspace(B, H, S), bias=ps[1].detach(), relu=True)
    sync()
    xv, wv = ref.round_trip(_f64(x)), ref.round_trip(_f64(ps[0]))
    want = np.maximum(xv @ wv.T + _f64(ps[1]), 0.0)
    mag = np.abs(xv) @ np.abs(wv).T + np.abs(_f64(ps[1]))
    assert np.all(np.abs(_f64(h1) - want) <= (S + 1) * 2.0 ** -23 * mag)


def test_binding_refusals(m):
    import torch
    x = torch.zeros((4, 64), device=dev())
    q = m.mx4_empty(4, 64)
    ws = m.mx4_matmul_workspace(4, 4, 64)
    y = torch.zeros((4, 4), device=dev())
    with pytest.raises(ValueError):
        m.mx4_quantize(x[:, :63], q)
    with pytest.raises(ValueError):
        m.mx4_quantize(x.double(), q)
    with pytest.raises(ValueError):
        m.mx4_quantize(torch.zeros((64, 4), device=dev()).t(), q)  # columns not neighbours
    with pytest.raises(ValueError):
        m.mx4_quantize(x, q, axis=2)
    with pytest.raises(ValueError):
        m.mx4_quantize(x.cpu(), q)
    with pytest.raises(ValueError):
        m.mx4_matmul(q, m.mx4_empty(4, 64), y[:, :3], ws)
    with pytest.raises(ValueError):
        m.mx4_matmul(q, m.mx4_empty(4, 64), y, ws, bias=torch.zeros(3, device=dev()))
    with pytest.raises(m.IqlhError):
        m.mx4_matmul(q, m.mx4_empty(4, 65), y, ws)
    with pytest.raises(m.IqlhError):
        m.mx4_matmul(q, m.mx4_empty(4, 64), y, ws[:16])
    with pytest.raises(ValueError):
        m.Mx4(q.codes[:, :16], q.scales, 4, 64)


@pytest.mark.parametrize("M", [1 << 29, 1 << 30])
def test_most_rows_of_one_column(m, M):
    """The most rows of the one-launch kernel and of a matrix.  Multiples of 1 up
    to 3 are exact in 4 bits, and so are their doubles in bf16."""
    import torch
    x = (torch.arange(M, dtype=torch.int32, device="cuda") % 7 - 3).to(torch.bfloat16)[:, None]
    b = m.mx4_empty(1, 1)
    m.mx4_quantize(torch.full((1, 1), 2.0, device="cuda"), b)
    out = torch.full((M, 1), 99.0, dtype=torch.bfloat16, device="cuda")
    m.mx4_linear(x, b, out, m.mx4_matmul_workspace(M, 1, 1))
    assert torch.equal(out, x * 2)
