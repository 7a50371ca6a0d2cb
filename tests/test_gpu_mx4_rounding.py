"""The 4-bit products on operands that do not lie on the 4-bit grid: every kernel
form, wide ranges within and between blocks, subnormal values, operands
quantised along their columns, and the value network over many rows.

A product's bound is that of its summation: each of at most K additions off by
2^-23 of a partial sum that is at most the sum of the terms' magnitudes (2^-24 to
nearest, twice that for an addition that truncates), and the output type's half step.  A
product with rows of the identity has one term that is not zero, which no
order of the sum rounds: it is the quantised value itself."""
import numpy as np
import pytest

from oracle import mx4 as ref
from tests.gpu_util import dev, sync

pytestmark = pytest.mark.gpu

HALF = {"float32": 2.0 ** -24, "bfloat16": 2.0 ** -8}


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


def _values(seed, r, c, lo=-12, hi=12):
    """Device floats of which a fifth are scaled by up to 2^lo .. 2^hi, as whole
    blocks are too; some zeros."""
    import torch
    g = torch.Generator(device=dev()).manual_seed(seed)
    x = torch.randn((r, c), generator=g, device=dev(), dtype=torch.float64)
    e = torch.randint(lo, hi + 1, (r, c), generator=g, device=dev())
    x *= torch.exp2(e * (torch.rand((r, c), generator=g, device=dev()) < 0.2))
    kb = -(-c // 32)
    x *= torch.exp2(torch.randint(lo, hi + 1, (r, kb), generator=g, device=dev()).double()).repeat_interleave(32, 1)[:, :c]
    x[torch.rand((r, c), generator=g, device=dev()) < 0.05] = 0.0
    return x


def _quantized(m, x, axis=1):
    q = m.mx4_empty(*x.shape, axis)
    m.mx4_quantize(x, q, axis=axis)
    return q


# every form of the linear: up to 16 rows, 17 to 64 and more in one launch, many rows, two launches
LINEARS = [(1, 8192), (3, 5001), (16, 1000), (17, 200), (33, 256), (64, 129), (300, 200), (64, 2000), (130, 700), (2000, 600),
           (16384, 333), (16389, 1000), (20000, 96)]


@pytest.mark.parametrize("xd", ["float32", "bfloat16", "float16"])
@pytest.mark.parametrize("mk", LINEARS)
def test_linear_takes_the_values_that_quantize_gives(m, mk, xd):
    import torch
    M, K = mk
    N = min(K, 512)
    scale = {"float32": 1.0, "bfloat16": 1.0, "float16": 2.0 ** -6}[xd]
    x = (_values(M + K, M, K, -8, 8) * scale).to(_t(xd))
    if xd == "float16":
        x = x.clamp(-60000.0, 60000.0)
    if M > 2:
        x[1] = float(np.float32(2.0 ** -24)) * torch.arange(K, device=dev()) % 7  # small and, in binary16, subnormal
        x[2, ::3] = 0.0
    at = torch.arange(K - N, K, device=dev())  # the identity's last N rows
    b = torch.zeros((N, K), device=dev())
    b[torch.arange(N, device=dev()), at] = 1.0
    y = torch.full((M, N), 7.0, device=dev())
    ws = m.mx4_matmul_workspace(M, N, K)
    ws.fill_(0xFF)
    m.mx4_linear(x, _quantized(m, b), y, ws)
    back = torch.full((M, K), 7.0, device=dev())
    m.mx4_dequantize(_quantized(m, x), back)
    sync()
    assert torch.equal(y, back[:, K - N:])
    rows = np.unique(np.linspace(0, M - 1, 40).astype(int))
    assert np.array_equal(_f64(back)[rows], ref.round_trip(_f64(x)[rows]))


def _check(got, av, bv, K, od, bias=None):
    want, mag = av @ bv.T, np.abs(av) @ np.abs(bv).T
    if bias is not None:
        want, mag = want + bias, mag + np.abs(bias)
        K = K + 1
    err = np.abs(got - want)
    assert np.all(err <= K * 2.0 ** -23 * mag + HALF[od] * 1.01 * np.abs(want)), np.max(err / (mag + 1e-300)) / (K * 2.0 ** -23)


# split by k (three sizes), straight from memory, tiles of 128 and 256 with K of up to 2048 and more
PRODUCTS = [(20, 700, 4000), (200, 333, 777), (500, 520, 900), (900, 850, 1500), (1500, 1411, 300), (1500, 1411, 600),
            (1400, 1500, 2100), (2000, 2100, 5000), (3584, 3600, 600), (3584, 3600, 2300), (8200, 1700, 1024)]


@pytest.mark.parametrize("od", sorted(HALF))
@pytest.mark.parametrize("mnk", PRODUCTS)
def test_products_of_wide_ranging_blocks(m, mnk, od):
    import torch
    M, N, K = mnk
    a, b = _values(M + 1, M, K).float(), _values(N + 2, N, K).float()
    bias = _values(3, 1, N)[0].float()
    y = torch.full((M, N), 7.0, dtype=_t(od), device=dev())
    ws = m.mx4_matmul_workspace(M, N, K)
    ws.fill_(0xFF)
    m.mx4_matmul(_quantized(m, a), _quantized(m, b), y, ws, bias=bias)
    sync()
    rows = np.unique(np.concatenate([[0, M - 1], np.linspace(0, M - 1, 60).astype(int)]))
    _check(_f64(y)[rows], ref.round_trip(_f64(a)[rows]), ref.round_trip(_f64(b)), K, od, _f64(bias))


@pytest.mark.parametrize("mnk", [(16390, 513, 333), (16384, 70, 1000), (20, 300, 250), (50, 130, 200), (300, 257, 100), (700, 300, 900)])
@pytest.mark.parametrize("xd", ["float32", "bfloat16"])
def test_linears_of_wide_ranging_blocks(m, mnk, xd):
    import torch
    M, N, K = mnk
    x, b = _values(M, M, K).to(_t(xd)), _values(N, N, K).float()
    for od in sorted(HALF):
        y = torch.full((M, N), 7.0, dtype=_t(od), device=dev())
        m.mx4_linear(x, _quantized(m, b), y, m.mx4_matmul_workspace(M, N, K))
        sync()
        rows = np.unique(np.concatenate([[0, M - 1], np.linspace(0, M - 1, 100).astype(int)]))
        _check(_f64(y)[rows], ref.round_trip(_f64(x)[rows]), ref.round_trip(_f64(b)), K, od)


@pytest.mark.parametrize("bnk", [(5001, 130, 77), (33, 64, 200), (16384, 128, 128), (700, 1, 1), (2050, 513, 96)])
@pytest.mark.parametrize("dt", ["float32", "bfloat16"])
def test_weight_gradient_from_operands_quantised_along_the_batch(m, bnk, dt):
    """dW[n][k] = sum over the batch of dy[i][n] x[i][k], and the input's
    gradient dx[i][k] = sum_n dy[i][n] w[n][k] with w quantised along n."""
    import torch
    B, N, K = bnk
    dy, x = _values(1, B, N, -3, 3).to(_t(dt)), _values(2, B, K, -3, 3).to(_t(dt))
    w = _values(4, N, K, -3, 3).to(_t(dt))
    dw, dx = torch.full((N, K), 7.0, device=dev()), torch.full((B, K), 7.0, device=dev())
    m.mx4_matmul(_quantized(m, dy, 0), _quantized(m, x, 0), dw, m.mx4_matmul_workspace(N, K, B))
    m.mx4_matmul(_quantized(m, dy, 1), _quantized(m, w, 0), dx, m.mx4_matmul_workspace(B, K, N))
    sync()
    _check(_f64(dw), ref.round_trip(_f64(dy).T), ref.round_trip(_f64(x).T), B, "float32")
    rows = np.unique(np.linspace(0, B - 1, 200).astype(int))
    _check(_f64(dx)[rows], ref.round_trip(_f64(dy)[rows]), ref.round_trip(_f64(w).T), N, "float32")


@pytest.mark.parametrize("net", [(256, 512, 0, 1), (128, 256, 160, 2), (100, 1024, 0, 1)])
def test_value_network_of_many_rows_with_trained_like_weights(m, net):
    """Batches large enough for the 128-row workgroups: V within the oracle's
    bound for hidden sums that are off by K 2^-23 of their terms."""
    import torch
    S, H, H2, G = net
    H2v, B = H2 or H, 32768 + 77
    g = np.random.default_rng(7)
    params = [np.concatenate([g.uniform(-1, 1, H * S) / np.sqrt(S), g.uniform(-1, 1, H) / np.sqrt(S),
                              g.uniform(-1, 1, H2v * H) / np.sqrt(H), g.uniform(-1, 1, H2v) / np.sqrt(H),
                              g.uniform(-1, 1, H2v) / np.sqrt(H2v), [0.1]]).astype(np.float32) for _ in range(G)]
    x = g.standard_normal((B, S)).astype(np.float32)
    tr = m.IqlTrainer(m.make_config(S, H, B, num_groups=G, hidden2=H2), np.concatenate(params))
    v = torch.zeros((G, B), device=dev())
    ws = tr.forward_values_mx4_workspace(B)
    ws.fill_(0xFF)
    tr.forward_values_mx4(torch.from_numpy(x).to(dev()), B, v, ws)
    sync()
    rows = np.unique(np.concatenate([np.arange(130), g.integers(0, B, 300), np.arange(B - 130, B)]))
    for k in range(G):
        want, bound = ref.value_network(params[k], S, H, H2v, x[rows], eps_scale=(max(S, H, H2v) + 2) * 2.0 ** -23)
        err = np.abs(_f64(v[k])[rows] - want)
        assert np.all(err <= bound), (k, np.max(err / bound))
    tr.close()


@pytest.mark.parametrize("mnk", [(1, 64, 96), (40, 24, 96), (300, 500, 700), (17000, 96, 160)])
def test_column_blocks_of_one_buffer(m, mnk):
    """x and out side by side in one buffer: taken, and equal to separate ones;
    one column over the border: refused."""
    import torch
    M, N, K = mnk
    buf = torch.zeros((M, K + N + 5), device=dev())
    buf[:, :K] = _values(5, M, K).float()
    x, y = buf[:, :K], buf[:, K:K + N]
    b = _quantized(m, _values(6, N, K).float())
    ws = m.mx4_matmul_workspace(M, N, K)
    want = torch.zeros((M, N), device=dev())
    m.mx4_linear(x.clone(), b, want, ws)
    before = x.clone()
    m.mx4_linear(x, b, y, ws)
    sync()
    assert torch.equal(y, want) and torch.equal(x, before) and int(buf[:, K + N:].count_nonzero()) == 0
    with pytest.raises(m.IqlhError, match="share memory"):
        m.mx4_linear(x, b, buf[:, K - 1:K - 1 + N], ws)
    region = torch.zeros(max(want.nbytes, ws.numel()), dtype=torch.uint8, device=dev())
    with pytest.raises(m.IqlhError, match="share memory"):
        m.mx4_linear(x, b, region[:want.nbytes].view(torch.float32).view(M, N), region[:ws.numel()])
