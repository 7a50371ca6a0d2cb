"""GPU parity of the norm and clip over tensor lists against the fp64 oracle.

Tolerances: the kernel's squares and sums are binary64, so a norm differs from
the oracle's by its one rounding to binary32 (2^-24 relative) plus n 2^-53.
The factor is one more such rounding; a clipped element carries the factor's
rounding and its product's own: 2^-24 + 2^-24 for binary32, 2^-24 + 2^-8 for
bfloat16, 2^-24 + 2^-11 for binary16, and half the type's smallest step where
the result is subnormal."""
import numpy as np
import pytest

from oracle import tensors as ref
from tests.gpu_util import dev, sync

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
HALF_STEP = {"float32": (2.0 ** -24, 2.0 ** -150), "bfloat16": (2.0 ** -8, 2.0 ** -134),
             "float16": (2.0 ** -11, 2.0 ** -25)}


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


def _t(name):
    import torch
    return getattr(torch, name)


def _make(lens, types, seed, offsets=None, scale=1.0):
    """Tensors of the given lengths, each a view `offset` elements into its own
    buffer (so that 16-byte boundaries fall anywhere)."""
    import torch
    g = torch.Generator().manual_seed(seed)
    out = []
    for i, n in enumerate(lens):
        off = offsets[i % len(offsets)] if offsets else 0
        x = torch.randn(n + off, generator=g, dtype=torch.float64) * scale * (1 + i % 3)
        out.append(x.to(_t(types[i % len(types)])).to(dev())[off:])
    return out


def _host(ts):
    import torch
    return [t.detach().to(torch.float64).cpu().numpy() for t in ts]


def _norm(m, ts, kind, each=True, flags=None, stream=None):
    import torch
    s = m.TensorSet(ts)
    ws = m.grad_norm_workspace(s)
    ws[64:].fill_(0xA5)
    out = torch.full((1,), -7.0, device=dev())
    oe = torch.full((len(ts),), -7.0, device=dev()) if each else None
    m.grad_norm(s, out, ws, kind=kind, out_each=oe, flags=flags, stream=stream)
    sync()
    assert int(ws[:64].count_nonzero()) == 0  # as every call leaves it
    return float(out[0]), None if oe is None else oe.cpu().numpy()


def _close(got, want, numel):
    return abs(got - want) <= (U32 * 1.0001 + numel * 2.0 ** -53) * abs(want) + 2.0 ** -150


LISTS = {
    "one_element": ([1], [0]),
    "ones_and_zeros": ([0, 1, 0, 2, 3, 1, 0], [0, 1, 2, 3]),
    "around_16_bytes": ([3, 4, 5, 7, 8, 9, 15, 16, 17, 31], [0, 1, 2, 3, 5, 7]),
    "around_a_piece": ([1023, 1024, 1025, 2047, 2048, 2049, 4099], [0, 1, 3, 7]),
    "value_networks": ([128 * 128, 128, 128 * 128, 128, 128, 1] * 2, [0]),
    "many_small": (list(range(0, 400)), [0, 1, 2]),
    "large_and_small": ([3_000_001, 5, 700_003, 0, 64, 5_000_011], [0, 1, 3]),
    "whole_32k_pieces": ([1 << 23, 3 * (1 << 20), (1 << 22) + 1], [0, 5]),
}
TYPES = {"f32": ["float32"], "bf16": ["bfloat16"], "f16": ["float16"], "mixed": ["float16", "float32", "bfloat16"]}


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("types", sorted(TYPES))
@pytest.mark.parametrize("name", sorted(LISTS))
def test_norm_and_each_tensors_norm(m, name, types, kind):
    lens, offs = LISTS[name]
    ts = _make(lens, TYPES[types], seed=11, offsets=offs)
    got, each = _norm(m, ts, kind)
    h = _host(ts)
    want = ref.norm(h, kind)
    print(name, types, kind, got, want, flush=True)
    assert _close(got, want, sum(lens))
    for i, x in enumerate(h):
        assert _close(float(each[i]), ref.norm([x], kind), lens[i]), i
    # without the per-tensor norms: the same bits
    assert _norm(m, ts, kind, each=False)[0] == got


def test_norm_of_a_set_without_elements(m):
    ts = _make([0, 0], ["float32"], 1)
    got, each = _norm(m, ts, 0)
    assert got == 0.0 and np.all(each == 0.0)
    assert _norm(m, ts, 1)[0] == 0.0


@pytest.mark.parametrize("scale", [1e-30, 1e-44, 1e25, 3e38])
def test_norm_where_binary32_squares_would_not_do(m, scale):
    import torch
    x = (torch.rand(5000, dtype=torch.float64) * 0.5 + 0.5) * scale
    ts = [x.to(torch.float32).to(dev())]
    got, _ = _norm(m, ts, 0)
    want = ref.norm(_host(ts), 0)
    if want > np.finfo(np.float32).max:
        assert got == np.inf
    else:
        assert abs(got - want) <= U32 * 1.0001 * want + 2.0 ** -150


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("value", ["nan", "inf", "-inf", "both"])
@pytest.mark.parametrize("place", [0, 1, 4097, -1])
def test_non_finite_values(m, kind, value, place):
    import torch
    for typ in ("float32", "bfloat16", "float16"):
        ts = _make([7, 9001, 64], [typ], 3, offsets=[0, 1])
        ts[1][place] = float("nan") if value == "both" else float(value)
        if value == "both":
            ts[2][5] = float("inf")
        flags = torch.zeros(1, dtype=torch.int32, device=dev())
        got, each = _norm(m, ts, kind, flags=flags)
        assert np.isnan(got) if value in ("nan", "both") else got == np.inf
        assert np.isfinite(each[0]) and not np.isfinite(each[1])
        assert int(flags[0]) == m.FLAG_NONFINITE_GRAD
        # a clip leaves every element as it is, in place and flat
        before = [t.clone() for t in ts]
        s = m.TensorSet(ts)
        ws = m.grad_norm_workspace(s)
        out = torch.zeros(2, device=dev())
        flat = torch.zeros(s.numel, device=dev())
        flags.zero_()
        m.grad_clip(s, 0.5, out, ws, kind=kind, flags=flags)
        m.grad_clip(s, 0.5, out, ws, kind=kind, flags=flags, out_flat=flat)
        sync()
        assert float(out[1]) == 1.0 and not np.isfinite(float(out[0]))
        assert int(flags[0]) == m.FLAG_NONFINITE_GRAD
        for a, b in zip(before, ts):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
        assert torch.equal(torch.cat([t.float() for t in ts]).nan_to_num(7.0), flat.nan_to_num(7.0))


def _check_clipped(ts, h, c, got):
    for t, x, y in zip(ts, h, got):
        u, tiny = HALF_STEP[str(t.dtype).split(".")[1]]
        want = x * c
        assert np.all(np.abs(y - want) <= (u + U32) * 1.0001 * np.abs(want) + tiny), np.max(np.abs(y - want))


@pytest.mark.parametrize("kind", [0, 1])
@pytest.mark.parametrize("types", sorted(TYPES))
@pytest.mark.parametrize("name", ["one_element", "ones_and_zeros", "around_16_bytes", "around_a_piece",
                                  "large_and_small"])
def test_clip_in_place(m, name, types, kind):
    import torch
    lens, offs = LISTS[name]
    ts = _make(lens, TYPES[types], seed=5, offsets=offs)
    h = _host(ts)
    n = ref.norm(h, kind)
    s = m.TensorSet(ts)
    ws = m.grad_norm_workspace(s)
    out = torch.zeros(2, device=dev())
    flags = torch.zeros(1, dtype=torch.int32, device=dev())
    # above the norm: nothing changes
    before = [t.clone() for t in ts]
    m.grad_clip(s, 2.0 * n, out, ws, kind=kind, flags=flags)
    sync()
    assert float(out[1]) == 1.0 and all(torch.equal(a, b) for a, b in zip(before, ts))
    # below it
    bound = float(np.float32(0.3 * n))
    m.grad_clip(s, bound, out, ws, kind=kind, flags=flags)
    sync()
    _, c, _ = ref.clip(h, bound, kind)
    assert _close(float(out[0]), n, sum(lens)) and abs(float(out[1]) - c) <= 1.01 * U32 * c
    assert int(flags[0]) == 0
    _check_clipped(ts, h, c, _host(ts))


@pytest.mark.parametrize("lead", [0, 1, 2, 3])
@pytest.mark.parametrize("types", sorted(TYPES))
@pytest.mark.parametrize("name", ["one_element", "ones_and_zeros", "around_16_bytes", "around_a_piece",
                                  "value_networks", "large_and_small"])
def test_clip_into_the_flat_vector(m, name, types, lead):
    import torch
    lens, offs = LISTS[name]
    ts = _make(lens, TYPES[types], seed=6, offsets=offs)
    h = _host(ts)
    n = ref.norm(h, 0)
    s = m.TensorSet(ts)
    ws = m.grad_norm_workspace(s)
    out = torch.zeros(2, device=dev())
    buf = torch.full((lead + s.numel + 5,), 9.5, device=dev())
    flat = buf[lead:lead + s.numel]
    before = [t.clone() for t in ts]
    for bound in (float(np.float32(0.01 * n)), 3.0 * n):
        m.grad_clip(s, bound, out, ws, out_flat=flat)
        sync()
        _, c, _ = ref.clip(h, bound, 0)
        want = np.concatenate(h) * c
        got = flat.double().cpu().numpy()
        assert np.all(np.abs(got - want) <= 2 * U32 * 1.0001 * np.abs(want) + 2.0 ** -149)
        assert all(torch.equal(a, b) for a, b in zip(before, ts))
        assert torch.all(buf[:lead] == 9.5) and torch.all(buf[lead + s.numel:] == 9.5)


def test_a_norm_at_the_bound_is_not_clipped(m):
    import torch
    t = torch.tensor([3.0, 4.0], device=dev())
    s = m.TensorSet([t])
    out = torch.zeros(2, device=dev())
    m.grad_clip(s, 5.0, out, m.grad_norm_workspace(s))
    sync()
    assert out.tolist() == [5.0, 1.0] and t.tolist() == [3.0, 4.0]
    m.grad_clip(s, float("inf"), out, m.grad_norm_workspace(s))
    sync()
    assert out.tolist() == [5.0, 1.0]
    m.grad_clip(s, 2.5, out, m.grad_norm_workspace(s))
    sync()
    assert out.tolist() == [5.0, 0.5] and t.tolist() == [1.5, 2.0]


def test_results_repeat_and_a_workspace_is_reused(m):
    import torch
    a = _make([1_000_003, 77], ["float32", "bfloat16"], 8)
    b = _make([1_000_003, 77], ["float32", "bfloat16"], 9)
    sa, sb = m.TensorSet(a), m.TensorSet(b)
    ws = m.grad_norm_workspace(sa)
    outs = torch.zeros(6, device=dev())
    for i, s in enumerate([sa, sb, sa, sb, sa, sb]):
        m.grad_norm(s, outs[i:i + 1], ws)
    sync()
    o = outs.tolist()
    assert o[0] == o[2] == o[4] and o[1] == o[3] == o[5] and o[0] != o[1]


def test_captured_clips_share_a_workspace_and_follow_new_gradients(m):
    import torch
    ts = _make([40_001, 3, 128], ["float32", "float16"], 4)
    keep = [t.clone() for t in ts]
    s = m.TensorSet(ts)
    ws = m.grad_norm_workspace(s)
    out = torch.zeros(2, device=dev())
    flat = torch.zeros(s.numel, device=dev())
    norm = torch.zeros(1, device=dev())
    graphs = []
    side = torch.cuda.Stream()
    for fn in (lambda: m.grad_clip(s, 1.0, out, ws, out_flat=flat), lambda: m.grad_norm(s, norm, ws)):
        fn()
        sync()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            fn()
        graphs.append(g)
    for k in range(4):
        for t, x in zip(ts, keep):
            t.copy_(x * (k + 1))
        flat.zero_()
        for g in graphs:
            g.replay()
        sync()
        got = (float(norm[0]), out.clone(), flat.clone())
        eager_out, eager_flat = torch.zeros(2, device=dev()), torch.zeros(s.numel, device=dev())
        side.wait_stream(torch.cuda.current_stream())
        m.grad_clip(s, 1.0, eager_out, ws, out_flat=eager_flat, stream=side)
        sync()
        assert torch.equal(got[1], eager_out) and torch.equal(got[2], eager_flat)
        assert got[0] == float(eager_out[0])


def test_calls_on_several_streams_at_once(m):
    """Sets and workspaces of their own on four streams, the sets dropped right
    after their calls."""
    import torch
    streams = [torch.cuda.Stream() for _ in range(4)]
    lists = [_make([50_000 + 7 * k, 33, 2000], ["float32", "bfloat16"], 60 + k) for k in range(4)]
    want = [ref.norm(_host(ts), 0) for ts in lists]
    outs = [torch.zeros(8, device=dev()) for _ in range(4)]
    flats = [torch.zeros(sum(t.numel() for t in ts), device=dev()) for ts in lists]
    wss = [m.grad_norm_workspace(m.TensorSet(ts)) for ts in lists]
    sync()
    for rep in range(8):
        for k, st in enumerate(streams):
            s = m.TensorSet(lists[k])
            m.grad_norm(s, outs[k][rep:rep + 1], wss[k], stream=st)
            m.grad_clip(s, 0.5, torch.zeros(2, device=dev()), wss[k], out_flat=flats[k], stream=st)
            del s
            torch.full((4096,), 7, dtype=torch.uint8, device=dev())  # would take the freed table's place
    sync()
    for k in range(4):
        assert all(_close(float(x), want[k], 60_000) for x in outs[k])
        c = 0.5 / want[k]
        x = np.concatenate(_host(lists[k]))
        assert np.all(np.abs(flats[k].double().cpu().numpy() - x * c) <= 2 * U32 * 1.001 * np.abs(x * c) + 2.0 ** -149)


def test_more_elements_than_32_bits_count(m):
    import torch
    n = (1 << 31) + 9
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB of free device memory")
    x = torch.full((n,), 0.5, dtype=torch.bfloat16, device=dev())
    y = torch.full((3,), 2.0, dtype=torch.float32, device=dev())
    x[-1] = -3.0
    s = m.TensorSet([x, y])
    out = torch.zeros(2, device=dev())
    flat = torch.zeros(s.numel, device=dev())
    m.grad_clip(s, 1.0, out, m.grad_norm_workspace(s), out_flat=flat)
    sync()
    want = np.sqrt((n - 1) * 0.25 + 9.0 + 12.0)
    assert _close(float(out[0]), want, n)
    c = 1.0 / want
    for i, v in ((0, 0.5), (n - 2, 0.5), (n - 1, -3.0), (n, 2.0), (n + 2, 2.0), ((1 << 31) - 1, 0.5)):
        assert abs(float(flat[i]) - v * c) <= 2 * U32 * 1.01 * abs(v * c), i
    assert float(flat.min()) == float(flat[n - 1]) and float(flat[:n - 1].max()) == float(flat[0])


def test_feeds_the_gradient_budget(m):
    """A network's gradients, clipped into the flat vector, as one source of
    the budgeted accumulation with Adam."""
    import torch
    from oracle import budget
    lens = [64 * 33, 64, 64 * 64, 64, 64, 1]
    a = _make(lens, ["float32", "bfloat16"], 21, scale=4.0)
    b = _make(lens, ["float32"], 22)
    n = sum(lens)
    flats = []
    for ts in (a, b):
        s = m.TensorSet(ts)
        flats.append(torch.zeros(n, device=dev()))
        m.grad_clip(s, 2.0, torch.zeros(2, device=dev()), m.grad_norm_workspace(s), out_flat=flats[-1])
    grad = torch.zeros(n, device=dev())
    norms = torch.zeros(3, device=dev())
    ws = torch.zeros(m.grad_budget_workspace_bytes(n, 2) // 4, device=dev())
    m.grad_budget_accumulate(grad, flats, (0.7, 0.3), (1.0, 1.0), n, 1.0, norms, None, ws)
    sync()
    src = [np.concatenate(ref.clip(_host(ts), 2.0)[2]) for ts in (a, b)]
    want, wn, _, _ = budget.accumulate(src, (0.7, 0.3), (1.0, 1.0), 1.0)
    assert np.linalg.norm(grad.double().cpu().numpy() - want) <= 1e-5 * np.linalg.norm(want)
    assert abs(float(norms[0]) - wn[0]) <= 1e-5 * wn[0]


def test_flat_output_inside_a_tensor_is_refused_beside_empty_tensors(m):
    import torch
    base = torch.zeros(4096, device="cuda")
    ts = m.TensorSet([base[:2048], base[1000:1000], base[3000:3000]])
    ws, out = m.grad_norm_workspace(ts), torch.empty(2, device="cuda")
    for lo in (0, 900, 2047 - 64):
        with pytest.raises(ValueError, match="shares memory"):
            m.grad_clip(ts, 1.0, out, ws, out_flat=base[lo:lo + 2048])
    m.grad_clip(ts, 1.0, out, ws, out_flat=base[2048:])
