"""The policy loss, its gradients, the clipping of their common norm and the orthogonalised
step as one run: a head over many actions and the embeddings of a batch's states, trained on
the device alone.  Each operator is held to its own bounds on the inputs that the one before
it left, and the run as a whole to itself, bit for bit, replayed from a graph and beside
another run on another stream."""
import numpy as np
import pytest

from oracle import ortho as ref_ortho
from tests import test_gpu_ortho as ortho
from tests import test_gpu_policy as policy
from tests.gpu_util import dev, sync

pytestmark = pytest.mark.gpu

LR, MU, MAX_NORM = 0.02, 0.9, 0.05


@pytest.fixture(scope="module")
def m():
    import offline_rl_step_amd as m
    return m


class Run:
    def __init__(self, m, seed, rows, dim, actions, dtype):
        import torch
        self.m = m
        self.c = c = policy._case(seed, rows, dim, actions, dtype)
        h, w = c["hidden"], c["weight"]
        self.out = dict(nll=torch.zeros(rows, device=dev()), lse=torch.zeros(rows, device=dev()),
                        loss=torch.zeros(1, device=dev()), dh=torch.zeros(rows, dim, dtype=h.dtype, device=dev()),
                        dw=torch.zeros(actions, dim, dtype=h.dtype, device=dev()), db=torch.zeros(actions, device=dev()))
        self.momentum = [torch.zeros(rows, dim, device=dev()), torch.zeros(actions, dim, device=dev())]
        self.clip = torch.zeros(2, device=dev())
        self.flags = torch.zeros(1, dtype=torch.int32, device=dev())
        self.grads = [self.out["dh"], self.out["dw"], self.out["db"]]
        self.set = m.TensorSet(self.grads)
        self.matrices = m.MatrixSet(self.grads[:2], [h, w], self.momentum)
        self.ws = (m.policy_loss_workspace(rows, actions, dim, h.dtype, grad=True), m.grad_norm_workspace(self.set),
                   m.orthogonalize_workspace(self.matrices))

    def gradients(self):
        c, o = self.c, self.out
        kw = dict(bias=c["bias"], row_weights=c["row_weights"])
        self.m.policy_loss(c["hidden"], c["weight"], c["taken"], o["nll"], o["lse"], self.ws[0], out_loss=o["loss"],
                           flags=self.flags, **kw)
        self.m.policy_loss_grad(c["hidden"], c["weight"], c["taken"], o["lse"], self.ws[0], d_hidden=o["dh"],
                                d_weight=o["dw"], d_bias=o["db"], **kw)

    def clipped(self):
        self.m.grad_clip(self.set, MAX_NORM, self.clip, self.ws[1], flags=self.flags)

    def update(self):
        self.m.muon_step(self.matrices, self.ws[2], LR, momentum=MU, flags=self.flags)
        self.c["bias"].add_(self.out["db"], alpha=-LR)

    def step(self):
        self.gradients()
        self.clipped()
        self.update()

    def state(self):
        return [self.c["hidden"], self.c["weight"], self.c["bias"], *self.momentum, *self.grads, self.clip,
                *(self.out[k] for k in ("nll", "lse", "loss"))]


SIZES = [(96, 64, 300), (40, 128, 12), (200, 72, 500)]


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("rows,dim,actions", SIZES)
def test_each_step_of_a_run(m, rows, dim, actions, dtype):
    run = Run(m, 3 + rows, rows, dim, actions, dtype)
    half = ortho.HALF[dtype]
    host = ortho._host
    for _ in range(3):
        run.gradients()
        sync()
        policy._check(run.c, run.out)
        before = [host(g) for g in run.grads]
        run.clipped()
        sync()
        norm = np.sqrt(sum((g * g).sum() for g in before))
        factor = min(1.0, MAX_NORM / norm)
        # the norm from binary64 sums, rounded to binary32, as the factor is, and their quotient
        assert abs(float(run.clip[0]) - norm) <= 2.0 ** -23 * norm
        assert abs(float(run.clip[1]) - factor) <= 2.0 ** -22 * factor
        for g, was, h in zip(run.grads, before, (half, half, 2.0 ** -24)):
            want = float(run.clip[1]) * was
            assert np.all(np.abs(host(g) - want) <= (h + 2.0 ** -24) * np.abs(want) + 2.0 ** -133)
        was = [host(t) for t in (*run.momentum, run.c["hidden"], run.c["weight"])]
        run.update()
        sync()
        for i, w in enumerate((run.c["hidden"], run.c["weight"])):
            g = host(run.grads[i])
            want_w, want_m = ref_ortho.muon(was[2 + i], was[i], g, LR, MU)
            assert np.all(np.abs(host(run.momentum[i]) - want_m)
                          <= 2.0 ** -24 * (np.abs(want_m) + np.abs(MU * was[i])) + 2.0 ** -149)
            u = g + MU * want_m
            planes = ortho._planes(m, g.shape, dtype)
            o = ref_ortho.orthogonalize(u)
            tol = 2 * ref_ortho.rate(LR, g.shape) * ortho._moved(u, planes, o)
            ortho._near(host(w), want_w, tol + 3 * 2.0 ** -24 * np.linalg.norm(was[2 + i]), half, (i, g.shape))
    assert run.flags.item() == 0


@pytest.mark.parametrize("dtype", ["float32", "float16"])
@pytest.mark.parametrize("rows,dim,actions", SIZES)
def test_a_run_in_a_graph_and_two_runs_at_once(m, rows, dim, actions, dtype):
    import torch
    eager = Run(m, 5, rows, dim, actions, dtype)
    for _ in range(4):
        eager.step()
    sync()
    run = Run(m, 5, rows, dim, actions, dtype)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run.step()
    beside = [Run(m, 5, rows, dim, actions, dtype) for _ in range(2)]
    side = [torch.cuda.Stream() for _ in beside]
    sync()
    for rep in range(4):
        graph.replay()
        for s, other in zip(side, beside):
            with torch.cuda.stream(s):
                other.step()
        if rep % 2:
            sync()
            torch.empty(1 << 20, device=dev()).fill_(float(rep))
    sync()
    for other in (run, *beside):
        for k, (a, b) in enumerate(zip(eager.state(), other.state())):
            assert torch.equal(a, b), k


@pytest.mark.parametrize("rows,dim,actions,dtype", [(2100, 24, 6500, "float32"),  # 234 tiles of 256, two planes
                                                    (1100, 24, 8200, "bfloat16"),  # 165, one
                                                    (300, 16, 17, "float16"), (300, 16, 16, "float16"),
                                                    (16, 40, 5000, "float32"), (17, 40, 5000, "float32"),
                                                    # the widest that few actions' and few rows' kernels take, and wider
                                                    (40, 1024, 16, "float32"), (40, 1025, 16, "float32"),
                                                    (16, 1980, 300, "float32"), (16, 4000, 300, "bfloat16"),
                                                    (16, 4104, 300, "bfloat16"), (3, 16384, 40, "float16")])
def test_where_the_kernels_change(m, rows, dim, actions, dtype):
    c = policy._case(7, rows, dim, actions, dtype)
    out = policy._run(m, c)
    sync()
    policy._check(c, out)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_gradients_of_wide_heads_in_tiles_of_256(m, dtype):
    """dW of 256 x 256 tiles (27 x 8 of them), its bounds as for the small ones."""
    c = policy._case(9, 70, 2040, 6700, dtype)
    out = policy._run(m, c)
    sync()
    policy._check(c, out)
