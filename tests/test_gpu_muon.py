"""The Muon step against its formulas in 64 bits.

Momentum: two fp32 roundings and that of its type.  The update: as
orthogonalisation's results (4e-3 in the 2-norm; its tests say why), rounded in
the master to half an fp32 step of the weight.
"""
import copy
import math

import pytest
import torch

from adamw_optimizer_step_sm_gb300 import adamw_sm as A
from adamw_optimizer_step_sm_gb300 import matrix as M
from adamw_optimizer_step_sm_gb300 import optim as OPT

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
# both kernels, tall, wide, batches, odd sizes, one element
SHAPES = [(128, 384), (512, 128), (4, 33, 70), (515, 300), (256, 256), (100, 1), (1, 7), (1, 1), (2, 3, 40, 24), (700, 130), (129, 1030)]


@pytest.fixture(autouse=True)
def _no_wait_ran_out():
    yield
    assert A.adamw_matrix_status() == 0


def exact_ortho(x, steps=5):
    x = x / torch.linalg.matrix_norm(x).clamp(min=1e-7)[..., None, None]
    a, b, c = M.COEFFICIENTS
    for _ in range(steps):
        g = x @ x.mT
        x = a * x + (b * g + c * (g @ g)) @ x
    return x


def params_of(shapes, seed=3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return [torch.nn.Parameter((torch.randn(s, generator=g, device="cuda") * 0.02).bfloat16()) for s in shapes]


def set_grads(params, seed, scale=1e-3):
    g = torch.Generator(device="cuda").manual_seed(seed)
    for p in params:
        p.grad.copy_((torch.randn(p.shape, generator=g, device="cuda") * scale).bfloat16())


def norms(x):
    return torch.linalg.matrix_norm(x.double()).max()


class Exact:
    """The step in 64 bits from the optimizer's state before it."""

    def __init__(self, opt, params, nesterov=True, scale="rms"):
        self.opt, self.nesterov, self.scale = opt, nesterov, scale
        self.before = [(p.grad.double().clone(), opt.state[p]["momentum"].double().clone(), opt.state[p]["master"].double().clone())
                       for p in params]
        self.params = params

    def check(self, momentum_dtype):
        for p, (g, m, w) in zip(self.params, self.before):
            group = next(x for x in self.opt.param_groups if any(q is p for q in x["params"]))
            mu, lr, decay = group["momentum"], float(group["lr"]), group["weight_decay"]
            m2 = m + (1 - mu) * (g - m)
            u = g + mu * (m2 - g) if self.nesterov else m2
            r, c = p.shape[-2:]
            s = 0.2 * math.sqrt(max(r, c)) if self.scale == "rms" else math.sqrt(max(1.0, r / c))
            o = exact_ortho(u)
            w2 = w * (1 - lr * decay) - lr * s * o
            st = self.opt.state[p]
            size = m.abs() + g.abs()
            assert (st["momentum"].double() - m2).abs().le(m2.abs() * torch.finfo(momentum_dtype).eps / 2 + size * 2.0 ** -23).all()
            room = 4e-3 * lr * s * torch.linalg.matrix_norm(o) + 2 * 2.0 ** -24 * torch.linalg.matrix_norm(w) + 1e-12
            assert (torch.linalg.matrix_norm(st["master"].double() - w2) <= room).all()
            assert torch.equal(p.detach(), st["master"].bfloat16())


@pytest.mark.parametrize("momentum_dtype", [F32, BF], ids=str)
@pytest.mark.parametrize("nesterov,scale", [(True, "rms"), (False, "spectral")])
def test_steps(momentum_dtype, nesterov, scale):
    params = params_of(SHAPES)
    opt = OPT.Muon(params, lr=1e-2, momentum=0.9, nesterov=nesterov, scale=scale, momentum_dtype=momentum_dtype)
    for step in range(4):
        set_grads(params, 10 + step)
        e = Exact(opt, params, nesterov, scale)
        opt.step()
        e.check(momentum_dtype)
        assert int(opt.last_nonfinite[0]) == 0
        opt.param_groups[0]["lr"] *= 0.5


def test_groups_have_their_own_rates():
    params = params_of(SHAPES)
    opt = OPT.Muon([{"params": params[:4], "lr": 1e-2, "weight_decay": 0.0}, {"params": params[4:], "momentum": 0.5}], lr=1e-3)
    set_grads(params, 1)
    e = Exact(opt, params)
    opt.step()
    e.check(F32)


def test_no_rate_keeps_the_weights():
    params = params_of(SHAPES)
    opt = OPT.Muon(params, lr=0.0)
    keep = [p.detach().clone() for p in params]
    set_grads(params, 1)
    opt.step()
    assert all(torch.equal(p, k) for p, k in zip(params, keep))


@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
def test_a_step_that_is_not_finite_writes_nothing(bad):
    params = params_of(SHAPES)
    opt = OPT.Muon(params, lr=1e-2)
    set_grads(params, 1)
    opt.step()
    state = lambda: [t.clone() for p in params for t in (p.detach(), opt.state[p]["momentum"], opt.state[p]["master"])]
    for which in range(len(params)):
        set_grads(params, 2)
        params[which].grad.view(-1)[-1] = bad
        before = state()
        opt.step()
        assert int(opt.last_nonfinite[0]) == 1
        assert all(torch.equal(a, b) for a, b in zip(before, state()))
    set_grads(params, 3)   # and the next one goes on
    e = Exact(opt, params)
    opt.step()
    assert int(opt.last_nonfinite[0]) == 0
    e.check(F32)


def test_zero_and_extreme_gradients():
    for scale in (0.0, 1e-30, 1e30):
        params = params_of(SHAPES)
        opt = OPT.Muon(params, lr=1e-2, weight_decay=0.0)
        keep = [p.detach().clone() for p in params]
        set_grads(params, 1, scale)
        opt.step()
        assert int(opt.last_nonfinite[0]) == 0
        for p, k in zip(params, keep):
            if scale < 1:   # below eps: hardly a step
                assert (p.float() - k.float()).abs().max() <= k.float().abs().max() * 2.0 ** -8
            else:
                step = (opt.state[p]["master"] - k.float()).double() / (-1e-2 * 0.2 * math.sqrt(max(p.shape[-2:])))
                o = exact_ortho(p.grad.double())
                # the step is lr times the update, on weights of fp32
                room = 4e-3 * torch.linalg.matrix_norm(o) + 2.0 ** -23 * torch.linalg.matrix_norm(k.double()) / 2e-3
                assert (torch.linalg.matrix_norm(step - o) <= room).all()


def test_through_a_model_with_a_global_clip():
    """Experts and a dense layer with Muon, the vectors with AdamW, one norm
    over both: as they are used together."""
    torch.manual_seed(0)
    dense, up, down = params_of([(64, 64), (4, 96, 64), (4, 64, 96)])
    bias = torch.nn.Parameter(torch.zeros(64, dtype=BF, device="cuda"))
    muon, adam = OPT.Muon([dense, up, down], lr=1e-2), OPT.AnyPrecisionAdamW([bias], lr=1e-2)
    clip = OPT.GlobalClip(muon, adam)
    at = torch.tensor([0, 60, 61, 190, 200], device="cuda")
    x, target = torch.randn(200, 64, device="cuda").bfloat16(), torch.randn(200, 64, device="cuda")
    pointers = [p.grad.data_ptr() for p in (dense, up, down, bias)]
    for _ in range(3):
        muon.zero_grad()
        adam.zero_grad()
        h = torch.nn.functional.linear(x, dense, bias)
        y = h + M.expert_linear(torch.relu(M.expert_linear(h, up, at)), down, at)
        (y.float() - target).square().mean().backward()
        norm = torch.sqrt(sum(p.grad.double().square().sum() for p in (dense, up, down, bias)))
        c = clip(0.5 * float(norm))
        assert abs(float(c.norm) - float(norm)) < 1e-5 * float(norm) and 0.49 < float(c.coef) < 0.51
        e = Exact(muon, [dense, up, down])
        muon.step()
        adam.step()
        e.check(F32)
    assert pointers == [p.grad.data_ptr() for p in (dense, up, down, bias)]   # backward wrote into the buffers


def test_captured_step_follows_the_rate():
    shapes = [(64, 48), (300, 200), (2, 130, 40)]
    a, b = params_of(shapes), params_of(shapes)
    opts = [OPT.Muon(p, lr=1e-2) for p in (a, b)]
    for p, o in zip((a, b), opts):
        set_grads(p, 1)
        o.step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        opts[0].step()
    for k, lr in enumerate((1e-2, 3e-3, 0.0)):
        for p, o in zip((a, b), opts):
            set_grads(p, 5 + k)
            o.param_groups[0]["lr"] = lr
        opts[0].push_rates()
        g.replay()
        opts[1].step()
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_same_bits_on_a_side_stream():
    a, b = params_of(SHAPES), params_of(SHAPES)
    x, y = OPT.Muon(a, lr=1e-2), OPT.Muon(b, lr=1e-2)
    side = torch.cuda.Stream()
    for k in range(3):
        set_grads(a, k)
        set_grads(b, k)
        x.step()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            y.step()
        torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_checkpoints_and_masters():
    params = params_of(SHAPES[:5])
    opt = OPT.Muon(params, lr=1e-2)
    for k in range(2):
        set_grads(params, k)
        opt.step()
    saved, weights = copy.deepcopy(opt.state_dict()), [p.detach().clone() for p in params]
    again = params_of(SHAPES[:5], seed=8)
    with torch.no_grad():
        for p, w in zip(again, weights):
            p.copy_(w)
    other = OPT.Muon(again, lr=1.0)
    other.load_state_dict(saved)
    for k in range(2, 4):
        for p, o in ((params, opt), (again, other)):
            set_grads(p, k)
            o.step()
    assert all(torch.equal(p, q) for p, q in zip(params, again))
    assert all(torch.equal(opt.state[p]["master"], other.state[q]["master"]) for p, q in zip(params, again))
    # a parameter changed in place is taken over; one set to what it was keeps its master
    master = opt.state[params[1]]["master"].clone()
    with torch.no_grad():
        params[0].mul_(2)
        params[1].copy_(params[1].clone())
    set_grads(params, 9)
    e = Exact(opt, params[2:3])
    first, w0 = params[0].detach().double(), opt.param_groups[0]["lr"]
    opt.step()
    e.check(F32)
    moved = torch.linalg.matrix_norm(opt.state[params[0]]["master"].double() - first)
    assert moved < 0.2 * w0 * math.sqrt(max(params[0].shape)) * 1.3 * math.sqrt(min(params[0].shape)) + 0.2 * w0 * torch.linalg.matrix_norm(first)
    assert not torch.equal(opt.state[params[1]]["master"], master)
    with torch.no_grad():
        params[2].data.zero_()
    opt.sync_master()
    assert (opt.state[params[2]]["master"] == 0).all()


def test_many_small_and_large_matrices():
    """More shapes than a launch holds, lists longer than its CTAs."""
    shapes = [(16 + 3 * i, 40 + i) for i in range(20)] + [(130 + 5 * i, 140 + 3 * i) for i in range(20)] + [(200, 24, 16), (30, 16, 300), (3, 900, 60)]
    params = params_of(shapes)
    opt = OPT.Muon(params, lr=1e-2)
    set_grads(params, 1)
    e = Exact(opt, params)
    opt.step()
    e.check(F32)


def test_refusals():
    vector = torch.nn.Parameter(torch.zeros(4, dtype=BF, device="cuda"))
    matrix = torch.nn.Parameter(torch.zeros(4, 6, dtype=BF, device="cuda"))
    with pytest.raises(ValueError):
        OPT.Muon([vector])
    with pytest.raises(TypeError):
        OPT.Muon([torch.nn.Parameter(torch.zeros(4, 6, device="cuda"))])
    with pytest.raises(TypeError):
        OPT.Muon([torch.nn.Parameter(matrix.detach().t())])
    for bad in (dict(steps=0), dict(steps=40), dict(eps=0.0), dict(coefficients=(1.0, 2.0)), dict(coefficients=(math.nan, 1.0, 1.0))):
        with pytest.raises((ValueError, A.AdamWError)):
            OPT.Muon([matrix], **bad)
    opt = OPT.Muon([matrix])
    matrix.grad = None
    with pytest.raises(RuntimeError):
        opt.step()
    with pytest.raises(ValueError):
        opt.load_state_dict({"param_groups": [], "state": {}})
    shared = torch.zeros(2, 4, 6, dtype=F32, device="cuda")
    bf = lambda: torch.zeros(4, 6, dtype=BF, device="cuda")
    with pytest.raises(A.AdamWError):   # a master twice
        A.MuonPlan([bf(), bf()], [bf(), bf()], [shared[0], shared[1]], [shared[0], shared[0]])
    with pytest.raises(TypeError):
        A.MuonPlan([bf()], [bf().float()], [shared[0]], [shared[1]])
    with pytest.raises(ValueError):
        A.MuonPlan([], [], [], [])
    plan = A.MuonPlan([bf()], [bf()], [shared[0]], [shared[1]])
    with pytest.raises(TypeError):
        plan.step(torch.zeros(3, device="cuda"), torch.zeros(1, dtype=torch.int32, device="cuda"))
    plan.close()
    plan.close()
