"""Clipping lists of gradients by their global norm, against fp64 on the CPU.

Tolerances, from the arithmetic: the norm is an exact-to-2^-40 sum of fp32
group sums, each good to about its length times 2^-24 at worst (3e-6; the
groups' errors average out): 1e-6 relative; the coefficient one rounding more;
an element one product and one rounding to its type more (half an ulp)."""
import math

import pytest
import torch

from adamw_optimizer_step_sm_gb300 import adamw_sm as A
from adamw_optimizer_step_sm_gb300.optim import AnyPrecisionAdamW, GlobalClip, MasterWeightAdamW

pytestmark = pytest.mark.gpu

DEV = "cuda"
BF, HF, F = torch.bfloat16, torch.float16, torch.float32
ROUND = {t: torch.finfo(t).eps / 2 for t in (BF, HF, F)}   # half an ulp


def _list(numels, types, seed, scale=1e-2):
    g = torch.Generator().manual_seed(seed)
    return [(torch.randn(n, generator=g) * scale).to(t).to(DEV) for n, t in zip(numels, types)]


def _norm64(grads, kind):
    xs = [g.cpu().double() for g in grads if g.numel()]
    if not xs:
        return 0.0
    return float(torch.cat([x.reshape(-1) for x in xs]).norm()) if kind == "l2" else max(float(x.abs().max()) for x in xs)


def _check(plan, grads, outs, before, max_norm, kind):
    norm = _norm64(before, kind)
    r = plan.clip(max_norm, norm=kind)
    if norm > torch.finfo(F).max:   # finite, but not in the fp32 it is reported in
        assert float(r.norm) == math.inf
    else:
        assert abs(float(r.norm) - norm) <= 1e-6 * norm + 1e-45
    coef = min(1.0, max_norm / (norm + 1e-6))
    assert abs(float(r.coef) - coef) <= 1.2e-6 * coef + 2.0 ** -150 and int(r.nonfinite) == 0
    for b, o in zip(before, outs):
        want = b.cpu().double() * coef
        got = o.cpu().double()
        tiny = {BF: 1e-40, HF: 2.0 ** -24, F: 1e-44}[o.dtype]
        assert ((got - want).abs() <= (ROUND[o.dtype] + 2e-6) * want.abs() + tiny).all()


@pytest.mark.parametrize("kind", ["l2", "max"])
@pytest.mark.parametrize("src", [BF, HF, F])
@pytest.mark.parametrize("dst", [BF, HF, F, None])
def test_types(src, dst, kind):
    numels = [1, 7, 8, 9, 0, 255, 4096, 16384, 16385, 70001, 300007]
    grads = _list(numels, [src] * len(numels), 3)
    before = [g.clone() for g in grads]
    outs = grads if dst is None else [torch.full((n,), 9.0, dtype=dst, device=DEV) for n in numels]
    plan = A.ClipPlan(grads, None if dst is None else outs)
    norm = _norm64(before, kind)
    _check(plan, grads, outs, before, norm / 3, kind)
    if dst is not None:
        assert all(torch.equal(a, b) for a, b in zip(grads, before))
        _check(plan, grads, outs, before, norm * 3, kind)    # not clipped: converted
        if dst == src:
            assert all(torch.equal(a, b) for a, b in zip(outs, before))
        _check(plan, grads, outs, before, math.inf, kind)
    plan.close()


def test_mixed_types_odd_alignment_and_surroundings():
    """Tensors at every element offset of shared buffers: nothing beside them is touched."""
    sizes = [5, 64, 1000, 33, 16400, 2, 70003]
    for trial, types in enumerate([(BF, F, HF, BF, F, F, BF), (F, BF, BF, HF, HF, F, F)]):
        bufs, grads, outs, obufs = [], [], [], []
        for k, (n, t) in enumerate(zip(sizes, types)):
            g = torch.Generator().manual_seed(k + trial)
            b = (torch.randn(n + 20, generator=g)).to(t).to(DEV)
            o = torch.full((n + 20,), 7.0, dtype=types[-1 - k], device=DEV)
            bufs.append(b)
            obufs.append(o)
            grads.append(b[k + trial:k + trial + n])
            outs.append(o[(3 * k) % 8:(3 * k) % 8 + n])
        before = [g.clone() for g in grads]
        keep = [b.clone() for b in bufs]
        plan = A.ClipPlan(grads, outs)
        _check(plan, grads, outs, before, 1.0, "l2")
        assert all(torch.equal(a, b) for a, b in zip(bufs, keep))
        for k, (n, o) in enumerate(zip(sizes, obufs)):
            at = (3 * k) % 8
            assert (o[:at] == 7).all() and (o[at + n:] == 7).all()
        inplace = A.ClipPlan(grads)
        _check(inplace, grads, grads, before, 0.5, "max")
        for k, (n, b, w) in enumerate(zip(sizes, bufs, keep)):
            at = k + trial
            assert torch.equal(b[:at], w[:at]) and torch.equal(b[at + n:], w[at + n:])


@pytest.mark.parametrize("scale", [1e-30, 1e-22, 1e-15, 1e10, 1e25, 1e37])
def test_magnitudes_whose_squares_leave_fp32(scale):
    grads = _list([3, 5000, 40000], [F, F, BF], 5, scale)
    before = [g.clone() for g in grads]
    outs = [torch.empty_like(g) for g in grads]
    _check(A.ClipPlan(grads, outs), grads, outs, before, 1.0, "l2")
    # beside ordinary ones
    grads += _list([9000], [F], 6, 1.0)
    before = [g.clone() for g in grads]
    outs = [torch.empty_like(g) for g in grads]
    _check(A.ClipPlan(grads, outs), grads, outs, before, 0.1, "l2")


def test_zeros_signs_and_empty():
    for grads in ([torch.zeros(50000, dtype=BF, device=DEV)], [-torch.zeros(9, device=DEV)],
                  [torch.zeros(0, device=DEV)]):
        for kind in ("l2", "max"):
            r = A.ClipPlan(grads).clip(1.0, norm=kind)
            assert float(r.norm) == 0.0 and float(r.coef) == 1.0 and int(r.nonfinite) == 0


@pytest.mark.parametrize("value", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("where", [0, 12345, 69999])
@pytest.mark.parametrize("kind", ["l2", "max"])
def test_non_finite_passes_through(value, where, kind):
    for dt in (BF, F):
        grads = _list([100, 70000], [F, dt], 8, 10.0)
        grads[1][where] = value
        before = [g.clone() for g in grads]
        outs = [torch.empty_like(g) for g in grads]
        r = A.ClipPlan(grads, outs).clip(1.0, norm=kind)
        assert int(r.nonfinite) == 1 and float(r.coef) == 1.0 and not math.isfinite(float(r.norm))
        for a, b in zip(outs, before):
            assert torch.equal(a.nan_to_num(nan=3.0), b.nan_to_num(nan=3.0))


def test_repeats_bit_for_bit_and_norm_only():
    grads = _list([1 << 20, 77777, 3], [F, BF, HF], 9)
    outs = [torch.empty_like(g) for g in grads]
    plan, only = A.ClipPlan(grads, outs), A.ClipPlan(grads, norm_only=True)
    first = None
    for _ in range(5):
        r = plan.clip(0.5)
        now = [float(r.norm), float(r.coef)] + [o.clone() for o in outs]
        if first is not None:
            assert now[:2] == first[:2] and all(torch.equal(a, b) for a, b in zip(now[2:], first[2:]))
        first = now
    before = [g.clone() for g in grads]
    r = only.clip(0.5)
    assert float(r.norm) == first[0] and all(torch.equal(a, b) for a, b in zip(grads, before))


def test_longer_than_32_bits():
    n = (1 << 31) + 1003
    g = torch.zeros(n, dtype=BF, device=DEV)
    g[-5:] = 3.0
    g[0] = 4.0
    r = A.ClipPlan([g]).clip(1.0)
    assert abs(float(r.norm) - math.sqrt(61.0)) < 1e-5
    assert abs(float(g[-1]) - 3 / math.sqrt(61.0)) < 2e-3 and float(g[n // 2]) == 0.0
    del g
    torch.cuda.empty_cache()


def test_capture_and_side_stream():
    grads = _list([100000, 50], [F, BF], 10)
    outs = [torch.empty_like(g) for g in grads]
    plan = A.ClipPlan(grads, outs)
    plan.clip(0.1)
    want = [o.clone() for o in outs]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    for o in outs:
        o.zero_()
    torch.cuda.synchronize()
    plan.clip(0.1, stream=s)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        plan.clip(0.1)
    for _ in range(2):
        for o in outs:
            o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))


def test_refusals():
    g = torch.zeros(64, device=DEV)
    for bad, exc in [
        (lambda: A.ClipPlan([]), ValueError),
        (lambda: A.ClipPlan([g], [g, g]), ValueError),
        (lambda: A.ClipPlan([g], norm_only=True, outs=[g]), ValueError),
        (lambda: A.ClipPlan([g.cpu()]), TypeError),
        (lambda: A.ClipPlan([g.double()]), TypeError),
        (lambda: A.ClipPlan([g[::2]]), TypeError),
        (lambda: A.ClipPlan([g], [g[:32]]), TypeError),
        (lambda: A.ClipPlan([g[:40]], [g[8:48]]), A.AdamWError),
        (lambda: A.ClipPlan([g[:32]], [g.view(BF)[:32]]), A.AdamWError),
        (lambda: A.ClipPlan([g]).clip(0.0), ValueError),
        (lambda: A.ClipPlan([g]).clip(float("nan")), ValueError),
        (lambda: A.ClipPlan([g]).clip(1.0, norm="l1"), ValueError),
    ]:
        with pytest.raises(exc):
            bad()


def test_global_clip_over_groups_and_optimizers():
    """One norm over two groups of one optimizer and a second optimizer, then
    their steps: as torch.nn.utils.clip_grad_norm_ over all parameters."""
    g = torch.Generator().manual_seed(1)
    make = lambda *s: torch.nn.Parameter((torch.randn(*s, generator=g) * 0.02).to(BF).to(DEV))
    params = [make(300, 40), make(40), make(1000, 33)]
    a = AnyPrecisionAdamW([{"params": [params[0]]}, {"params": [params[1]], "weight_decay": 0.0}], lr=1e-3)
    b = MasterWeightAdamW([params[2]], lr=1e-3)
    clip = GlobalClip(a, b)
    for step in range(3):
        a.zero_grad()
        b.zero_grad()
        for k, p in enumerate(params):
            new = torch.randn(p.shape, generator=g).to(BF).to(DEV)
            if step == 1 and k == 1:
                p.grad = new.clone()      # a gradient of the caller's own
            else:
                p.grad.copy_(new)
        before = [p.grad.clone() for p in params]
        norm = _norm64(before, "l2")
        r = clip(0.5)
        assert abs(float(r.norm) - norm) <= 1e-6 * norm
        for p, w in zip(params, before):
            want = w.cpu().double() * (0.5 / (norm + 1e-6))
            assert ((p.grad.cpu().double() - want).abs() <= (ROUND[BF] + 2e-6) * want.abs() + 1e-40).all()
        old = [p.detach().clone() for p in params]
        a.step()
        b.step()
        assert all(not torch.equal(p.detach(), o) for p, o in zip(params, old))
    params[0].grad = None
    with pytest.raises(RuntimeError):
        clip(1.0)
