"""The fine-tuning operators on the GPU against their definitions in 64 bits,
written out here on the CPU.

Tolerances, set from the arithmetic before the first run (u = 2^-24 is fp32's
rounding unit):
  * log-probabilities, entropies: the exponentials and sums of a row are good
    to a few u relative, the final subtraction rounds at the magnitude of the
    row's largest (x - m): 4e-6 absolute for |x| up to about 30, 2e-6 relative.
  * gradients in fp32: a probability's relative error is u times the size of
    its exponent (at most about 30) plus a few u: 1e-5 relative to the row's
    largest entry of |d|.  In bf16 / fp16 one rounding more: half an ulp
    (2^-8, 2^-11) of the value itself, plus fp16's subnormal spacing 2^-25.
  * losses, statistics: sums are error-free, terms good to a few u: 2e-6
    relative to the mean of the terms' magnitudes.
"""
import math

import pytest
import torch

from adamw_optimizer_step_sm_gb300 import adamw_sm as A
from adamw_optimizer_step_sm_gb300 import losses as L

pytestmark = pytest.mark.gpu

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
ROUND = {k: torch.finfo(v).eps / 2 if k != "fp32" else 0.0 for k, v in TYPES.items()}   # half an ulp
INF = float("inf")


def _gen(seed):
    return torch.Generator(device="cpu").manual_seed(seed)


# --------------------------------------------------- definitions, in 64 bits

def _rows64(logits, targets, scale, ignore=-100):
    """(logp, entropy, p, log p) of rows [n, v] in fp64 on the CPU; rows
    without a distribution: logp -inf, entropy 0, p 0."""
    x = logits.detach().cpu().double() * scale
    t = targets.cpu()
    m = x.amax(1, keepdim=True)
    m = torch.where(torch.isinf(m) & (m < 0), torch.zeros_like(m), m)
    s = torch.exp(x - m).sum(1, keepdim=True)
    empty = s[:, 0] == 0
    lp = x - m - torch.log(s)
    p = torch.where(empty[:, None], torch.zeros_like(lp), torch.exp(lp))
    ent = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(1)
    logp = lp.gather(1, t.clamp(0, x.shape[1] - 1)[:, None])[:, 0]
    logp = torch.where(empty, torch.full_like(logp, -INF), logp)
    off = t == ignore
    logp[off], ent[off] = 0.0, 0.0
    return logp, ent, p, lp, off, empty


def _grad64(r64, targets, dl, dh, scale):
    logp, ent, p, lp, off, empty = r64
    t = targets.cpu()
    g = -dl[:, None] * p
    g[torch.arange(g.shape[0]), t.clamp(0, g.shape[1] - 1)] += dl
    if dh is not None:
        g -= dh[:, None] * torch.where(p > 0, p * (lp + ent[:, None]), torch.zeros_like(p))
    g *= scale
    g[off | empty] = 0.0
    return g


def _logits(n, v, dtype, seed, masked=0):
    g = _gen(seed)
    x = (torch.randn(n, v, generator=g) * 3).to(TYPES[dtype])
    t = torch.randint(0, v, (n,), generator=g)
    if masked:
        x[:, torch.randperm(v, generator=g)[:masked]] = -INF
    return x, t


def _close_logp(got, want):
    got = got.cpu().double().reshape(-1)
    both = torch.isfinite(want)
    assert torch.equal(torch.isfinite(got), both)
    assert torch.equal(got[~both].nan_to_num(nan=7.0), want[~both].nan_to_num(nan=7.0))
    bad = (got[both] - want[both]).abs() > 4e-6 + 2e-6 * want[both].abs()
    assert not bad.any(), (got[both] - want[both]).abs().max()


def _close_grad(got, want, dtype):
    got = got.cpu().double().reshape(want.shape)
    top = want.abs().amax(1, keepdim=True)
    tol = 1e-5 * top + ROUND[dtype] * want.abs() + (2.0 ** -25 if dtype == "fp16" else 1e-38)
    bad = (got - want).abs() > tol
    assert not bad.any(), ((got - want).abs() / tol).max()


# ------------------------------------------------------- log-probabilities

SHAPES = [(1, 1), (3, 2), (5, 7), (9, 31), (2, 33), (70, 257), (11, 1000), (8, 1024), (7, 1025), (6, 4096),
          (5, 4097), (4, 8192), (3, 8193), (3, 50257), (2, 50272), (1, 131072)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("n,v", SHAPES)
def test_logprob_and_gradient(n, v, dtype):
    x, t = _logits(n, v, dtype, n * 1000 + v, masked=v // 9)
    if n > 2:
        t[1] = -100
    scale = 1 / 0.7
    xd, td = x.to(DEV), t.to(DEV)
    r = L.token_logprob(xd, td, temperature=0.7, entropy=True)
    want = _rows64(x, t, scale)
    _close_logp(r.logp, want[0])
    _close_logp(r.entropy, want[1])
    plain = L.token_logprob(xd, td, temperature=0.7)
    assert plain.entropy is None
    _close_logp(plain.logp, want[0])
    g = _gen(v)
    dl, dh = torch.randn(n, generator=g), 0.3 * torch.randn(n, generator=g)
    d = L.token_logprob_backward(xd, td, r, dl.to(DEV), dh.to(DEV), temperature=0.7)
    _close_grad(d, _grad64(want, t, dl.double(), dh.double(), scale), dtype)
    d = L.token_logprob_backward(xd, td, r, dl.to(DEV), temperature=0.7)
    _close_grad(d, _grad64(want, t, dl.double(), None, scale), dtype)
    # in place, the same bits
    e = xd.clone()
    L.token_logprob_backward(e, td, r, dl.to(DEV), temperature=0.7, out=e)
    assert torch.equal(e, d)


@pytest.mark.parametrize("v", [50, 64, 1501, 5003, 9000])
@pytest.mark.parametrize("view", ["shift", "tail", "pad", "batch_second", "odd_start"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_logprob_strides(view, v, dtype):
    b, s = 3, 5
    g = _gen(v)
    base = (torch.randn(b * (s + 1) * (v + 3) + 1, generator=g) * 3).to(TYPES[dtype]).to(DEV)
    if view == "shift":
        x = base[:b * (s + 1) * v].view(b, s + 1, v)[:, :-1]
    elif view == "tail":
        x = base[:b * (s + 1) * v].view(b, s + 1, v)[:, 1:]
    elif view == "pad":
        x = base[:b * s * (v + 3)].view(b, s, v + 3)[:, :, :v]
    elif view == "batch_second":
        x = base[:b * s * v].view(s, b, v).transpose(0, 1)
    else:
        x = base[1:1 + b * s * v].view(b, s, v)
    t = torch.randint(0, v, (b, s), generator=g).to(DEV)
    flat = x.reshape(-1, v)
    want = _rows64(flat, t.reshape(-1), 1.0)
    r = L.token_logprob(x, t, entropy=True)
    _close_logp(r.logp, want[0])
    _close_logp(r.entropy, want[1])
    dl = torch.randn(b, s, generator=g)
    before = base.clone()
    d = L.token_logprob_backward(x, t, r, dl.to(DEV))
    want_d = _grad64(want, t.reshape(-1), dl.reshape(-1).double(), None, 1.0)
    _close_grad(d.reshape(-1, v), want_d, dtype)
    # into a contiguous tensor of the caller's, whatever its rows' alignment
    out = torch.empty(b * s * v + 1, dtype=x.dtype, device=DEV)[1:].view(b, s, v)
    L.token_logprob_backward(x, t, r, dl.to(DEV), out=out)
    assert torch.equal(out, d)
    assert torch.equal(base, before)
    # in place writes the view's rows and nothing beside them
    L.token_logprob_backward(x, t, r, dl.to(DEV), out=x)
    assert torch.equal(x, d)
    changed = base != before
    inside = torch.zeros_like(base, dtype=torch.bool)
    inside.as_strided(x.shape, x.stride(), x.storage_offset()).fill_(True)
    assert not (changed & ~inside).any()


@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("v", [40, 3001])
def test_logprob_empty_rows_masks_and_non_finite(v, dtype):
    low = torch.finfo(TYPES[dtype]).min
    x, t = _logits(9, v, dtype, 5)
    x[0] = -INF                       # no distribution
    x[1] = low                        # masked by the type's lowest value throughout: uniform
    x[2, :] = -INF
    x[2, 3] = 1.0                     # one token left, and it is the target
    t[2] = 3
    x[3, 5] = -INF                    # the target itself is masked
    t[3] = 5
    x[4, 7] = float("nan")
    x[5, 7] = INF
    x[6, 1:] = low
    t[7] = v                          # outside the vocabulary
    t[8] = -5
    xd, td = x.to(DEV), t.to(DEV)
    r = L.token_logprob(xd, td, entropy=True)
    want = _rows64(x, t, 1.0)
    lp, h = r.logp.cpu().double(), r.entropy.cpu().double()
    assert lp[0] == -INF and h[0] == 0.0
    assert abs(lp[1] + math.log(v)) < 1e-5 and abs(h[1] - math.log(v)) < 1e-5
    assert lp[2] == 0.0 and h[2] == 0.0
    assert lp[3] == -INF and abs(h[3] - want[1][3]) < 1e-5
    assert torch.isnan(lp[[4, 5, 7, 8]]).all() and torch.isnan(h[[4, 5, 7, 8]]).all()
    assert abs(lp[6] - want[0][6]) < 1e-5 * max(1.0, abs(float(want[0][6]))) and abs(h[6]) < 1e-6
    dl, dh = torch.ones(9, device=DEV), torch.full((9,), 0.5, device=DEV)
    for entropy in (None, dh):
        d = L.token_logprob_backward(xd, td, r, dl, entropy).cpu().double()
        assert (d[0] == 0).all()
        assert torch.isnan(d[[4, 7, 8]]).all() and torch.isnan(d[5]).any()
        good = [1, 2, 3, 6]
        w = _grad64(want, t, dl.cpu().double(), None if entropy is None else dh.cpu().double(), 1.0)
        _close_grad(d[good], w[good], dtype)
        assert torch.isfinite(d[good]).all()


def test_logprob_nothing_to_do():
    x = torch.zeros(0, 100, dtype=torch.bfloat16, device=DEV)
    r = L.token_logprob(x, torch.zeros(0, dtype=torch.int64, device=DEV), entropy=True)
    assert r.logp.shape == (0,) and r.entropy.shape == (0,)
    assert L.token_logprob_backward(x, torch.zeros(0, dtype=torch.int64, device=DEV), r, r.logp).shape == (0, 100)
    one = L.token_logprob(torch.zeros(7, device=DEV), torch.tensor(2, device=DEV), entropy=True)
    assert one.logp.shape == () and abs(float(one.logp) + math.log(7)) < 1e-6
    # every row ignored: nothing is read, everything is written
    x = torch.full((6, 3000), float("nan"), device=DEV)
    t = torch.full((6,), -100, device=DEV)
    r = L.token_logprob(x, t, entropy=True)
    assert (r.logp == 0).all() and (r.entropy == 0).all()
    assert (L.token_logprob_backward(x, t, r, torch.ones(6, device=DEV)) == 0).all()


def test_logprob_offsets_past_32_bits():
    """Rows whose elements start past 2^32 bytes and 2^31 elements."""
    v, n = 65536, 33000   # 2.16e9 bf16 elements
    x = torch.zeros(n, v, dtype=torch.bfloat16, device=DEV)
    g = _gen(3)
    last = (torch.randn(4, v, generator=g) * 3).bfloat16()
    x[-4:] = last.to(DEV)
    t = torch.randint(0, v, (n,), generator=g)
    r = L.token_logprob(x, t.to(DEV), entropy=True)
    want = _rows64(last, t[-4:], 1.0)
    _close_logp(r.logp[-4:], want[0])
    assert (r.logp[:-4] + math.log(v)).abs().max() < 1e-5
    dl = torch.ones(n, device=DEV)
    L.token_logprob_backward(x, t.to(DEV), r, dl, out=x)
    _close_grad(x[-4:], _grad64(want, t[-4:], torch.ones(4).double(), None, 1.0), "bf16")
    del x
    torch.cuda.empty_cache()


@pytest.mark.parametrize("v", [17, 2050])
def test_logprob_gradient_by_differences_and_autograd(v):
    x, t = _logits(4, v, "fp32", 11)
    t[2] = -100
    leaf = x.to(DEV).requires_grad_(True)
    r = L.token_logprob(leaf, t.to(DEV), temperature=1.3, entropy=True)
    wl, wh = torch.tensor([1.0, -2.0, 0.5, 0.7]), torch.tensor([0.3, 0.2, -1.0, 0.1])
    ((r.logp * wl.to(DEV)).sum() + (r.entropy * wh.to(DEV)).sum()).backward()
    got = leaf.grad.cpu().double()

    def value(z):
        a = _rows64(z, t, 1 / 1.3)
        return (a[0] * wl.double()).sum() + (a[1] * wh.double()).sum()
    z, eps = x.double(), 1e-5
    for i, j in [(0, 0), (0, int(t[0])), (1, 3), (1, int(t[1])), (2, 5), (3, v - 1), (3, int(t[3]))]:
        up, down = z.clone(), z.clone()
        up[i, j] += eps
        down[i, j] -= eps
        diff = float(value(up) - value(down)) / (2 * eps)
        assert abs(float(got[i, j]) - diff) < 1e-5 + 1e-5 * abs(diff), (i, j)
    assert (got[2] == 0).all()
    # only one of the two outputs used
    leaf.grad = None
    L.token_logprob(leaf, t.to(DEV), entropy=True).entropy.sum().backward()
    assert torch.isfinite(leaf.grad).all() and leaf.grad.abs().max() > 0
    with torch.no_grad():
        assert not L.token_logprob(leaf, t.to(DEV)).logp.requires_grad


# -------------------------------------------------------------- policy loss

def _policy64(logp, old, adv, ref, ent, on, starts, o):
    """stats, counts, d_logp, d_entropy by loops over sequences, in fp64."""
    n = logp.numel()
    rows = len(starts) - 1
    spans = [torch.arange(starts[i], starts[i + 1]) for i in range(rows)]
    used = [s[on[s]] for s in spans]
    filled = sum(1 for s in used if len(s))
    tokens = sum(len(s) for s in used)
    w = torch.zeros(n, dtype=torch.float64)
    A_ = torch.zeros(n, dtype=torch.float64)
    for i, s in enumerate(used):
        if len(s):
            w[s] = {"token": 1 / max(tokens, 1), "sequence": 1 / (len(s) * max(filled, 1)),
                    "fixed": 1 / o["divisor"]}[o["reduce"]]
            A_[s] = adv.double()[s] if adv.numel() == n and o["per_token"] else adv.double()[i]
    use = w > 0
    z = lambda v: torch.where(use, v.double(), torch.zeros(n, dtype=torch.float64))
    lp = z(logp).requires_grad_(True)
    d = lp - z(old)
    r = torch.exp(d)
    surrogate = torch.minimum(r * A_, torch.clamp(r, 1 - o["clip_low"], 1 + o["clip_high"]) * A_)
    if o["dual"]:
        surrogate = torch.where(A_ < 0, torch.maximum(surrogate, o["dual"] * A_), surrogate)
    kl = torch.zeros(n, dtype=torch.float64)
    if ref is not None:
        k = lp - z(ref)
        kl = {"k1": k, "k2": k * k / 2, "k3": torch.exp(-k) - 1 + k}[o["kl"]]
    h = z(ent) if ent is not None else torch.zeros(n, dtype=torch.float64)
    parts = [(-surrogate * w).sum(), (kl * w).sum(), (h * w).sum()]
    loss = parts[0] + o["kl_coef"] * parts[1] - o["entropy_coef"] * parts[2]
    if n:
        loss.backward()
    up, down = A_ > 0, A_ < 0
    off = (up & (r > 1 + o["clip_high"])) | (down & (r < 1 - o["clip_low"]))
    if o["dual"]:
        off = off | (down & (r > o["dual"]))
    stats = [loss, *parts, (off.double() * w).sum(), ((r - 1 - d) * w).sum()]
    scale = [(v.abs() * w).sum() for v in (surrogate, kl, h, off.double(), r - 1 - d)]
    grad = lp.grad if n else torch.zeros(0, dtype=torch.float64)
    return torch.stack([s.detach() for s in stats]), torch.stack(scale).detach(), [tokens, filled], grad, \
        -o["entropy_coef"] * w


def _policy_inputs(n, rows, seed, packed, share=0.3):
    g = _gen(seed)
    logp = -torch.rand(n, generator=g).pow(3) * 8
    old = logp - torch.randn(n, generator=g) * 0.25
    # no token within rounding of a clip edge (log 0.8, log 1.28, log 3)
    d = logp - old
    for edge in (math.log(0.8), math.log(1.28), math.log(3.0)):
        old = torch.where((d - edge).abs() < 1e-4, old - 1e-3, old)
    ref = logp + torch.randn(n, generator=g) * 0.3
    ent = torch.rand(n, generator=g) * 4
    on = torch.rand(n, generator=g) >= share
    if packed:
        cuts = sorted(int(c) for c in torch.randint(0, n + 1, (rows - 1,), generator=g))
        starts = [0, *cuts, n]
    else:
        starts = [i * (n // rows) for i in range(rows + 1)]
    return logp, old, ref, ent, on, starts, g


def _check_policy(got, want, with_entropy, grad_scale=1.0):
    stats, sizes, counts, grad, dh = want
    s = got.stats.cpu().double()
    assert got.counts.tolist() == counts
    tol = 2e-6 * sizes + 1e-12
    assert ((s[1:] - stats[1:]).abs() <= tol).all(), (s, stats)
    assert abs(float(s[0] - stats[0])) <= 4e-6 * float(sizes[:3].sum()) + 1e-12
    g = got.d_logp.cpu().double().reshape(-1)
    assert ((g - grad * grad_scale).abs() <= 4e-6 * (grad * grad_scale).abs() + 4e-7 * grad.abs().max() * abs(grad_scale)).all()
    if with_entropy:
        h = got.d_entropy.cpu().double().reshape(-1)
        assert ((h - dh * grad_scale).abs() <= 4e-7 * (dh * grad_scale).abs()).all()


@pytest.mark.parametrize("reduce", ["token", "sequence", "fixed"])
@pytest.mark.parametrize("n,rows,packed", [(1, 1, False), (1, 3, True), (6, 6, False), (40, 5, False),
                                           (257, 7, True), (5000, 1, False), (5003, 900, True),
                                           (70000, 10, True), (196608, 4096, False)])
def test_policy_loss(n, rows, packed, reduce):
    logp, old, ref, ent, on, starts, g = _policy_inputs(n, rows, n + rows, packed)
    kl = {"token": "k3", "sequence": "k2", "fixed": "k1"}[reduce]
    per_token = reduce != "sequence"
    adv = torch.randn(n if per_token else rows, generator=g) + 0.2
    o = dict(clip_low=0.2, clip_high=0.28, dual=3.0 if reduce == "token" else 0.0, kl=kl, kl_coef=0.05,
             entropy_coef=0.01, reduce=reduce, divisor=float(n), per_token=per_token)
    want = _policy64(logp, old, adv, ref, ent, on, starts, o)
    shape = (n,) if packed or rows == 1 else (rows, n // rows)
    put = lambda v: v.to(DEV).view(shape)
    off = torch.tensor(starts, device=DEV) if packed else None
    # garbage where the mask is off
    bad = torch.where(on, 0.0, float("nan"))
    args = dict(ref_logp=put(ref + bad), entropy=put(ent + bad), mask=put(on), offsets=off, clip_low=0.2,
                clip_high=0.28, dual_clip=o["dual"], kl=kl, kl_coef=0.05, entropy_coef=0.01, reduce=reduce,
                divisor=float(n), grad_scale=0.25)
    a = put(adv + bad) if per_token else adv.to(DEV)
    got = L.policy_loss(put(logp + bad), put(old + bad), a, **args)
    _check_policy(got, want, True, 0.25)
    again = L.policy_loss(put(logp + bad), put(old + bad), a, **args)
    assert all(torch.equal(p, q) for p, q in zip(got, again))
    # without the optional parts
    o.update(kl_coef=0.0, entropy_coef=0.0, dual=0.0)
    on1 = torch.ones(n, dtype=torch.bool)
    want = _policy64(logp, old, adv, None, None, on1, starts, o)
    got = L.policy_loss(put(logp), put(old), put(adv) if per_token else adv.to(DEV), offsets=off, clip_low=0.2,
                        clip_high=0.28, reduce=reduce, divisor=float(n))
    assert got.d_entropy is None
    _check_policy(got, want, False)


@pytest.mark.parametrize("n,rows", [(40000, 15000), (40000, 3000), (3000, 2500), (17000, 9000)])
@pytest.mark.parametrize("reduce", ["token", "sequence"])
def test_policy_loss_many_short_sequences(n, rows, reduce):
    """More sequences than lanes among a warp's tokens, empty ones, and tokens
    before the first and after the last."""
    logp, old, ref, ent, on, starts, g = _policy_inputs(n, rows, n - rows, True)
    starts = [min(max(s, 100), n - 50) for s in starts]
    adv = torch.randn(rows, generator=g) + 0.2
    o = dict(clip_low=0.2, clip_high=0.28, dual=0.0, kl="k3", kl_coef=0.05, entropy_coef=0.01, reduce=reduce,
             divisor=1.0, per_token=False)
    want = _policy64(logp, old, adv, ref, ent, on, starts, o)
    d = lambda v: v.to(DEV)
    got = L.policy_loss(d(logp), d(old), d(adv), ref_logp=d(ref), entropy=d(ent), mask=d(on),
                        offsets=torch.tensor(starts, device=DEV), clip_low=0.2, clip_high=0.28, kl_coef=0.05,
                        entropy_coef=0.01, reduce=reduce)
    _check_policy(got, want, True)
    assert (got.d_logp[:100] == 0).all() and (got.d_logp[n - 50:] == 0).all()
    # targets in place of the mask: the fused form counts the same tokens
    x = torch.randn(n, 8, generator=g).to(DEV)
    t = torch.where(on, torch.randint(0, 8, (n,), generator=g), -100).to(DEV)
    lp = L.token_logprob(x, t)
    r = L.policy_loss_logits(x, t, d(old), d(adv), offsets=torch.tensor(starts, device=DEV), reduce=reduce)
    p = L.policy_loss(lp.logp, d(old), d(adv), mask=d(on), offsets=torch.tensor(starts, device=DEV), reduce=reduce)
    assert torch.equal(r.counts, got.counts) and torch.equal(r.logp, lp.logp)
    assert (r.stats - p.stats).abs().max() <= 1e-6 * p.stats.abs().max() + 1e-7
    back = L.token_logprob_backward(x, t, lp, p.d_logp)
    assert (r.d_logits - back).abs().max() <= 1e-6 * back.abs().max()


@pytest.mark.parametrize("n", [1000, 40000])
def test_losses_replayed_and_on_two_streams(n):
    """Counts, tickets and sums start afresh in every replay, and calls on two
    streams do not share them."""
    logp, old, ref, ent, on, starts, g = _policy_inputs(n, 50, n, False)
    args = [v.to(DEV).view(50, n // 50) for v in (logp, old)]
    adv = [torch.randn(50, generator=g).to(DEV) for _ in range(2)]
    mask = on.to(DEV).view(50, -1)
    call = lambda k: (L.policy_loss(*args, adv[k], mask=mask, reduce="sequence"), L.preference_loss(args[k], args[1 - k]))
    flat = lambda rs: [v for r in rs for v in r if v is not None]
    want = [[v.clone() for v in flat(call(k))] for k in range(2)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(10):
        for k, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[k].append(flat(call(k)))
    torch.cuda.synchronize()
    for k in range(2):
        for r in got[k]:
            assert all(torch.equal(a, b) for a, b in zip(r, want[k]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = flat(call(0))
    for _ in range(3):
        for v in r:
            v.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(r, want[0]))


def test_policy_loss_edges():
    t = lambda *v: torch.tensor(v, device=DEV)
    # nothing counts: zeros, no division by zero
    z = torch.zeros(2, 3, device=DEV)
    for reduce in ("token", "sequence", "fixed"):
        r = L.policy_loss(z, z, t(1.0, 1.0), mask=torch.zeros(2, 3, dtype=torch.bool, device=DEV), reduce=reduce)
        assert (r.stats == 0).all() and r.counts.tolist() == [0, 0] and (r.d_logp == 0).all()
    r = L.policy_loss(torch.zeros(0, device=DEV), torch.zeros(0, device=DEV), torch.zeros(0, device=DEV))
    assert (r.stats == 0).all() and r.counts.tolist() == [0, 0]
    # tokens before the first and after the last offset count for nothing
    off = t(2, 4, 4, 5)
    lp = t(9.0, 9.0, 0.1, 0.2, 0.3, 9.0, 9.0)
    r = L.policy_loss(lp, torch.zeros(7, device=DEV), t(1.0, 1.0, 1.0), offsets=off, clip_high=1.0, reduce="sequence")
    assert r.counts.tolist() == [3, 2]
    assert r.d_logp[[0, 1, 5, 6]].abs().max() == 0
    e = torch.exp(lp.double())
    want = -(0.5 * (e[2] + e[3]) / 2 + 0.5 * e[4])
    assert abs(float(r.stats[0]) - float(want)) < 1e-6
    # a token the policy no longer produces (logp -inf): ratio 0, no gradient
    r = L.policy_loss(t(-INF, 0.0), t(-1.0, 0.0), t(1.0), clip_low=0.2)
    assert r.d_logp.tolist() == [0.0, -0.5]
    # a NaN that counts is seen; masked it is not
    nan = float("nan")
    r = L.policy_loss(t(nan, 0.0), t(0.0, 0.0), t(1.0))
    assert torch.isnan(r.stats[0]) and torch.isnan(r.d_logp[0]) and r.d_logp[1] == -0.5
    # exactly on the edge the unclipped branch holds; above it none
    h = torch.tensor(math.log1p(0.25), dtype=torch.float32)
    up = torch.nextafter(h, torch.tensor(1.0))
    r = L.policy_loss(torch.stack([h, up]).to(DEV), torch.zeros(2, device=DEV), t(1.0), clip_high=0.25)
    assert r.d_logp[0] < 0 and r.d_logp[1] == 0


# ------------------------------------------------------ policy loss from logits

@pytest.mark.parametrize("dtype", ["bf16", "fp16", "fp32"])
@pytest.mark.parametrize("b,s,v", [(1, 1, 5), (2, 3, 60), (3, 40, 1000), (2, 9, 1025), (2, 3, 4096), (2, 3, 4099),
                                   (3, 7, 7001), (2, 5, 50257), (40, 13, 3000), (1, 2, 200000)])
def test_policy_loss_logits(b, s, v, dtype):
    n = b * s
    g = _gen(v + n)
    x = (torch.randn(b, s + 1, v, generator=g) * 2).to(TYPES[dtype])
    t = torch.randint(0, v, (b, s), generator=g)
    if n > 3:
        t[0, 1] = -100
        t[-1, 0] = -100
    scale = 1 / 1.2
    flat = x[:, :-1].reshape(-1, v)
    r64 = _rows64(flat, t.reshape(-1), scale)
    logp = r64[0]
    d = torch.randn(n, generator=g) * 0.2
    for edge in (math.log(0.8), math.log(1.2)):   # an edge is decided by a logp's last bit
        d = torch.where((d - edge).abs() < 1e-3, d + 4e-3, d)
    old = (logp - d).float()
    ref = (logp + torch.randn(n, generator=g) * 0.3).float()
    adv = torch.randn(b, generator=g) + 0.3
    on = t.reshape(-1) != -100
    for reduce, ec in (("token", 0.0), ("sequence", 0.02)):
        o = dict(clip_low=0.2, clip_high=0.2, dual=0.0, kl="k3", kl_coef=0.1, entropy_coef=ec, reduce=reduce,
                 divisor=1.0, per_token=False)
        want = _policy64(logp, old, adv, ref, r64[1] if ec else None, on, [i * s for i in range(b + 1)], o)
        xd = x.to(DEV)
        got = L.policy_loss_logits(xd[:, :-1], t.to(DEV), old.view(b, s).to(DEV), adv.to(DEV),
                                   ref_logp=ref.view(b, s).to(DEV), temperature=1.2, kl_coef=0.1,
                                   entropy_coef=ec, reduce=reduce)
        _close_logp(got.logp, logp)
        assert got.counts.tolist() == want[2]
        # a log-probability is good to 4e-6 + 2e-6 |x|: so are the ratios, relative
        err = 4e-6 + 2e-6 * float(logp[torch.isfinite(logp)].abs().max())
        sizes = want[1]
        assert ((got.stats.cpu().double()[1:] - want[0][1:]).abs() <= 4 * err * (sizes + 1)).all()
        wd = _grad64(r64, t.reshape(-1), want[3], want[4] if ec else None, scale)
        top = wd.abs().amax(1, keepdim=True)
        tol = (1e-5 + 4 * err) * (top + 1.0 / n) + ROUND[dtype] * wd.abs() + (2.0 ** -25 if dtype == "fp16" else 1e-38)
        dd = got.d_logits.cpu().double().reshape(-1, v)
        assert ((dd - wd).abs() <= tol).all(), ((dd - wd).abs() / tol).max()
        assert (dd[~on] == 0).all()
        # over the logits themselves, and twice: the same bits
        before = xd.clone()
        again = L.policy_loss_logits(xd[:, :-1], t.to(DEV), old.view(b, s).to(DEV), adv.to(DEV),
                                     ref_logp=ref.view(b, s).to(DEV), temperature=1.2, kl_coef=0.1,
                                     entropy_coef=ec, reduce=reduce, out=xd[:, :-1])
        assert torch.equal(again.d_logits, got.d_logits) and torch.equal(again.stats, got.stats)
        assert torch.equal(xd[:, -1], before[:, -1])


def test_policy_loss_logits_odd_rows():
    """No distribution, a target outside the vocabulary, tokens outside every sequence."""
    for v in (33, 3000):
        x = torch.randn(6, v, generator=_gen(2)).to(DEV)
        x[1] = -INF
        t = torch.tensor([0, 1, 2, v, -100, 3], device=DEV)
        off = torch.tensor([0, 2, 5], device=DEV)   # the last token is in no sequence
        zero = torch.zeros(6, device=DEV)
        r = L.policy_loss_logits(x, t, zero, torch.ones(2, device=DEV), offsets=off, entropy=True)
        assert r.counts.tolist() == [4, 2]
        assert r.logp[1] == -INF and torch.isnan(r.logp[3]) and r.logp[4] == 0
        d = r.d_logits
        assert (d[1] == 0).all() and torch.isnan(d[3]).all() and (d[4] == 0).all() and (d[5] == 0).all()
        assert torch.isfinite(d[0]).all() and d[0].abs().max() > 0
    r = L.policy_loss_logits(torch.zeros(0, 9, device=DEV), torch.zeros(0, dtype=torch.int64, device=DEV),
                             torch.zeros(0, device=DEV), torch.zeros(0, device=DEV))
    assert r.d_logits.shape == (0, 9) and (r.stats == 0).all()


@pytest.mark.parametrize("dtype,v", [("fp32", 450001), ("bf16", 900004)])
def test_policy_loss_logits_rows_too_long_for_a_cluster(dtype, v):
    x, t = _logits(3, v, dtype, 4)
    r64 = _rows64(x, t, 1.0)
    old = (r64[0] - torch.tensor([0.05, 0.3, -0.1])).float()
    o = dict(clip_low=0.2, clip_high=0.2, dual=0.0, kl="k3", kl_coef=0.0, entropy_coef=0.1, reduce="token",
             divisor=1.0, per_token=True)
    adv = torch.tensor([1.0, 0.5, -2.0])
    want = _policy64(r64[0], old, adv, None, r64[1], torch.ones(3, dtype=torch.bool), [0, 3], o)
    r = L.policy_loss_logits(x.to(DEV), t.to(DEV), old.to(DEV), adv.to(DEV), entropy_coef=0.1)
    _close_logp(r.logp, r64[0])
    wd = _grad64(r64, t, want[3], want[4], 1.0)
    got = r.d_logits.cpu().double()
    tol = 2e-4 * wd.abs().amax(1, keepdim=True) + ROUND[dtype] * wd.abs() + 1e-38
    assert ((got - wd).abs() <= tol).all()


# ---------------------------------------------------------- preference loss

def _preference64(logp, ref, on, starts, o):
    b = (len(starts) - 1) // 2
    lp = logp.double().requires_grad_(True)
    x = lp - ref.double() if o["ref"] == "token" else lp
    S = []
    for i in range(2 * b):
        k = torch.arange(starts[i], starts[i + 1])
        k = k[on[k]]
        s = x[k].sum()
        if o["ref"] == "sequence":
            s = s - ref.double()[i]
        S.append(s / max(len(k), 1) if o["average"] else s)
    S = torch.stack(S)
    D = S[:b] - S[b:]
    h = o["beta"] * D - o["margin"]
    ls = torch.nn.functional.logsigmoid
    losses = {"sigmoid": lambda: -(1 - o["eps"]) * ls(h) - o["eps"] * ls(-h), "hinge": lambda: torch.relu(1 - h),
              "ipo": lambda: (D - 0.5 / o["beta"]) ** 2}[o["kind"]]()
    if losses.requires_grad:
        losses.mean().backward()
    grad = lp.grad if lp.grad is not None else torch.zeros_like(lp)
    return losses.detach(), (o["beta"] * S).detach(), grad, D.detach(), h.detach()


@pytest.mark.parametrize("kind", ["sigmoid", "hinge", "ipo"])
@pytest.mark.parametrize("ref", ["token", "sequence", None])
@pytest.mark.parametrize("b,n,packed,average", [(1, 2, False, False), (1, 7, True, True), (4, 2000, False, False),
                                                (3, 30000, True, True), (700, 9000, True, False),
                                                (1, 100002, False, True)])
def test_preference_loss(b, n, packed, average, ref, kind):
    g = _gen(b + n)
    rows = 2 * b
    n = n // rows * rows if not packed else n
    logp = -torch.rand(n, generator=g).pow(3) * 4
    on = torch.rand(n, generator=g) >= 0.3
    starts = [0, *sorted(int(c) for c in torch.randint(0, n + 1, (rows - 1,), generator=g)), n] if packed \
        else [i * (n // rows) for i in range(rows + 1)]
    r = None
    if ref == "token":
        r = logp + torch.randn(n, generator=g) * 0.2
    elif ref == "sequence":
        r = torch.randn(rows, generator=g) * 3
    o = dict(ref=ref, average=average, beta=0.1, margin=0.0 if kind == "ipo" else 0.2, kind=kind,
             eps=0.1 if kind == "sigmoid" else 0.0)
    losses, rewards, grad, D, h = _preference64(logp, r, on, starts, o)
    bad = torch.where(on, 0.0, float("nan"))
    shape = (n,) if packed else (rows, n // rows)
    put = lambda v: v.to(DEV).view(shape)
    rd = None if r is None else put(r + bad) if ref == "token" else r.to(DEV)
    args = dict(mask=put(on), offsets=torch.tensor(starts, device=DEV) if packed else None, beta=0.1,
                margin=o["margin"], kind=kind, label_smoothing=o["eps"], length_average=average, grad_scale=0.5)
    got = L.preference_loss(put(logp + bad), rd, **args)
    # S: terms rounded to fp32 once (u |x|), error-free sums, one rounding of S
    size = torch.tensor([float(logp[torch.arange(starts[i], starts[i + 1])].abs().sum()) for i in range(rows)])
    err = 3e-7 * (rewards.abs() / 0.1 + (0 if ref else 0) + 1e-3 * size + 1e-6)
    assert ((got.rewards.cpu().double() - rewards).abs() <= 0.1 * err + 1e-9).all()
    dD = err[:b] + err[b:] + 2e-7 * D.abs()
    slope = {"sigmoid": 0.1, "hinge": 0.1, "ipo": None}[kind]
    slope = 2 * (D - 5).abs() if slope is None else slope
    assert ((got.losses.cpu().double() - losses).abs() <= slope * dD + dD * dD + 1e-6 * losses.abs() + 1e-7).all()
    s = got.stats.cpu().double()
    assert abs(float(s[0] - losses.mean())) <= float((slope * dD + dD * dD + 1e-6 * losses.abs()).mean()) + 1e-7
    sure = D.abs() > dD
    assert abs(float(s[1]) - float((D > 0).double().mean())) <= float((~sure).double().mean()) + 1e-7
    assert abs(float(s[2] - h.mean())) <= float(0.1 * dD.mean() + 1e-6 * h.abs().mean()) + 1e-7
    want = 0.5 * grad
    d = got.d_logp.cpu().double().reshape(-1)
    # the slope's own error: at most its second derivative (beta^2 / 4, 0, 2) times D's
    second = {"sigmoid": 0.0025, "hinge": 0.0, "ipo": 2.0}[kind]
    slack = torch.zeros(n, dtype=torch.float64)
    for i in range(rows):
        k = torch.arange(starts[i], starts[i + 1])
        slack[k] = 0.5 * second * float(dD[i % b]) / b
    assert ((d - want).abs() <= 2e-6 * want.abs() + slack + 1e-12).all()
    assert (d[~on] == 0).all()
    again = L.preference_loss(put(logp + bad), rd, **args)
    assert all(torch.equal(p, q) for p, q in zip(got, again))


def test_preference_edges():
    t = lambda *v: torch.tensor(v, device=DEV)
    # both sides empty: the loss at h = 0, no gradient
    r = L.preference_loss(torch.zeros(2, 3, device=DEV), mask=torch.zeros(2, 3, dtype=torch.bool, device=DEV),
                          length_average=True)
    assert abs(float(r.losses[0]) - math.log(2)) < 1e-6 and (r.d_logp == 0).all()
    # large margins neither overflow nor lose the small side
    r = L.preference_loss(t([2000.0], [-2000.0], [-2000.0], [2000.0]), beta=1.0)
    assert r.losses.tolist() == [4000.0, 0.0] or r.losses.tolist() == [0.0, 4000.0]
    assert torch.isfinite(r.d_logp).all()
    # tokens outside every sequence
    lp = t(5.0, -1.0, -2.0, 5.0)
    r = L.preference_loss(lp, offsets=t(1, 2, 3))
    assert r.d_logp[0] == 0 and r.d_logp[3] == 0 and r.d_logp[1] < 0 < r.d_logp[2]
    assert abs(float(r.rewards[0]) + 0.1) < 1e-7
    # no tokens at all
    r = L.preference_loss(torch.zeros(0, device=DEV), offsets=t(0, 0, 0))
    assert abs(float(r.stats[0]) - math.log(2)) < 1e-6


def test_losses_together_reach_the_logits():
    """logits -> log-probabilities -> preference loss -> gradient, by autograd, against fp64."""
    x, t = _logits(4 * 6, 700, "fp32", 8)
    leaf = x.view(4, 6, 700).to(DEV).requires_grad_(True)
    r = L.token_logprob(leaf, t.view(4, 6).to(DEV))
    p = L.preference_loss(r.logp, beta=0.3)
    r.logp.backward(p.d_logp)
    z = x.double().requires_grad_(True)
    lp = torch.log_softmax(z, 1).gather(1, t[:, None])[:, 0].view(4, 6).sum(1)
    loss = -torch.nn.functional.logsigmoid(0.3 * (lp[:2] - lp[2:])).mean()
    loss.backward()
    assert abs(float(p.stats[0]) - float(loss.detach())) < 1e-5
    assert (leaf.grad.cpu().double().view(-1, 700) - z.grad).abs().max() < 1e-5 * z.grad.abs().max() + 1e-8


def test_side_stream_and_graph():
    """On a stream of the caller's, and replayed from a CUDA graph."""
    x, t = _logits(30, 5000, "bf16", 9)
    xd, td = x.to(DEV), t.to(DEV)
    old, adv = torch.full((30,), -9.0, device=DEV), torch.ones(1, device=DEV)
    want = L.policy_loss_logits(xd, td, old, adv, entropy=True)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        got = L.policy_loss_logits(xd, td, old, adv, entropy=True)
    s.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = L.policy_loss_logits(xd, td, old, adv, entropy=True)
    keep = [w.clone() for w in want]
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, keep))


# ----------------------------------------------------------------- refusals

def test_refusals():
    x = torch.zeros(4, 10, device=DEV)
    t = torch.zeros(4, dtype=torch.int64, device=DEV)
    z = torch.zeros(4, device=DEV)
    r = L.token_logprob(x, t)
    for bad, exc in [
        (lambda: L.token_logprob(x.cpu(), t), TypeError),
        (lambda: L.token_logprob(x.double(), t), TypeError),
        (lambda: L.token_logprob(x, t.int()), TypeError),
        (lambda: L.token_logprob(x, t[:3]), ValueError),
        (lambda: L.token_logprob(x, t, temperature=0.0), ValueError),
        (lambda: L.token_logprob(x.t(), torch.zeros(10, dtype=torch.int64, device=DEV)), ValueError),
        (lambda: L.token_logprob(torch.zeros(4, 0, device=DEV), t), ValueError),
        (lambda: L.token_logprob_backward(x, t, r, z[:2]), ValueError),
        (lambda: L.token_logprob_backward(x, t, r, z, z), ValueError),
        (lambda: L.token_logprob_backward(x, t, r, z, out=x[:, :5]), ValueError),
        (lambda: L.token_logprob_backward(x, t, r, z, out=torch.zeros(1, 10, device=DEV).expand(4, 10)), A.AdamWError),
        (lambda: L.policy_loss(z, z, z, kl_coef=0.1), ValueError),
        (lambda: L.policy_loss(z, z, z, entropy_coef=0.1), ValueError),
        (lambda: L.policy_loss(z, z, z, kl="k4"), ValueError),
        (lambda: L.policy_loss(z, z, z, clip_low=1.5), A.AdamWError),
        (lambda: L.policy_loss(z, z, z, dual_clip=0.5), A.AdamWError),
        (lambda: L.policy_loss(z, z, z, reduce="fixed", divisor=0.0), A.AdamWError),
        (lambda: L.policy_loss(z, z.half(), z), TypeError),
        (lambda: L.policy_loss(z, z, z[:3]), ValueError),
        (lambda: L.policy_loss(z, z, z, mask=torch.ones(4, device=DEV)), TypeError),
        (lambda: L.policy_loss(z, z, z, offsets=torch.zeros(2, device=DEV)), TypeError),
        (lambda: L.preference_loss(z), ValueError),
        (lambda: L.preference_loss(z.view(2, 2), beta=0.0), A.AdamWError),
        (lambda: L.preference_loss(z.view(2, 2), kind="ipo", margin=0.1), A.AdamWError),
        (lambda: L.preference_loss(z.view(2, 2), kind="hinge", label_smoothing=0.1), A.AdamWError),
        (lambda: L.preference_loss(z.view(2, 2), kind="other"), ValueError),
        (lambda: L.preference_loss(z.view(2, 2), torch.zeros(3, device=DEV)), ValueError),
        (lambda: L.policy_loss_logits(x, t, z, z[:3]), ValueError),
        (lambda: L.policy_loss_logits(x, t, z, z, kl_coef=0.1), ValueError),
    ]:
        with pytest.raises(exc):
            bad()
    # an output that overlaps the logits without being them
    buf = torch.zeros(50, device=DEV)
    with pytest.raises(A.AdamWError) as e:
        L.token_logprob_backward(buf[:40].view(4, 10), t, r, z, out=buf[10:].view(4, 10))
    assert e.value.status == A.ADAMW_ERR_INVALID_ARG
