"""Products grouped by expert and their gradients against sums in 64 bits.

Tolerance of one element: half a step of its type, eps / 2 relative, and the
fp32 sum of K products: each of the tensor cores' additions (16 products at a
time) and of the lanes' is off by at most 2^-23 of the partial sum, which is
below S = sum |x| |w|: (K / 16 + 16) 2^-23 S covers both, K / 8 additions a
lane of the streaming kernel among them (K / 256 + 16 a lane).
"""
import pytest
import torch

from adamw_optimizer_step_sm_gb300 import adamw_sm as A
from adamw_optimizer_step_sm_gb300 import matrix as M

pytestmark = pytest.mark.gpu

BF, HALF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _no_wait_ran_out():
    yield
    assert A.adamw_matrix_status() == 0


def bounds(offsets, tokens):
    """The groups that the call makes of any offsets."""
    out = []
    for v in offsets:
        out.append(max(out[-1] if out else 0, min(max(v, 0), tokens)))
    return out


def products(x, w, ends):
    """(y, sum |x| |w|)"""
    y, s = (torch.zeros(x.shape[0], w.shape[1], dtype=torch.float64, device="cuda") for _ in range(2))
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if a < b:
            y[a:b] = x[a:b].double() @ w[e].double().t()
            s[a:b] = x[a:b].double().abs() @ w[e].double().abs().t()
    return y, s


def outer(dy, x, ends):
    shape = len(ends) - 1, dy.shape[1], x.shape[1]
    dw, s = (torch.zeros(shape, dtype=torch.float64, device="cuda") for _ in range(2))
    for e, (a, b) in enumerate(zip(ends, ends[1:])):
        if a < b:
            dw[e] = dy[a:b].double().t() @ x[a:b].double()
            s[e] = dy[a:b].double().abs().t() @ x[a:b].double().abs()
    return dw, s


def close(got, want, k):
    value, size = want
    room = value.abs() * (torch.finfo(got.dtype).eps / 2) + size * ((k / 16 + 16) * 2.0 ** -23)
    if got.dtype == HALF:
        room = room + 2.0 ** -25   # subnormals
    assert (got.double() - value).abs().le(room).all(), float(((got.double() - value).abs() - room).max())


def rand(*shape, dtype=BF, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def offsets_of(values):
    return torch.tensor(values, dtype=torch.int64, device="cuda")


def check(tokens, n, k, offsets, dtype=BF, x=None, w=None, dy=None):
    e = len(offsets) - 1
    x = rand(tokens, k, dtype=dtype) if x is None else x
    w = rand(e, n, k, dtype=dtype, seed=2) if w is None else w
    dy = rand(tokens, n, dtype=dtype, seed=3) if dy is None else dy
    at, ends = offsets_of(offsets), bounds(offsets, tokens)
    y = M.expert_linear(x, w, at)
    close(y, products(x, w, ends), k)
    dx, dw = M.expert_linear_backward(dy, x, w, at)
    close(dx, products(dy, w.mT, ends), n)
    close(dw, outer(dy, x, ends), tokens)
    outside = torch.ones(tokens, dtype=torch.bool, device="cuda")
    outside[ends[0]:ends[-1]] = False
    assert (y[outside] == 0).all() and (dx[outside] == 0).all()
    return y, dx, dw


CASES = [  # tokens, n, k, offsets
    (1, 1, 1, [0, 1]), (1, 8, 8, [0, 1]), (3, 64, 64, [0, 1, 1, 3]), (16, 100, 200, [0, 16]), (17, 100, 200, [0, 17]),
    (128, 128, 64, [0, 128]), (129, 136, 72, [0, 129]), (300, 264, 520, [0, 100, 300]), (301, 261, 515, [0, 100, 100, 301]),
    (1000, 257, 129, [0, 1, 2, 3, 999, 1000]), (700, 33, 1027, [0, 0, 0, 700, 700]), (2000, 512, 256, [0, 640, 1280, 2000]),
    (4096, 1024, 512, [0, 4096]), (900, 1024, 64, [i * 900 // 64 for i in range(65)]), (64, 24, 4096, [0, 10, 64]),
    (2500, 768, 1536, [0, 2, 1200, 1210, 2500]), (40, 2048, 40, [0, 7, 40]),
]


@pytest.mark.parametrize("tokens,n,k,offsets", CASES, ids=str)
@pytest.mark.parametrize("dtype", [BF, HALF], ids=str)
def test_sizes(tokens, n, k, offsets, dtype):
    check(tokens, n, k, offsets, dtype)


@pytest.mark.parametrize("tokens", [12, 100, 1000])
@pytest.mark.parametrize("offsets", [[3, 5, 9], [0, 0, 0], [12, 12, 12], [-7, 4, 10 ** 12], [9, 2, 11], [5, 5, 2 ** 62],
                                     [-2 ** 63, -1, 8], [100, 50, 12]], ids=str)
def test_any_offsets(tokens, offsets):
    """Rows before, behind and between; offsets outside the rows; descending."""
    check(tokens, 72, 80, offsets)
    check(tokens, 33, 45, offsets)


def test_what_is_outside_does_not_matter():
    """NaN and inf in rows of no expert, and in the next group's rows within a
    step of the sums over tokens."""
    for tokens, offsets in ((14, [2, 5, 9]), (400, [3, 70, 71, 203, 390])):
        x, dy, w = rand(tokens, 72), rand(tokens, 80, seed=3), rand(len(offsets) - 1, 80, 72, seed=2)
        clean = check(tokens, 80, 72, offsets, x=x, w=w, dy=dy)
        x2, dy2 = x.clone(), dy.clone()
        for t in (x2, dy2):
            t[:offsets[0]] = float("nan")
            t[offsets[-1]:] = float("inf")
        at = offsets_of(offsets)
        y = M.expert_linear(x2, w, at)
        dx, dw = M.expert_linear_backward(dy2, x2, w, at)
        assert torch.equal(y, clean[0]) and torch.equal(dx, clean[1]) and torch.equal(dw, clean[2])
        x2[offsets[1]:offsets[2]] = float("nan")   # one expert's tokens
        y = M.expert_linear(x2, w, at)
        _, dw = M.expert_linear_backward(dy2, x2, w, at)
        assert y[offsets[1]:offsets[2]].isnan().all() and dw[1].isnan().all()
        keep = [i for i in range(tokens) if not offsets[1] <= i < offsets[2]]
        assert torch.equal(y[keep], clean[0][keep])
        assert all(torch.equal(dw[e], clean[2][e]) for e in range(len(offsets) - 1) if e != 1)


@pytest.mark.parametrize("tokens", [9, 300])
def test_strides(tokens):
    offsets = [0, tokens // 3, tokens - 1]
    big = rand(tokens + 4, 200)
    weights = rand(3, 90, 210, seed=2)
    for x in (big[2:tokens + 2, 8:88], big[1:tokens + 1, 3:83], big[:tokens, 10:181:2][:, :80], big[:1, :80].expand(tokens, 80)):
        for w in (weights[:2, :64, :80], weights[1:, 1:65, 5:85], weights[:, :80, :64].mT[:2], weights[:2, 3:83, 7:71].mT,
                  weights[:1, :64, :80].expand(2, 64, 80), weights[::2, :64, 1:81]):
            for dy in (rand(tokens, 64, seed=3), rand(1, 1, seed=4).expand(tokens, 64), rand(tokens, 70, seed=5)[:, 3:67]):
                check(tokens, 64, 80, offsets, x=x, w=w, dy=dy)


def test_gradient_of_a_transposed_weight_has_its_layout():
    x, w = rand(100, 64), rand(2, 64, 48, seed=2).mT
    _, dw = M.expert_linear_backward(rand(100, 48, seed=3), x, w, offsets_of([0, 50, 100]))
    assert dw.stride() == w.stride()


@pytest.mark.parametrize("dtype", [BF, HALF, F32], ids=str)
@pytest.mark.parametrize("n,k", [(64, 96), (33, 45), (300, 264)])
def test_given_results(dtype, n, k):
    """y and dw in any of the three types, at any alignment, and added to what
    is there."""
    offsets = [0, 130, 130, 297]
    x, w, dy = rand(300, k), rand(3, n, k, seed=2), rand(300, n, seed=3)
    at, ends = offsets_of(offsets), bounds(offsets, 300)
    for phase in (0, 1, 8):
        room = torch.full((300 * n + 40,), 5.0, dtype=dtype, device="cuda")
        out = room[phase:phase + 300 * n].view(300, n)
        assert M.expert_linear(x, w, at, out=out) is out
        close(out, products(x, w, ends), k)
        assert (room[:phase] == 5).all() and (room[phase + 300 * n:] == 5).all()
        room = torch.full((3 * n * k + 40,), 5.0, dtype=dtype, device="cuda")
        d = room[phase:phase + 3 * n * k].view(3, n, k)
        before = d._version
        assert M.expert_linear_backward(dy, x, w, at, need=(False, True), d_weight=d)[1] is d
        want = outer(dy, x, ends)
        close(d, want, 300)
        assert d._version > before
        first = d.double()
        M.expert_linear_backward(dy, x, w, at, need=(False, True), d_weight=d, accumulate=True)
        close(d, (first + want[0], want[1]), 300)
        assert torch.equal(d[1], torch.zeros_like(d[1]))
        assert (room[:phase] == 5).all() and (room[phase + 3 * n * k:] == 5).all()
    t = torch.zeros(3, k, n, dtype=dtype, device="cuda").mT
    M.expert_linear_backward(dy, x, w, at, need=(False, True), d_weight=t, accumulate=True)
    close(t, outer(dy, x, ends), 300)


def test_accumulate_leaves_experts_without_tokens():
    d = rand(3, 40, 48, dtype=F32)
    keep = d.clone()
    M.expert_linear_backward(rand(50, 40), rand(50, 48), rand(3, 40, 48), offsets_of([0, 50, 50, 50]), need=(False, True), d_weight=d,
                             accumulate=True)
    assert torch.equal(d[1:], keep[1:]) and not torch.equal(d[0], keep[0])


@pytest.mark.parametrize("tokens", [5, 200])
def test_autograd(tokens):
    offsets = offsets_of([0, tokens // 2, tokens])
    x, w = rand(tokens, 40).requires_grad_(), rand(2, 24, 40, seed=2).requires_grad_()
    dy = rand(tokens, 24, seed=3)
    y = M.expert_linear(x, w, offsets)
    y.backward(dy)
    dx, dw = M.expert_linear_backward(dy, x.detach(), w.detach(), offsets)
    assert torch.equal(x.grad, dx) and torch.equal(w.grad, dw)
    # one of the two, an expanded gradient, no gradient
    z = M.expert_linear(x.detach(), w, offsets)
    g, = torch.autograd.grad(z.sum(), w)
    close(g, outer(torch.ones_like(dy), x.detach(), [0, tokens // 2, tokens]), tokens)
    g, = torch.autograd.grad(M.expert_linear(x, w.detach(), offsets).float().sum(), x)
    close(g, products(torch.ones_like(dy), w.detach().mT, [0, tokens // 2, tokens]), 24)
    with torch.no_grad():
        assert not M.expert_linear(x, w, offsets).requires_grad


def test_gradient_against_differences():
    """The derivative of sum(c y) along a direction, by a difference of the
    definition in 64 bits."""
    tokens, ends = 60, [0, 25, 60]
    x, w, c = rand(tokens, 32), rand(2, 16, 32, seed=2), rand(tokens, 16, seed=3)
    dx, dw = M.expert_linear_backward(c, x, w, offsets_of(ends))
    vx, vw = rand(tokens, 32, seed=4).double(), rand(2, 16, 32, seed=5).double()
    f = lambda h: (products(x.double() + h * vx, w.double() + h * vw, ends)[0] * c.double()).sum()
    h = 1e-3
    slope = (f(h) - f(-h)) / (2 * h)   # exact for a bilinear form, but for fp64's rounding
    got = (dx.double() * vx).sum() + (dw.double() * vw).sum()
    # each gradient element is off by at most 2^-9 of its value: a random walk over them
    room = 2.0 ** -9 * 6 * ((dx.double() * vx).square().sum() + (dw.double() * vw).square().sum()).sqrt()
    assert abs(got - slope) < room


def test_a_run_of_layers():
    """Two layers of experts with a non-linearity between, as they are used:
    against torch in fp64."""
    tokens, ends = 333, [0, 100, 101, 330]
    at = offsets_of(ends)
    x = rand(tokens, 64).requires_grad_()
    up, down = (rand(3, 96, 64, seed=2) * 0.1).requires_grad_(), (rand(3, 64, 96, seed=3) * 0.1).requires_grad_()
    z = x + M.expert_linear(torch.relu(M.expert_linear(x, up, at)), down, at)
    z.backward(rand(tokens, 64, seed=4))
    xd, ud, dd = (t.detach().double().requires_grad_() for t in (x, up, down))
    parts = [xd[a:b] + torch.relu(xd[a:b] @ ud[e].t()) @ dd[e].t() for e, (a, b) in enumerate(zip(ends, ends[1:]))]
    want = torch.cat(parts + [xd[ends[-1]:]])
    want.backward(rand(tokens, 64, seed=4).double())
    for got, ref in ((z, want), (x.grad, xd.grad), (up.grad, ud.grad), (down.grad, dd.grad)):
        # a handful of bf16 roundings (half a step 2^-9 each in the 2-norm) between
        assert (got.detach().double() - ref).norm() < 5 * 2.0 ** -9 * ref.norm()


def test_same_bits():
    for tokens, n, k, offsets in CASES[-6:]:
        x, w, dy, at = rand(tokens, k), rand(len(offsets) - 1, n, k), rand(tokens, n), offsets_of(offsets)
        first = (M.expert_linear(x, w, at), *M.expert_linear_backward(dy, x, w, at))
        for _ in range(10):
            again = (M.expert_linear(x, w, at), *M.expert_linear_backward(dy, x, w, at))
            assert all(torch.equal(a, b) for a, b in zip(first, again))


@pytest.mark.parametrize("tokens", [6, 700])
def test_streams_and_graphs(tokens):
    x, w, dy = rand(tokens, 136), rand(5, 72, 136, seed=2), rand(tokens, 72, seed=3)
    at = offsets_of([0, 1, tokens // 2, tokens // 2, tokens - 1, tokens])
    def call():
        return (M.expert_linear(x, w, at), *M.expert_linear_backward(dy, x, w, at))
    want = call()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(call())
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for g in got for a, b in zip(g, want))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = call()
    for offsets in ([0, 0, 2, 3, 3, tokens], [1, 2, 3, 4, 4, 4], [0, 1, 2, 3, 4, 5]):   # other groups, the same graph
        at.copy_(offsets_of(offsets))
        x.copy_(rand(tokens, 136, seed=sum(offsets)))
        g.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, call()))


def test_a_thousand_experts():
    counts = [(7 * i) % 5 for i in range(1024)]
    offsets = [sum(counts[:i]) for i in range(1025)]
    check(offsets[-1] + 3, 40, 24, offsets)
    with pytest.raises(A.AdamWError):
        M.expert_linear(rand(4, 8), rand(1025, 8, 8), offsets_of([0] * 1026))


def test_empty():
    at = offsets_of([0, 0, 0])
    assert M.expert_linear(rand(0, 24), rand(2, 16, 24), at).shape == (0, 16)
    dx, dw = M.expert_linear_backward(rand(0, 16), rand(0, 24), rand(2, 16, 24), at)
    assert dx.shape == (0, 24) and (dw == 0).all()
    for tokens in (3, 100):   # sums of nothing are zeros
        y = M.expert_linear(rand(tokens, 0), rand(2, 16, 0), offsets_of([0, 1, tokens]))
        assert y.shape == (tokens, 16) and (y == 0).all()
        assert M.expert_linear(rand(tokens, 8), rand(2, 0, 8), offsets_of([0, 1, tokens])).shape == (tokens, 0)
        dx, dw = M.expert_linear_backward(rand(tokens, 0), rand(tokens, 8), rand(2, 0, 8), offsets_of([0, 1, tokens]))
        assert (dx == 0).all() and dw.shape == (2, 0, 8)


def test_large():
    """Offsets beyond 2^31 elements in tokens, weights and results."""
    tokens, k = 2 ** 31 // 4096 + 300, 4096
    x = torch.zeros(tokens, k, dtype=BF, device="cuda")
    x[-300:] = rand(300, k)
    w = rand(2, 64, k, seed=2)
    at = offsets_of([0, tokens - 300, tokens])
    y = M.expert_linear(x, w, at)
    close(y[-300:], products(x[-300:], w[1:], [0, 300]), k)
    assert (y[:-300] == 0).all()
    dx, dw = M.expert_linear_backward(y, x, w, at)
    close(dx[-300:], products(y[-300:], w[1:].mT, [0, 300]), 64)
    close(dw[1:], outer(y[-300:], x[-300:], [0, 300]), 300)
    assert (dw[0] == 0).all()
    del x, y, dx
    w = torch.zeros(9, 16384, 16384, dtype=BF, device="cuda")   # 2.4e9 elements
    w[8, -50:] = rand(50, 16384)
    for tokens in (4, 40):
        x = rand(tokens, 16384, seed=7)
        y = M.expert_linear(x, w, offsets_of([0] * 9 + [tokens]))
        close(y[:, -50:], products(x, w[8:, -50:], [0, tokens]), 16384)
        assert (y[:, :-50] == 0).all()
    del w
    torch.cuda.empty_cache()


def test_refusals():
    x, w, at = rand(6, 8), rand(2, 4, 8), offsets_of([0, 3, 6])
    dy = rand(6, 4)
    calls = [
        lambda: M.expert_linear(x.float(), w.float(), at), lambda: M.expert_linear(x, w.half(), at),
        lambda: M.expert_linear(x, w, at.int()), lambda: M.expert_linear(x, w, at[:2]), lambda: M.expert_linear(x, w, at.cpu()),
        lambda: M.expert_linear(x[0], w, at), lambda: M.expert_linear(x, w[0], at), lambda: M.expert_linear(x[:, :7], w, at),
        lambda: M.expert_linear(x, w[:0], at[:1]), lambda: M.expert_linear(x, w, at, out=rand(6, 5)),
        lambda: M.expert_linear(x, w, at, out=rand(4, 6).t()),
        lambda: M.expert_linear(x.clone().requires_grad_(), w, at, out=rand(6, 4)),
        lambda: M.expert_linear(x, w, at, out=x[:, :4]),          # over its own input
        lambda: M.expert_linear_backward(dy.half(), x, w, at), lambda: M.expert_linear_backward(dy[:5], x, w, at),
        lambda: M.expert_linear_backward(dy[:, :3], x, w, at), lambda: M.expert_linear_backward(dy, x, w, at, accumulate=True),
        lambda: M.expert_linear_backward(dy, x, w, at, d_weight=rand(2, 4, 7)),
        lambda: M.expert_linear_backward(dy, x, w, at, d_weight=torch.zeros(2, 4, 8, dtype=torch.float64, device="cuda")),
        lambda: M.expert_linear_backward(dy, x, w, at, d_weight=torch.zeros(2, 8, 16, device="cuda")[:, ::2, ::2]),
        lambda: M.expert_linear_backward(dy, x, w, at, d_weight=torch.zeros(1, 4, 8, device="cuda").expand(2, 4, 8)),
    ]
    for call in calls:
        with pytest.raises((TypeError, ValueError, RuntimeError)):
            call()
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises((RuntimeError, NotImplementedError)):
            M.expert_linear(torch.autograd.forward_ad.make_dual(x, x), w, at)
