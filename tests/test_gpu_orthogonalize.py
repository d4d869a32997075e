"""Newton-Schulz orthogonalisation against the iteration in 64 bits.

Tolerance.  Entries are rounded to fp16 at four places of a step, each off by
at most 2^-12 of its value, rms 2^-12 / sqrt(3) = 1.4e-4.  What they change
of the next X (singular values about 1 or less): Q and the X that it multiplies
enter with |Q| <= 2.8 each, G with |b + 2 c G| <= 4.8, twice over its two
factors: 1.4e-4 (2.8^2 + 2.8^2 + 2 * 4.8^2)^0.5 = 1.1e-3 a step (2-norm, relative).  A later
step multiplies it by |p'| <= 1.6 about there; over the last steps that adds up
to less than 2.8 times one step's: 3.1e-3.  Rounding the result to bf16 (half
a step, 2^-8, rms 2.3e-3 at most) or fp16 (2^-11) comes on top, in
quadrature: 4e-3 for all.
"""
import math

import pytest
import torch

from adamw_optimizer_step_sm_gb300 import adamw_sm as A
from adamw_optimizer_step_sm_gb300 import matrix as M

pytestmark = pytest.mark.gpu

TOL = 4e-3
BF, HALF, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(autouse=True)
def _no_wait_ran_out():
    yield
    assert A.adamw_matrix_status() == 0


def exact(x, steps=5, coefficients=M.COEFFICIENTS, eps=1e-7):
    """By the definition: the matrix multiplied in every step, from the left."""
    x = x.double()
    x = x / torch.linalg.matrix_norm(x).clamp(min=eps)[..., None, None]
    rows = [coefficients] if not hasattr(coefficients[0], "__len__") else list(coefficients)
    for k in range(steps):
        a, b, c = rows[min(k, len(rows) - 1)]
        g = x @ x.mT
        x = a * x + (b * g + c * (g @ g)) @ x
    return x


def off(y, want):
    """The largest relative error of a matrix of the batch, in the 2-norm."""
    d = torch.linalg.matrix_norm(y.double() - want) / torch.linalg.matrix_norm(want)
    return float(d.max())


def rand(*shape, dtype=F32, seed=1, scale=1.0, rank=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    if rank is None:
        x = torch.randn(shape, generator=g, device="cuda")
    else:
        x = torch.randn(*shape[:-1], rank, generator=g, device="cuda") @ torch.randn(*shape[:-2], rank, shape[-1], generator=g, device="cuda")
    return (x * scale).to(dtype)


# both kernels (the small one up to 128 x 1024), one to eight CTAs of a cluster,
# every tile shape's edges, sides that are no multiple of 8, tall and wide
SHAPES = [(1, 1), (1, 7), (9, 1), (2, 3), (16, 16), (17, 33), (64, 128), (128, 128), (127, 129), (128, 1024), (1000, 100), (1024, 128),
          (129, 129), (128, 1025), (130, 2000), (255, 257), (515, 1031), (1031, 515), (300, 1), (1, 1500), (768, 768), (640, 200),
          (2, 1100), (4, 3000), (8, 5000), (3000, 3), (16, 4096), (2500, 64), (128, 1500), (1100, 127)]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("dtype", [BF, HALF, F32], ids=str)
def test_shapes_and_types(shape, dtype):
    x = rand(*shape, dtype=dtype)
    want = exact(x)
    for out in (BF, F32):
        y = M.orthogonalize(x, dtype=out)
        assert y.dtype == out and y.shape == x.shape
        assert off(y, want) < TOL


@pytest.mark.parametrize("shape", [(12, 4, 1100), (12, 2000, 8), (6, 128, 64), (8, 3, 50), (5, 100, 1030)], ids=str)
def test_thin_matrices(shape):
    """Few singular values, whose errors do not average out: held to half the
    tolerance, at many scales of them."""
    for seed in range(4):
        x = rand(*shape, seed=seed)
        x *= torch.logspace(0, -2, shape[-1 if shape[-1] < shape[-2] else -2], device="cuda")[(None, slice(None)) if shape[-1] < shape[-2] else (slice(None), None)]
        assert off(M.orthogonalize(x, dtype=F32), exact(x)) < TOL / 2


@pytest.mark.parametrize("length", [1, 2, 3, 33, 144, 300, 1000, 1030, 2000])
@pytest.mark.parametrize("side", [1, 2, 3, 5, 8, 17, 32])
def test_smallest_sides(side, length):
    """Sides of up to 32, whose few errors do not average out: every operand is two
    fp16 there, each rounding at most 2^-22 of its value whatever its sign.  Q and the
    X that it multiplies enter with 2.8 each, G's factors with 4.8 each: 15.2 2^-22 =
    3.6e-6 a step at most.  A step multiplies an error by a = 3.44 at most, so five
    leave (1 + 3.44 + ... + 3.44^4) 3.6e-6 = 7.1e-4."""
    length = max(side, length)
    for seed, dtype in enumerate((BF, HALF, F32)):
        for shape in ((200, side, length), (200, length, side)):
            x = rand(*shape, dtype=dtype, seed=seed)
            want = exact(x) if shape[1] == side else exact(x.mT).mT   # the same, of the smaller side
            assert off(M.orthogonalize(x, dtype=F32), want) < 7.1e-4


@pytest.mark.parametrize("shape", [(7, 64, 96), (3, 2, 33, 40), (200, 16, 20), (5, 257, 130), (2, 3, 300, 299)], ids=str)
def test_batches(shape):
    x = rand(*shape, dtype=BF)
    scale = torch.logspace(-6, 6, math.prod(shape[:-2]), device="cuda").view(*shape[:-2], 1, 1).bfloat16()
    x = x * scale   # each matrix has its own norm
    assert off(M.orthogonalize(x), exact(x)) < TOL


@pytest.mark.parametrize("shape,rank", [((96, 200), 3), ((768, 768), 8), ((2048, 512), 64), ((512, 3000), 100)], ids=str)
def test_few_directions(shape, rank):
    """Singular values of zero: rounding must not reach them, where five steps
    multiply by 485."""
    x = rand(*shape, rank=rank, dtype=F32)
    y, want = M.orthogonalize(x, dtype=F32), exact(x)
    assert off(y, want) < TOL
    # the input's own fp32 rounding, 2^-24 of it, grows to 485 times that: 3e-5
    assert int(torch.linalg.matrix_rank(want, rtol=1e-3)) == rank
    s = torch.linalg.svdvals(y.double())
    assert s[:rank].min() > 0.6 and s[0] < 1.3 and (s[rank:] < 0.05).all()


def test_singular_values():
    y = M.orthogonalize(rand(400, 700), dtype=F32)
    s = torch.linalg.svdvals(y.double())
    assert 0.6 < s.min() and s.max() < 1.25


@pytest.mark.parametrize("shape", [(100, 60), (300, 500)], ids=str)
@pytest.mark.parametrize("steps", [1, 2, 3, 10, 32])
def test_steps(shape, steps):
    x = rand(*shape)
    # a contraction: the classical coefficients, whose errors do not grow
    c = (1.875, -1.25, 0.375)
    assert off(M.orthogonalize(x, steps=steps, coefficients=c, dtype=F32), exact(x, steps, c)) < TOL


@pytest.mark.parametrize("shape", [(100, 60), (300, 500)], ids=str)
def test_coefficients_of_each_step(shape):
    x = rand(*shape)
    c = [(3.4445, -4.775, 2.0315), (2.5, -2.5, 1.0), (1.875, -1.25, 0.375)]
    for steps in (2, 3, 5):   # fewer than the list's, as many, more
        assert off(M.orthogonalize(x, steps=steps, coefficients=c, dtype=F32), exact(x, steps, c)) < TOL


@pytest.mark.parametrize("shape", [(64, 96), (300, 200)], ids=str)
def test_scale_of_the_input(shape):
    x = rand(*shape)
    want = M.orthogonalize(x)
    for e in (-120, -60, -30, 30, 60, 120):   # squares beyond fp32 in both directions
        y = M.orthogonalize(x * 2.0 ** e, eps=1e-38)
        assert torch.equal(y, want) or off(y, want.double()) < 2e-3   # a power of two changes the norm's rounding at most
    assert off(M.orthogonalize(x * 1e-12), exact(x * 1e-12)) < TOL   # below eps: not brought to norm 1
    assert off(M.orthogonalize(x * 1e-12, eps=1e-20), exact(x)) < TOL


@pytest.mark.parametrize("shape", [(3, 64, 96), (3, 300, 200), (3, 100, 1000)], ids=str)
def test_zeros_and_non_finite(shape):
    for bad in (math.inf, -math.inf, math.nan):
        x = rand(*shape, dtype=BF)
        x[0] = 0
        x[1, 5, 7] = bad
        y = M.orthogonalize(x)
        assert (y[0] == 0).all() and y[1].isnan().all() and off(y[2:], exact(x[2:])) < TOL


def test_rows_of_zeros():
    x = rand(200, 300)
    x[50:] = 0
    y = M.orthogonalize(x, dtype=F32)
    assert (y[50:] == 0).all() and off(y, exact(x)) < TOL
    x = rand(60, 500)
    x[:, 17:] = 0
    y = M.orthogonalize(x, dtype=F32)
    assert (y[:, 17:] == 0).all() and off(y, exact(x)) < TOL


@pytest.mark.parametrize("dtype", [BF, F32], ids=str)
@pytest.mark.parametrize("shape", [(64, 90), (300, 200)], ids=str)
def test_strides(shape, dtype):
    r, c = shape
    wide = rand(2, r + 3, c + 5, dtype=dtype)
    views = [wide[:, 1:r + 1, 3:c + 3], wide[:, ::2, :][:, :r // 2, 1:c], wide.mT[:, :c, 2:r], wide[0, :r, :c], wide[0].mT[3:c, 1:r],
             wide[:, :, ::2], wide[:1].expand(4, -1, -1), wide[:, None].expand(2, 3, r + 3, c + 5)]
    for v in views:
        y = M.orthogonalize(v)
        assert y.shape == v.shape and off(y, exact(v)) < TOL
        assert off(M.orthogonalize(v.mT).mT, exact(v)) < TOL
    assert wide.equal(rand(2, r + 3, c + 5, dtype=dtype))   # not written


@pytest.mark.parametrize("shape", [(4, 64, 90), (2, 300, 200), (100, 1000), (257, 511)], ids=str)
def test_out(shape):
    x = rand(*shape, dtype=BF)
    want = M.orthogonalize(x)
    for dtype in (BF, HALF, F32):
        room = torch.full((x.numel() + 64,), 7.0, dtype=dtype, device="cuda")
        for phase in (0, 1, 8, 16):   # elements past a boundary
            out = room[phase:phase + x.numel()].view(shape)
            assert M.orthogonalize(x, out=out) is out
            assert off(out, want.double()) < 2.0 ** -8 + 1e-6
            assert (room[:phase] == 7).all() and (room[phase + x.numel():] == 7).all()
            room.fill_(7.0)
    y, version = x.clone(), None
    version = y._version
    assert M.orthogonalize(y, out=y) is y and torch.equal(y, want) and y._version > version


def test_same_bits():
    for shape in ((64, 96), (3, 100, 1000), (300, 200), (2, 700, 900)):
        x = rand(*shape, dtype=BF)
        a = M.orthogonalize(x, dtype=F32)
        for _ in range(5):
            assert torch.equal(M.orthogonalize(x, dtype=F32), a)


def test_a_batch_is_its_matrices():
    for shape in ((6, 64, 96), (6, 300, 200)):
        x = rand(*shape, dtype=BF)
        y = M.orthogonalize(x, dtype=F32)
        one = torch.stack([M.orthogonalize(m, dtype=F32) for m in x])
        assert off(y, one.double()) < 2e-3   # other tiles, the same sums


def test_empty():
    for shape in ((0, 5), (5, 0), (0, 3, 4), (2, 0, 3, 4)):
        assert M.orthogonalize(torch.empty(shape, device="cuda")).shape == shape


@pytest.mark.parametrize("shape", [(64, 96), (4, 300, 200)], ids=str)
def test_streams_and_graphs(shape):
    x = rand(*shape, dtype=BF)
    want = M.orthogonalize(x)
    side, other = torch.cuda.Stream(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    other.wait_stream(torch.cuda.current_stream())
    got = []
    for _ in range(8):   # two calls at once
        for s in (side, other):
            with torch.cuda.stream(s):
                got.append(M.orthogonalize(x))
    torch.cuda.synchronize()
    assert all(torch.equal(g, want) for g in got)
    graphs, outs = [], []
    for _ in range(2):
        g, y = torch.cuda.CUDAGraph(), torch.empty_like(x)
        with torch.cuda.graph(g):
            M.orthogonalize(x, out=y)
        graphs.append(g)
        outs.append(y)
    for seed in (1, 2, 3):
        x.copy_(rand(*shape, dtype=BF, seed=seed))
        for g in graphs:
            g.replay()
        torch.cuda.synchronize()
        want = M.orthogonalize(x)
        assert all(torch.equal(y, want) for y in outs)


def test_many_calls_in_a_row():
    """Kernels that follow one another closely, of every tile shape."""
    xs = [rand(*s, dtype=BF) for s in ((300, 200), (2, 1024, 1024), (64, 64), (2048, 300), (8, 512, 512), (100, 1000))]
    want = [M.orthogonalize(x) for x in xs]
    for _ in range(30):
        assert all(torch.equal(M.orthogonalize(x), w) for x, w in zip(xs, want))


def test_large():
    """More elements than 2^31 in a batch (bf16), checked at both ends."""
    n = 2 ** 31 // (1024 * 512) + 2
    x = torch.empty(n, 512, 1024, dtype=BF, device="cuda")
    x[:] = rand(512, 1024, dtype=BF)
    x[-1] = rand(512, 1024, dtype=BF, seed=9)
    y = M.orthogonalize(x)
    want = exact(torch.stack([x[0], x[-1]]))
    assert off(torch.stack([y[0], y[-1]]), want) < TOL
    assert torch.equal(y[0], y[n // 2])
    del x, y
    torch.cuda.empty_cache()


def test_refusals():
    x = rand(8, 9)
    for bad, error in (((x[0],), ValueError), ((x.double(),), TypeError), ((x.long(),), TypeError)):
        with pytest.raises(error):
            M.orthogonalize(*bad)
    for kw in (dict(steps=0), dict(steps=33), dict(eps=0.0), dict(eps=-1.0), dict(coefficients=(1.0, 2.0)), dict(dtype=torch.float64),
               dict(out=x[:4]), dict(out=torch.empty(9, 8, device="cuda").t()), dict(out=torch.empty(8, 9)),
               dict(out=torch.empty(8, 9, dtype=torch.float64, device="cuda"))):
        with pytest.raises((ValueError, TypeError, A.AdamWError)):
            M.orthogonalize(x, **kw)
    leaf = x.clone().requires_grad_()
    with pytest.raises(RuntimeError):
        M.orthogonalize(leaf)
    with torch.no_grad():
        M.orthogonalize(leaf)
    room = torch.empty(200, device="cuda")
    with pytest.raises(A.AdamWError):   # reaches into its source
        M.orthogonalize(room[:72].view(8, 9), out=room[8:80].view(8, 9))
    with torch.autograd.forward_ad.dual_level():
        with pytest.raises(RuntimeError):
            M.orthogonalize(torch.autograd.forward_ad.make_dual(x, x))
