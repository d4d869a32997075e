"""The matrix operators at the ends of what their calls allow: against
definitions in 64 bits, with the tolerances of test_gpu_experts.py and
test_gpu_orthogonalize.py unless a test says why it has another."""
import math

import pytest
import torch

from adamw_optimizer_step_sm_gb300 import adamw_sm as A
from adamw_optimizer_step_sm_gb300 import matrix as M
from adamw_optimizer_step_sm_gb300 import optim as OPT
from test_gpu_experts import _no_wait_ran_out, check, close, offsets_of, outer, products, rand  # noqa: F401
from test_gpu_orthogonalize import TOL, exact, off

pytestmark = pytest.mark.gpu

BF, HALF, F32 = torch.bfloat16, torch.float16, torch.float32


# ------------------------------------------------- one matrix for all experts --

@pytest.mark.parametrize("tokens", [9, 300])
@pytest.mark.parametrize("dtype", [BF, HALF], ids=str)
@pytest.mark.parametrize("n,k", [(64, 80), (264, 520), (33, 45)])
def test_one_matrix_for_all_experts(tokens, dtype, n, k):
    """A stride of 0 between the experts' matrices, rows that TMA reads in place
    (strides of 8 elements) or not, and the transposed views of such weights."""
    offsets = [1, tokens // 3, tokens // 3, tokens // 2, tokens - 1]
    rows = (k + 7) // 8 * 8
    for w in (rand(1, n, rows, dtype=dtype, seed=2)[:, :, :k].expand(4, n, k), rand(n, k + 1, dtype=dtype, seed=2)[:, :k].expand(4, n, k),
              rand(1, k, (n + 7) // 8 * 8, dtype=dtype, seed=2)[:, :, :n].mT.expand(4, n, k)):
        assert w.stride(0) == 0
        y, dx, dw = check(tokens, n, k, offsets, dtype=dtype, w=w)
        again = check(tokens, n, k, offsets, dtype=dtype, w=w.clone(memory_format=torch.contiguous_format))
        if tokens > 16 and w.stride(2) == 1:   # as of copies of it, to the bit
            assert all(torch.equal(a, b) for a, b in zip((y, dx, dw), again))


def test_gradient_of_one_matrix_for_all_experts():
    """Through expand: the gradients of the experts are added up."""
    w = rand(1, 64, 80, seed=2).requires_grad_()
    x, dy, ends = rand(300, 80), rand(300, 64, seed=3), [0, 100, 120, 300]
    M.expert_linear(x, w.expand(3, 64, 80), offsets_of(ends)).backward(dy)
    dw, size = outer(dy, x, ends)
    # one rounding to bf16 of each, one of their sum; the third for second orders
    room = dw.abs().sum(0) * 3 * 2.0 ** -8 + size.sum(0) * (300 / 16 + 16) * 2.0 ** -23
    assert (w.grad[0].double() - dw.sum(0)).abs().le(room).all()


@pytest.mark.parametrize("tokens", [9, 300])
def test_experts_that_alternate_by_rows(tokens):
    """The matrices' rows by turns: strides between experts smaller than those
    between rows."""
    big, turned = rand(64, 4, 80, seed=2), rand(80, 4, 64, seed=3)
    for w in (big.permute(1, 0, 2), turned.permute(1, 2, 0), big.permute(1, 0, 2)[:, :, 3:77]):
        check(tokens, 64, w.shape[2], [0, tokens // 4, tokens // 3, tokens // 2, tokens], w=w)


# --------------------------------------------------------- norms beyond fp32's --

SMALL_AND_LARGE = pytest.mark.parametrize("shape", [(3, 64, 96), (3, 20, 30), (2, 100, 1000), (3, 300, 200), (2, 40, 2000)], ids=str)


@SMALL_AND_LARGE
@pytest.mark.parametrize("eps", [1e-7, 1e-36, 1e-38, 1e-45])
def test_zero_matrices_give_zeros(shape, eps):
    """2^12 / eps is beyond fp32 from 1.2e-35 down."""
    x = rand(*shape, dtype=F32)
    want = M.orthogonalize(x, eps=eps)
    x[1] = 0
    y = M.orthogonalize(x, eps=eps)
    assert (y[1] == 0).all() and torch.equal(y[0], want[0])


@SMALL_AND_LARGE
def test_norms_of_the_smallest_and_largest_numbers(shape):
    """Down to subnormal elements, whose few bits are the matrix's own."""
    for scale in (1e-36, 1e-40, 1e-43):
        x = rand(*shape, dtype=F32) * scale
        assert off(M.orthogonalize(x, eps=1e-45, dtype=F32), exact(x, eps=2.0 ** -149)) < TOL
    x = rand(*shape, dtype=F32) * 1e-36   # below eps: not brought to norm 1
    assert off(M.orthogonalize(x, eps=1e-32, dtype=F32), exact(x, eps=1e-32)) < TOL
    x = rand(*shape, dtype=F32).sign() * 3e38
    assert off(M.orthogonalize(x, dtype=F32), exact(x)) < TOL


@pytest.mark.parametrize("eps", [1e-7, 1e-38])
def test_muon_step_of_no_gradient(eps):
    """Momentum and update are zeros: the weights only decay, whatever eps."""
    params = [torch.nn.Parameter(rand(*s, seed=4)) for s in ((64, 96), (300, 200), (2, 40, 1030))]
    opt = OPT.Muon(params, lr=0.25, weight_decay=0.5, eps=eps)
    before = [opt.state[p]["master"].clone() for p in params]
    opt.step()
    assert int(opt.last_nonfinite[0]) == 0
    for p, w in zip(params, before):
        assert torch.equal(opt.state[p]["master"], w * 0.875) and (opt.state[p]["momentum"] == 0).all()


# ------------------------------------------------------ captured steps' rates --

def _two_muons(**kw):
    out = []
    for _ in range(2):
        params = [torch.nn.Parameter(rand(*s, seed=4)) for s in ((64, 48), (300, 200))]
        out.append((params, OPT.Muon(params, lr=1e-2, **kw)))
    return out


def _grads(params, seed):
    for k, p in enumerate(params):
        p.grad.copy_(rand(*p.shape, seed=seed + 100 * k))


@pytest.mark.parametrize("warm", [False, True])
def test_capture_does_not_record_rates(warm):
    """Rates changed since the last step, or never written: the capture is
    refused, before anything of the step is recorded; pushed first, the replays
    take what is pushed for each."""
    (a, x), (b, y) = _two_muons()
    if warm:
        for p, o in ((a, x), (b, y)):
            _grads(p, 1)
            o.step()
        x.param_groups[0]["lr"] = y.param_groups[0]["lr"] = 5e-3
    before = [p.detach().clone() for p in a]
    with pytest.raises(RuntimeError, match="push_rates"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            x.step()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, before))
    x.push_rates()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.step()
    junk = []
    for k, lr in enumerate((5e-3, 2e-3, 2e-3, 0.0, 1e-2)):
        for p, o in ((a, x), (b, y)):
            _grads(p, 5 + k)
            o.param_groups[0]["lr"] = lr
        x.push_rates()
        junk.append(torch.full((4,), 1e3).pin_memory())   # what a released pinned block may hold next
        g.replay()
        y.step()
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        if k == 2:   # a step between replays
            for p, o in ((a, x), (b, y)):
                o.step()
            assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_capture_does_not_record_an_adamw_step_rates():
    """The same of the other optimizers of the module, whose replays keep the
    rates of the step before the capture."""
    out = []
    for _ in range(2):
        params = [torch.nn.Parameter(rand(40, 50, seed=4)), torch.nn.Parameter(rand(77, seed=5))]
        out.append((params, OPT.AnyPrecisionAdamW(params, lr=1e-2)))
    (a, x), (b, y) = out
    for p, o in out:
        _grads(p, 1)
        o.step()
        o.param_groups[0]["lr"] = 4e-3
    held = torch.full((64,), 200, dtype=torch.uint8).pin_memory()
    del held   # a pinned block that could be taken in a capture
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph()):
            x.step()
    x.step()
    y.step()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        x.step()
    for _ in range(3):
        g.replay()
        y.step()
        assert all(torch.equal(p, q) for p, q in zip(a, b))


# ------------------------------------------------------------- very long sums --

def test_sums_longer_than_a_fixed_wait():
    """Tiles of 4.2e6 steps of 64 k, about a second of one SM: the epilogue's wait
    for them has its time for each step.  All but the last rows are zeros, whose
    sums are exact."""
    n = 2 ** 28
    x, dy = (torch.zeros(n + 300, 8, dtype=BF, device="cuda") for _ in range(2))
    x[-300:], dy[-300:] = rand(300, 8), rand(300, 8, seed=3)
    w = rand(2, 8, 8, seed=2)
    _, dw = M.expert_linear_backward(dy, x, w, offsets_of([0, 0, n + 300]), need=(False, True))
    close(dw[1:], outer(dy[-300:], x[-300:], [0, 300]), 300)
    assert (dw[0] == 0).all()
    del x, dy
    x, w = torch.zeros(17, n, dtype=BF, device="cuda"), torch.zeros(1, 8, n, dtype=BF, device="cuda")
    x[:, -300:], w[:, :, -300:] = rand(17, 300), rand(1, 8, 300, seed=2)
    y = M.expert_linear(x, w, offsets_of([0, 17]))
    close(y, products(x[:, -300:], w[:, :, -300:], [0, 17]), 300)
    del x, w
    torch.cuda.empty_cache()


# --------------------------------------------------------- waits that run out --

@pytest.fixture
def expiring():
    """Kernels say that a wait of theirs ran out, though none did."""
    A.adamw_matrix_test_expire(True)
    yield
    A.adamw_matrix_test_expire(False)
    A.adamw_matrix_status()


@pytest.mark.parametrize("shapes", [[(64, 48)], [(300, 200)], [(40, 1500), (700, 130)], [(300, 200), (64, 48), (2, 100, 1000)]], ids=str)
def test_a_step_reports_its_waits(expiring, shapes):
    """In its own word, without a synchronisation, and in the device's; one whose
    gradients are not finite besides says both; the next one is as ever."""
    params = [torch.nn.Parameter(rand(*s, seed=4)) for s in shapes]
    opt = OPT.Muon(params, lr=1e-2)
    for bad, word in ((False, 2), (True, 3)):
        _grads(params, 1)
        if bad:
            params[0].grad.view(-1)[0] = float("inf")
        opt.step()
        assert int(opt.last_nonfinite[0]) == word
        assert A.adamw_matrix_status() == 1
    A.adamw_matrix_test_expire(False)
    opt.sync_master()
    _grads(params, 2)
    opt.step()
    assert int(opt.last_nonfinite[0]) == 0
    assert A.adamw_matrix_status() == 0


@pytest.mark.parametrize("shape", [(64, 48), (300, 200)], ids=str)
def test_a_call_reports_its_waits(expiring, shape):
    x = rand(*shape)
    y = M.orthogonalize(x)
    assert A.adamw_matrix_status() == 1
    A.adamw_matrix_test_expire(False)
    assert torch.equal(M.orthogonalize(x), y)
    assert A.adamw_matrix_status() == 0


# --------------------------------------------------- sums of G over a cluster --

def _nearly_orthogonal(side, length, seed):
    """Integers of which every operand of one step is exact in fp16: rows 0 and 1
    whose product is 1, though its parts over each 128 columns are thousands (more
    than 11 bits), and row 2, which makes the norm a power of two."""
    g = torch.Generator().manual_seed(seed)
    z = torch.zeros(side, length, dtype=torch.int64)
    z[:2] = torch.randint(-40, 41, (2, length), generator=g)
    z[0, ::3] = 0   # where the result is the product alone, times row 1
    z[:2, 3:9] = 0
    rest = 1 - int(z[0] @ z[1])
    high = round(rest / 64)
    z[0, 3], z[1, 3], z[0, 4], z[1, 4] = 1, rest - 64 * high, 64, high
    size = int((z * z).sum())
    norm = 1
    while norm * norm < size:
        norm *= 2
    z[2, 5:9] = torch.tensor(_squares(norm * norm - size, 4))
    assert int((z * z).sum()) == norm * norm and int(z.abs().max()) <= 2048 and int(z[0] @ z[1]) == 1
    return z, norm


def _squares(n, count):
    """Numbers whose squares add up to n: four always do."""
    if count == 1:
        return [math.isqrt(n)] if math.isqrt(n) ** 2 == n else None
    for a in range(math.isqrt(n), -1, -1):
        rest = _squares(n - a * a, count - 1)
        if rest is not None:
            return [a] + rest
    return None


@pytest.mark.parametrize("side", [33, 64, 128, 20])
@pytest.mark.parametrize("length", [128, 200, 256, 500, 1000, 1024])
@pytest.mark.parametrize("turned", [False, True])
def test_sums_over_a_cluster_are_fp32(side, length, turned):
    """One step of X <- G X: the sum over the cluster's parts is 1 to the bit, as are
    the results that consist of it alone (products of integers in fp32)."""
    for seed in range(4):
        z, norm = _nearly_orthogonal(side, length, seed)
        x = z.float().cuda()
        y = M.orthogonalize(x.mT.contiguous() if turned else x, steps=1, coefficients=(0.0, 1.0, 0.0), dtype=F32)
        y = (y.mT if turned else y).double().cpu() * float(norm) ** 3
        alone = (z[0] == 0) & (z[1] != 0)
        assert int(alone.sum()) > length // 5
        assert torch.equal(y[0][alone], z[1][alone].double())


# ------------------------------------------------------------------ workspaces --

@pytest.mark.parametrize("tokens", [1, A.EXPERT_STREAM_ROWS])
def test_few_tokens_need_no_copy_of_the_weights(tokens):
    x, w, at = rand(tokens, 1023), rand(4, 512, 1023, seed=2), offsets_of([0, 0, 1, 1, tokens])
    M.expert_linear(x, w, at)
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    torch.cuda.reset_peak_memory_stats()
    y = M.expert_linear(x, w, at)
    torch.cuda.synchronize()
    assert torch.cuda.max_memory_allocated() - before <= 2 * y.numel() * y.element_size() + 4096
    close(y, products(x, w, [0, 0, 1, 1, tokens]), 1023)
    check(tokens + 1, 512, 1023, [0, 0, 1, 1, tokens + 1], w=w)   # one more does


# ------------------------------------------- the C entry points by themselves --

def _workspace(nbytes):
    return torch.full((max(nbytes, 1) + 512,), 255, dtype=torch.uint8, device="cuda")   # NaN wherever it is read first


@pytest.mark.parametrize("dtype", [BF, HALF, F32], ids=str)
@pytest.mark.parametrize("n,k", [(64, 96), (33, 45), (300, 264)])
@pytest.mark.parametrize("tokens", [5, 300])
def test_outer_is_what_backward_gives(dtype, n, k, tokens):
    """adamw_expert_outer, with a workspace of exactly its size: the same bits as
    adamw_expert_backward's gradient, and as sums in 64 bits say; added too, and
    exchanged (the gradient of transposed weights)."""
    ends = [0, tokens // 3, tokens // 3, tokens - 1]
    dy, x, at = rand(tokens, n, seed=3), rand(tokens, k), offsets_of(ends)
    w = rand(3, n, k, seed=2)
    nbytes = A.adamw_expert_workspace(M._matrices(dy), M._matrices(x))
    assert (nbytes > 0) == (n % 8 > 0)
    work = _workspace(nbytes)
    stream = torch.cuda.current_stream().cuda_stream
    for exchanged in (False, True):
        left, right = (x, dy) if exchanged else (dy, x)
        dw = torch.full((3, left.shape[1], right.shape[1]), 7.0, dtype=dtype, device="cuda")
        ref = torch.full_like(dw, 3.0)
        view = ref.mT if exchanged else ref
        for accumulate in (0, 1):
            before = dw.double()
            A.adamw_expert_outer(M._matrices(left), M._matrices(right), at.data_ptr(), M._matrices(dw), accumulate, work.data_ptr(), stream)
            M.expert_linear_backward(dy, x, w, at, need=(False, True), d_weight=view, accumulate=bool(accumulate))
            assert torch.equal(dw, ref)
            want, size = outer(left, right, ends)
            close(dw, (want + before, size + before.abs()) if accumulate else (want, size), tokens)
        assert (work[nbytes:] == 255).all()


@pytest.mark.parametrize("dtype", [BF, HALF], ids=str)
@pytest.mark.parametrize("n,k", [(64, 96), (33, 45), (300, 264)])
@pytest.mark.parametrize("tokens", [5, 16, 300])
def test_transposed_rows_are_what_backward_gives(dtype, n, k, tokens):
    """adamw_expert_rows of the gradient of y, w taken transposed: dx, to the bit."""
    ends = [1, tokens // 3, tokens // 3, tokens - 1]
    dy, w, at = rand(tokens, n, dtype=dtype, seed=3), rand(3, n, k, dtype=dtype, seed=2), offsets_of(ends)
    nbytes = A.adamw_expert_workspace(M._matrices(dy), M._matrices(w))
    work = _workspace(nbytes)
    dx = torch.full((tokens, k), 7.0, dtype=dtype, device="cuda")
    A.adamw_expert_rows(M._matrices(dy), M._matrices(w), 1, at.data_ptr(), M._matrices(dx), work.data_ptr(),
                        torch.cuda.current_stream().cuda_stream)
    assert torch.equal(dx, M.expert_linear_backward(dy, rand(tokens, k, dtype=dtype), w, at, need=(True, False))[0])
    close(dx, products(dy, w.mT, ends), n)
    assert (work[nbytes:] == 255).all()
    # and of weights that lie transposed, as they are
    y = torch.full((tokens, n), 7.0, dtype=F32, device="cuda")
    turned, x = w.mT.contiguous(), rand(tokens, k, dtype=dtype)
    work = _workspace(A.adamw_expert_workspace(M._matrices(x), M._matrices(turned)))
    A.adamw_expert_rows(M._matrices(x), M._matrices(turned), 1, at.data_ptr(), M._matrices(y), work.data_ptr(),
                        torch.cuda.current_stream().cuda_stream)
    close(y, products(x, w, ends), k)


# --------------------------------------------------------------------- results --

def test_results_that_require_a_gradient_are_refused():
    """As an in-place write to them is by torch."""
    x, w, at = rand(6, 8), rand(2, 4, 8, seed=2), offsets_of([0, 3, 6])
    leaf = torch.zeros(6, 4, dtype=BF, device="cuda").requires_grad_()
    for out in (leaf, leaf * 1):
        keep = out.detach().clone()
        with pytest.raises(RuntimeError, match="gradient"):
            M.expert_linear(x, w, at, out=out)
        assert torch.equal(out, keep)
    with torch.no_grad():
        M.expert_linear(x, w, at, out=leaf)
    close(leaf.detach(), products(x, w, [0, 3, 6]), 8)


# --------------------------------------------------- rows that end inside 16 bytes --

@pytest.mark.parametrize("dtype", [BF, HALF, F32], ids=str)
@pytest.mark.parametrize("cols", [40, 41, 44, 47, 255, 258])
@pytest.mark.parametrize("tokens", [5, 17, 300])
def test_what_lies_behind_a_row_stays(dtype, cols, tokens):
    """Results in views of wider rows, at strides that TMA could take: y, the weights'
    gradient either way round, and ends of memory."""
    k, ends = 72, [0, tokens // 2, tokens]
    x, w, dy, at = rand(tokens, k), rand(2, cols, k, seed=2), rand(tokens, cols, seed=3), offsets_of(ends)
    wide = (cols + 7) // 8 * 8
    flat = torch.full((tokens * wide + 64,), 5.0, dtype=dtype, device="cuda")
    y = flat.as_strided((tokens, cols), (wide, 1))
    M.expert_linear(x, w, at, out=y)
    close(y, products(x, w, ends), k)
    flat.as_strided((tokens, cols), (wide, 1)).fill_(5.0)
    assert (flat == 5).all()
    flat = torch.full((2 * 72 * max(wide, 72) * 4 + 64,), 5.0, dtype=dtype, device="cuda")
    for view in (flat.as_strided((2, k, cols), (k * wide, wide, 1)).mT, flat.as_strided((2, cols, k), (cols * 72, 72, 1))):
        M.expert_linear_backward(dy, x, w, at, need=(False, True), d_weight=view)
        close(view, outer(dy, x, ends), tokens)
        view.fill_(5.0)
        assert (flat == 5).all()
    # one row, whose end is the next parameter's beginning
    M.expert_linear_backward(dy, x[:, :1], w[:1, :, :1], offsets_of([0, tokens]), need=(False, True), d_weight=flat[:cols].view(1, 1, cols).mT)
    close(flat[:cols].view(1, 1, cols).mT, outer(dy, x[:, :1], [0, tokens]), tokens)
    assert (flat[cols:] == 5).all()


@pytest.mark.parametrize("dtype", [BF, HALF], ids=str)
@pytest.mark.parametrize("tokens", [9, 300])
@pytest.mark.parametrize("n,k", [(64, 41), (61, 45), (61, 127), (33, 264)])
def test_what_lies_behind_a_row_does_not_matter(dtype, tokens, n, k):
    """NaN between rows of operands that TMA reads as they lie: the same bits as of
    contiguous ones."""
    def padded(*shape, seed):
        t = torch.full((*shape[:-1], (shape[-1] + 7) // 8 * 8 + 8), float("nan"), dtype=dtype, device="cuda")
        t[..., :shape[-1]] = rand(*shape, dtype=dtype, seed=seed)
        return t[..., :shape[-1]]

    x, w, dy, at = padded(tokens, k, seed=1), padded(2, n, k, seed=2), padded(tokens, n, seed=3), offsets_of([0, tokens // 2, tokens])
    args = [t.clone(memory_format=torch.contiguous_format) for t in (dy, x, w)]
    y, want = M.expert_linear(x, w, at), M.expert_linear(args[1], args[2], at)
    assert torch.equal(y, want) or tokens <= A.EXPERT_STREAM_ROWS
    close(y, products(args[1], args[2], [0, tokens // 2, tokens]), k)
    assert all(torch.equal(a, b) for a, b in zip(M.expert_linear_backward(dy, x, w, at), M.expert_linear_backward(*args, at)))


@pytest.mark.parametrize("dtype", [BF, HALF, F32], ids=str)
@pytest.mark.parametrize("n,k", [(64, 96), (33, 45), (300, 264)])
@pytest.mark.parametrize("room", [0, 3, 8])
def test_results_whose_rows_alternate(dtype, n, k, room):
    """Gradients of three experts, row by row in turn, with or without room between
    them: places between the rows are left as they were."""
    ends = [0, 130, 131, 297]
    x, w, dy, at = rand(300, k), rand(3, n, k, seed=2), rand(300, n, seed=3), offsets_of(ends)
    for turned in (False, True):
        rows, cols = (k, n) if turned else (n, k)
        buffer = torch.full((rows, 3, cols + room), 5.0, dtype=dtype, device="cuda")
        d = buffer.permute(1, 0, 2)[:, :, :cols]
        d = d.mT if turned else d
        want, size = outer(dy, x, ends)
        M.expert_linear_backward(dy, x, w, at, need=(False, True), d_weight=d)
        close(d, (want, size), 300)
        first = d.double()
        M.expert_linear_backward(dy, x, w, at, need=(False, True), d_weight=d, accumulate=True)
        close(d, (want + first, size + first.abs()), 300)
        assert (buffer[:, :, cols:] == 5).all()


@pytest.mark.parametrize("shape", [(3, 64, 96), (3, 300, 200), (3, 100, 45)], ids=str)
def test_orthogonalised_rows_that_alternate(shape):
    x = rand(*shape)
    want = M.orthogonalize(x)
    buffer = torch.full((shape[1], 3, shape[2] + 5), 7.0, dtype=BF, device="cuda")
    y = buffer.permute(1, 0, 2)[:, :, :shape[2]]
    work = torch.empty(A.adamw_orthogonalize_workspace(*shape), dtype=torch.uint8, device="cuda")
    A.adamw_orthogonalize(M._matrices(x), M._matrices(y), A.ortho_options(5, M.COEFFICIENTS, 1e-7), work.data_ptr(),
                          torch.cuda.current_stream().cuda_stream)
    assert torch.equal(y, want) and (buffer[:, :, shape[2]:] == 7).all()


# ---------------------------------------------------------- more than five steps --

@pytest.mark.parametrize("shape", [(24, 100), (64, 128), (100, 300), (300, 500), (512, 1024), (1100, 400)], ids=str)
@pytest.mark.parametrize("steps", [6, 7, 8])
def test_more_steps_of_the_usual_coefficients(shape, steps):
    """p(s) = 3.4445 s - 4.775 s^3 + 2.0315 s^5 is no contraction.  After five steps every
    singular value of these matrices (0.013 of the norm or more, 3.44 times as much a
    step) is in [0.682, 1.2025], p's extrema; a step takes that to [0.682, 1.134], where
    |p'| and the differences that a matrix function has in its place, (p(s) -+ p(t)) /
    (s -+ t), are at most 1.83 (at 1.2025: 3.97, once).  So a step multiplies an error by
    1.83 (the sixth by 3.97) and adds its own 1.1e-3, beginning at TOL after five, all
    relative to a norm that is between 0.682 and 1.2025 times the root of the rank."""
    x = rand(*shape, dtype=F32)
    room = TOL
    for k in range(6, steps + 1):
        room = room * (3.97 if k == 6 else 1.83) + 1.1e-3
    assert off(M.orthogonalize(x, steps=steps, dtype=F32), exact(x, steps)) < room * 1.2025 / 0.682
