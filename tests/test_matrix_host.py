"""Host-side checks of the matrix operators' C ABI: workspace sizes and
refusals.  No GPU: every call here is refused before anything is launched, or
has nothing to do (addresses are never dereferenced)."""
import math

import pytest
import torch

from adamw_optimizer_step_sm_gb300 import adamw_sm as A
from adamw_optimizer_step_sm_gb300 import matrix as M
from adamw_optimizer_step_sm_gb300 import optim as OPT

BAD, MIS, BIG = A.ADAMW_ERR_INVALID_ARG, A.ADAMW_ERR_MISALIGNED, A.ADAMW_ERR_TOO_LARGE
P = 1 << 40   # addresses that are never read
Q, W = 2 << 40, 3 << 40


def _m(**k):
    d = dict(data=P, batch=1, rows=64, cols=96, batch_stride=64 * 96, row_stride=96, dtype=A.DTYPE_BF16, pad_=0)
    d.update(k)
    return A.adamw_matrices_t(*(d[n] for n, _ in A.adamw_matrices_t._fields_))


def _status(f, *args):
    with pytest.raises(A.AdamWError) as e:
        f(*args)
    return e.value.status


# -------------------------------------------------------- orthogonalisation --

def _options(steps=5, coefficients=M.COEFFICIENTS, eps=1e-7):
    return A.ortho_options(steps, coefficients, eps)


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), BAD), (dict(rows=-1), BAD), (dict(cols=-1), BAD), (dict(row_stride=-1), BAD),
    (dict(batch_stride=-1), BAD), (dict(dtype=3), BAD), (dict(dtype=-1), BAD), (dict(data=None), BAD),
    (dict(data=P + 1), MIS), (dict(rows=(1 << 20) + 1), BIG), (dict(cols=(1 << 20) + 1), BIG),
    (dict(batch=(1 << 20) + 1), BIG), (dict(row_stride=1 << 41), BIG),
])
def test_matrices_are_checked(change, status):
    assert _status(A.adamw_orthogonalize, _m(**change), _m(**dict(change, data=change.get("data", Q))), _options(), W) == status


@pytest.mark.parametrize("change", [
    dict(rows=65), dict(cols=95), dict(batch=2), dict(row_stride=95),                  # another shape, rows that overlap
    dict(data=P + 2), dict(data=P, dtype=A.DTYPE_FP16), dict(data=P, row_stride=100),  # overlaps the source
])
def test_orthogonalize_destination(change):
    assert _status(A.adamw_orthogonalize, _m(), _m(**dict(dict(data=Q), **change)), _options(), W) == BAD


@pytest.mark.parametrize("options", [
    dict(steps=0), dict(steps=33), dict(eps=0.0), dict(eps=-1.0), dict(eps=math.nan), dict(eps=math.inf),
    dict(coefficients=(math.nan, 0.0, 0.0)), dict(coefficients=(1.0, math.inf, 0.0)), dict(coefficients=[(1.0, 1.0, 1.0)] * 33),
])
def test_iteration_is_checked(options):
    assert _status(A.adamw_orthogonalize, _m(), _m(data=Q), _options(**options), W) == BAD


def test_orthogonalize_workspace():
    assert _status(A.adamw_orthogonalize, _m(), _m(data=Q), _options(), 0) == BAD
    assert _status(A.adamw_orthogonalize, _m(), _m(data=Q), _options(), W + 16) == MIS
    ws = A.adamw_orthogonalize_workspace
    assert ws(1, 64, 96) % 256 == 0 and ws(1, 64, 96) > 0
    assert ws(2, 2048, 2048) > ws(1, 2048, 2048) >= 10 * 2048 * 2048
    for refused in ((-1, 2, 2), (1, -2, 2), (1, 2, (1 << 20) + 1), ((1 << 20) + 1, 2, 2), (1 << 20, 1 << 20, 1 << 20)):
        assert ws(*refused) == 0
    # nothing to do: nothing is looked at
    for empty in (dict(batch=0), dict(rows=0), dict(cols=0)):
        A.adamw_orthogonalize(_m(data=None, **empty), _m(data=None, **empty), _options(), 0)


def test_three_coefficients_a_step():
    with pytest.raises(ValueError):
        A.ortho_options(5, [(1.0, 2.0)], 1e-7)


# ---------------------------------------------------------------------- Muon --

def _muon(**k):
    d = dict(param=P, grad=Q, momentum=W, master=4 << 40, batch=1, rows=64, cols=96)
    d.update(k)
    return A.adamw_muon_tensor_t(*(d[n] for n, _ in A.adamw_muon_tensor_t._fields_))


def _muon_options(**k):
    d = dict(ortho=_options(), nesterov=1, scale=1, momentum_dtype=A.DTYPE_FP32)
    d.update(k)
    return A.adamw_muon_options_t(*(d[n] for n, _ in A.adamw_muon_options_t._fields_))


@pytest.mark.parametrize("change,status", [
    (dict(batch=-1), BAD), (dict(rows=-1), BAD), (dict(cols=-1), BAD), (dict(param=None), BAD), (dict(grad=None), BAD),
    (dict(momentum=None), BAD), (dict(master=None), BAD), (dict(param=P + 1), MIS), (dict(grad=Q + 1), MIS),
    (dict(momentum=W + 2), MIS), (dict(master=(4 << 40) + 2), MIS), (dict(rows=1 << 21), BIG), (dict(batch=1 << 21), BIG),
    (dict(grad=P), BAD), (dict(momentum=P + 4), BAD), (dict(master=W + 64), BAD),   # buffers that overlap
])
def test_muon_list_is_checked(change, status):
    assert _status(A.adamw_muon_plan_create, [_muon(**change)], _muon_options()) == status


def test_muon_list_of_two():
    other = _muon(param=5 << 40, grad=6 << 40, momentum=7 << 40, master=8 << 40)
    for name in ("param", "grad", "momentum", "master"):
        twice = _muon(param=5 << 40, grad=6 << 40, momentum=7 << 40, master=8 << 40)
        setattr(twice, name, getattr(_muon(), name))
        assert _status(A.adamw_muon_plan_create, [_muon(), twice], _muon_options()) == BAD
    # a list that passes the checks gets as far as the device
    if not torch.cuda.is_available():
        assert _status(A.adamw_muon_plan_create, [_muon(), other], _muon_options()) == A.ADAMW_ERR_CUDA


@pytest.mark.parametrize("change", [dict(nesterov=2), dict(nesterov=-1), dict(scale=2), dict(scale=-1),
                                    dict(momentum_dtype=A.DTYPE_FP16), dict(momentum_dtype=7), dict(ortho=_options(steps=0))])
def test_muon_options_are_checked(change):
    assert _status(A.adamw_muon_plan_create, [_muon()], _muon_options(**change)) == BAD


def test_muon_step_pointers():
    assert _status(A.adamw_muon_step, 0, P, Q) == BAD
    A.adamw_muon_plan_destroy(0)


def test_muon_front_end_refuses():
    p = torch.nn.Parameter(torch.zeros(4, 4, dtype=torch.bfloat16))   # not on a GPU
    with pytest.raises(TypeError):
        OPT.Muon([p])
    for bad in (dict(scale="max"), dict(momentum_dtype=torch.float16)):
        with pytest.raises(ValueError):
            OPT.Muon([p], **bad)
    for bad in (dict(lr=-1.0), dict(momentum=1.0), dict(weight_decay=-0.1), dict(lr=math.nan)):
        with pytest.raises(ValueError):
            OPT.Muon([p], **bad)


# ------------------------------------------------------------------- experts --

def _x(**k):
    return _m(**dict(dict(rows=40, cols=96, row_stride=96), **k))


def _w(**k):
    return _m(**dict(dict(data=Q, batch=4), **k))


def _y(**k):
    return _m(**dict(dict(data=W, rows=40, cols=64, row_stride=64), **k))


@pytest.mark.parametrize("x,w,y,status", [
    (dict(batch=2), {}, {}, BAD), (dict(dtype=A.DTYPE_FP32), {}, {}, BAD), (dict(dtype=A.DTYPE_FP16), {}, {}, BAD),
    (dict(cols=95), {}, {}, BAD), ({}, dict(batch=0), {}, BAD), ({}, {}, dict(cols=63), BAD), ({}, {}, dict(rows=41), BAD),
    ({}, {}, dict(batch=2), BAD), ({}, {}, dict(dtype=5), BAD), ({}, {}, dict(row_stride=63), BAD), (dict(data=None), {}, {}, BAD),
    ({}, dict(data=None), {}, BAD), ({}, {}, dict(data=None), BAD), ({}, dict(batch=1025), {}, BIG),
    (dict(rows=(1 << 30) + 1), {}, dict(rows=(1 << 30) + 1), BIG), (dict(data=P + 1), {}, {}, MIS), ({}, dict(data=Q + 1), {}, MIS),
    ({}, {}, dict(data=W + 1), MIS), ({}, {}, dict(data=P + 2), BAD), ({}, {}, dict(data=Q + 64), BAD),
])
def test_expert_rows_are_checked(x, w, y, status):
    assert _status(A.adamw_expert_rows, _x(**x), _w(**w), 0, 5 << 40, _y(**y)) == status


def test_expert_rows_pointers():
    assert _status(A.adamw_expert_rows, _x(), _w(), 2, 5 << 40, _y()) == BAD
    assert _status(A.adamw_expert_rows, _x(), _w(), 1, 5 << 40, _y()) == BAD       # the transposed sizes do not match
    assert _status(A.adamw_expert_rows, _x(), _w(), 0, 0, _y()) == BAD
    assert _status(A.adamw_expert_rows, _x(), _w(), 0, (5 << 40) + 4, _y()) == MIS
    odd = _x(row_stride=97)
    assert _status(A.adamw_expert_rows, odd, _w(), 0, 5 << 40, _y(), 0) == BAD     # a copy needs the workspace
    assert _status(A.adamw_expert_rows, odd, _w(), 0, 5 << 40, _y(), W + 128) == MIS
    A.adamw_expert_rows(_x(rows=0, data=None), _w(), 0, 0, _y(rows=0, data=None))  # no rows: nothing to do


@pytest.mark.parametrize("dy,x,dw,status", [
    (dict(rows=41), {}, {}, BAD), (dict(dtype=A.DTYPE_FP16), {}, {}, BAD), ({}, {}, dict(rows=63), BAD), ({}, {}, dict(cols=95), BAD),
    ({}, {}, dict(batch=0), BAD), ({}, {}, dict(row_stride=95), BAD), ({}, {}, dict(batch_stride=64 * 96 - 1), BAD),
    ({}, {}, dict(batch=1025), BIG), (dict(batch=2), {}, {}, BAD), ({}, {}, dict(data=P), BAD), ({}, {}, dict(data=(4 << 40) + 8), BAD),
])
def test_expert_outer_is_checked(dy, x, dw, status):
    args = _y(**dict(dict(data=4 << 40), **dy)), _x(**x), 5 << 40, _w(**dw)
    assert _status(A.adamw_expert_outer, *args) == status


def test_expert_backward_is_checked():
    f, big = A.adamw_expert_backward, 6 << 40
    dy, x, w = _y(data=4 << 40), _x(), _w()
    dx, dw = _x(data=W), _w(data=big)
    o = 5 << 40
    for bad, status in ((dict(dy=_y(data=4 << 40, rows=41)), BAD), (dict(x=_x(cols=95)), BAD), (dict(w=_w(rows=63)), BAD), (dict(transposed=2), BAD),
                        (dict(dx=_x(data=W, cols=95)), BAD), (dict(dx=_x(data=4 << 40)), BAD), (dict(dw=_w(data=big, batch=3)), BAD),
                        (dict(dw=_w(data=W)), BAD), (dict(dx=_x(data=P)), BAD), (dict(dw=_w(data=Q)), BAD), (dict(dw_transposed=1), BAD), (dict(dw_transposed=2), BAD), (dict(accumulate=2), BAD),
                        (dict(offsets=0), BAD), (dict(offsets=o + 4), MIS), (dict(dw=_w(data=big, batch=1025)), BIG)):
        args = dict(dy=dy, x=x, w=w, transposed=0, offsets=o, dx=dx, dw=dw, dw_transposed=0, accumulate=0)
        args.update(bad)
        assert _status(f, *args.values()) == status, bad
    odd = _y(data=4 << 40, row_stride=65)
    assert _status(f, odd, x, w, 0, o, dx, dw) == BAD              # a copy needs the workspace
    assert _status(f, odd, x, w, 0, o, dx, dw, 0, 0, W + 128) == MIS
    assert A.adamw_expert_backward_workspace(odd, x, w) == 40 * 64 * 2
    f(dy, x, w, 0, o, None, None)                                  # nothing wanted


def test_expert_workspace():
    ws = A.adamw_expert_workspace
    assert ws(_x(), _w()) == 0
    assert ws(_x(row_stride=97), _w()) == 40 * 96 * 2
    assert ws(_x(data=P + 2), _w(batch_stride=64 * 96 + 1)) == 40 * 96 * 2 + 4 * 64 * 96 * 2
    assert ws(_x(cols=91, row_stride=91), _w(cols=91, row_stride=91)) == 40 * 96 * 2 + 4 * 64 * 96 * 2
    assert ws(_x(dtype=A.DTYPE_FP32), _w()) == 0   # refused by the call


@pytest.mark.parametrize("call", [
    lambda t: M.orthogonalize(t),
    lambda t: M.expert_linear(t, t[None], torch.zeros(2, dtype=torch.int64)),
    lambda t: M.expert_linear_backward(t, t, t[None], torch.zeros(2, dtype=torch.int64)),
])
def test_tensors_are_on_a_gpu(call):
    with pytest.raises(TypeError):
        call(torch.zeros(4, 4, dtype=torch.bfloat16))


def test_status_pointer():
    assert A.load().adamw_matrix_status(None) == BAD
