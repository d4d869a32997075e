"""Host-side checks of the matrix operators at the ends of what their calls
allow (no GPU; addresses are never dereferenced)."""
import torch

from adamw_optimizer_step_sm_gb300 import adamw_sm as A
from test_matrix_host import BAD, BIG, MIS, P, Q, W, _m, _muon, _muon_options, _options, _status, _w, _x, _y  # noqa: F401


def test_one_matrix_for_all_experts_is_copied_once():
    """Strides of 0 between matrices: one matrix is what the products read, and
    all that an unaligned one takes of the workspace."""
    ws, back = A.adamw_expert_workspace, A.adamw_expert_backward_workspace
    one = 64 * 96 * 2
    assert ws(_x(), _w(batch_stride=0)) == 0
    assert ws(_x(), _w(batch_stride=0, row_stride=97)) == one
    assert ws(_x(), _w(batch_stride=0, data=Q + 2)) == one
    assert ws(_x(), _w(batch_stride=96, row_stride=97)) == 4 * one
    assert back(_y(), _x(), _w(batch_stride=0, row_stride=97)) == one
    assert back(_y(row_stride=65), _x(row_stride=97), _w(batch_stride=0)) == (40 * 64 + 40 * 96) * 2


def test_few_rows_need_a_workspace_for_the_transposed_product_alone():
    """Weights that TMA cannot read: streamed up to ADAMW_EXPERT_STREAM_ROWS rows (the
    call gets as far as the device), copied where they are taken transposed or
    rows are more."""
    few = A.EXPERT_STREAM_ROWS
    odd = _w(row_stride=97)
    if not torch.cuda.is_available():
        assert _status(A.adamw_expert_rows, _x(rows=few), odd, 0, 5 << 40, _y(rows=few), 0) == A.ADAMW_ERR_CUDA
    assert _status(A.adamw_expert_rows, _x(rows=few + 1), odd, 0, 5 << 40, _y(rows=few + 1), 0) == BAD
    back = _m(data=W, rows=few, cols=96, row_stride=96)
    assert _status(A.adamw_expert_rows, _m(rows=few, cols=64, row_stride=64), odd, 1, 5 << 40, back, 0) == BAD


def test_results_have_places_of_their_own():
    """Matrices whose rows alternate pass the checks (and get as far as the device);
    ones that reach into each other do not."""
    apart = [dict(batch=3, batch_stride=96, row_stride=3 * 96), dict(batch=3, batch_stride=100, row_stride=2 * 100 + 96),
             dict(batch=3, rows=1, batch_stride=96, row_stride=0)]
    shared = [dict(batch=3, batch_stride=95, row_stride=3 * 96), dict(batch=3, batch_stride=96, row_stride=3 * 96 - 1),
              dict(batch=3, batch_stride=96, row_stride=0), dict(batch=3, batch_stride=0, row_stride=96), dict(batch=2, batch_stride=64 * 96 - 1), dict(batch=3, rows=1, batch_stride=95)]
    for how, layouts in ((A.ADAMW_ERR_CUDA, apart), (BAD, shared)):
        if how != BAD and torch.cuda.is_available():
            continue
        for layout in layouts:
            rows = layout.get("rows", 64)
            src = _m(batch=layout["batch"], rows=rows)
            assert _status(A.adamw_orthogonalize, src, _m(**dict(layout, data=Q)), _options(), W) == how, layout
            dy, x = _y(cols=rows, row_stride=64), _x(data=4 << 40)
            assert _status(A.adamw_expert_outer, dy, x, 5 << 40, _m(**dict(layout, data=Q))) == how, layout


def test_strides_whose_products_pass_64_bits():
    """Rows of 2^30 at strides of 2^40 reach past 2^64: a batch of them is no less
    refused where its matrices begin inside each other."""
    big = dict(batch=2, rows=1 << 30, cols=8, row_stride=1 << 40, batch_stride=1 << 39, data=Q)
    dy, x = _m(data=4 << 40, rows=4, cols=1 << 30, row_stride=1 << 30), _m(rows=4, cols=8, row_stride=8)
    assert _status(A.adamw_expert_outer, dy, x, 5 << 40, _m(**dict(big, batch=3, batch_stride=4))) == BAD
    assert _status(A.adamw_expert_outer, dy, x, 5 << 40, _m(**dict(big, batch=3, batch_stride=1 << 40))) == BAD
