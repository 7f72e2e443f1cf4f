"""Rows of the paged-cache calls that lie over one another: refused on the host
(CPU; the neighbours that are accepted run in test_gpu_kv_overlap.py)."""
import pytest

from tests.test_kv_cpu import INVALID, UNSUPPORTED, append, attend, lib  # noqa: F401

A = 1 << 24
ROW = 8 * 128 * 2  # bytes of a row of 8 heads


@pytest.mark.parametrize("rows,stride", [(10, 1024), (10, 1536), (1, 1024)])
def test_results_over_the_queries_are_refused(lib, rows, stride):  # noqa: F811
    q_end = A + ((rows - 1) * stride + 1024) * 2
    call = dict(q=A, q_stride=stride, n_rows=rows)
    for out in (A, A + 16, q_end - 16, A - rows * ROW + 16):
        assert attend(lib, out=out, **call) == INVALID
    # behind and before the queries it is another check that refuses
    for out in (q_end, A - rows * ROW):
        assert attend(lib, out=out, D=96, **call) == UNSUPPORTED


def test_rotated_queries_over_the_inputs_are_refused(lib):  # noqa: F811
    """q_out over a fused projection's rows: blocks would read what others wrote.
    (In place, q_out = q with contiguous rows, is the one exception.)"""
    far = A << 4
    fused = dict(q=A, k=A + ROW, v=A + ROW + 512, q_stride=1536, k_stride=1536, v_stride=1536)
    end = A + 10 * 1536 * 2
    for out in (A, A + ROW, A + 1536 * 2, end - 16):
        assert append(lib, out=out, **fused) == INVALID
    for name in ("q", "k", "v"):
        apart = dict(dict(q=far, k=2 * far, v=3 * far), **{name: A})
        assert append(lib, out=A + 16, **apart) == INVALID
        if name != "q":
            assert append(lib, out=A, **apart) == INVALID
