"""Rows behind one another in one buffer, which the checks of overlapping rows
must let pass."""
import pytest
import torch

from speculative_decoding_05_b200 import dspark as D

from tests.kv_reference import Problem
from tests.test_gpu_attn import attend
from tests.test_gpu_kv import append, freqs, rows_for

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("before", [False, True])
def test_neighbours_in_one_buffer(before):
    p = Problem([9, 2], [40, 0], 8, 2, 128, seed=51)
    n = p.n_rows
    want, _ = attend(p)
    both = torch.full((2 * n, 8, 128), 7.0, dtype=p.act, device="cuda")
    q, out = (both[n:], both[:n]) if before else (both[:n], both[n:])
    q.copy_(p.q)
    ws = D.workspace(D.dspark_attn_workspace_size(2, 8, 2, 128, 9), "cuda")
    D.dspark_attn_verify(q, p.k_cache, p.v_cache, *p.markers(), out, ws, 9)
    assert torch.equal(out, want) and torch.equal(q, p.q)

    q, k, v = rows_for(p, 1)
    want, _ = append(p, q, k, v, inv_freq=freqs(128))
    both.fill_(7.0)
    own, out = (both[n:], both[:n]) if before else (both[:n], both[n:])
    own.copy_(q)
    append(p, own, k, v, q_out=out, inv_freq=freqs(128))
    assert torch.equal(out, want) and torch.equal(own, q)


def test_results_over_the_queries_are_refused_by_the_binding():
    p = Problem([9], [40], 8, 2, 128, seed=52)
    ws = D.workspace(D.dspark_attn_workspace_size(1, 8, 2, 128, 9), "cuda")
    with pytest.raises(D.DSparkError) as err:
        D.dspark_attn_verify(p.q, p.k_cache, p.v_cache, *p.markers(), p.q, ws, 9)
    assert err.value.code == 1
