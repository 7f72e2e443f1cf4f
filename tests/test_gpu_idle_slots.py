"""Idle slots in a captured step: draft, cut, one target layer, LM-head verify
and the cache's advance, with slots that pause for some steps and go on."""
import pytest
import torch

from speculative_decoding_05_b200 import dspark as D
from speculative_decoding_05_b200 import workloads as WL
from speculative_decoding_05_b200.step import DSparkStep

from tests.test_gpu_target_step import BF, DM, E4, Target, check_layer

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", [BF, E4])
def test_a_slot_pauses_and_goes_on(cache):
    B, K, steps = 6, 4, 6
    w = WL.get("serving", V=2048, r=64, B=B, K=K, seed=8)
    inp = WL.make_inputs(w, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    # slot 1 pauses for two steps, slot 4 starts late, slot 5 never runs
    pause = torch.zeros(steps, B, dtype=torch.bool, device="cuda")
    pause[2:4, 1] = pause[:3, 4] = pause[:, 5] = True
    uni = [{n: torch.rand(inp[n].shape, generator=g, device="cuda")
            for n in ("u_draft", "u_accept", "u_res")} for _ in range(steps)]
    step = DSparkStep(w.V, w.r, B, K, B * (K + 1), inp["U"].dtype)
    t = Target(w.V, B, K, cache, 5)
    t.prefill(torch.randint(0, w.V, (B, 21), generator=g, device="cuda"))
    cur = dict(inp, **{n: u.clone() for n, u in uni[0].items()})
    prev = inp["prev_token"].clone()
    idle, before = torch.zeros(B, dtype=torch.bool, device="cuda"), t.kv.cache_len.clone()
    lens = torch.zeros(B, dtype=torch.int32, device="cuda")
    ws = D.workspace(D.dspark_verify_lmhead_workspace_size(w.V, w.r, B, K, DM, B * (K + 1)), "cuda")

    def one():
        before.copy_(t.kv.cache_len)
        step.draft(cur, prev_token=prev)
        step.prefix(cur, True)
        lens.copy_(step.verify_len.masked_fill(idle, -1))
        hidden = t.hidden(prev, step.tokens, lens)
        D.dspark_verify_lmhead(hidden, t.head, t.rows, lens.clamp_min(0), cur["base"], cur["U"],
                               cur["W"], prev, cur["inv_temp"], step.tokens, step.p_tok,
                               step.ref_max, step.ref_sum, cur["u_accept"], cur["u_res"],
                               step.n_accepted, step.out_tokens, ws, last_token=step.last_token,
                               draft_bias=step.draft_bias)
        t.kv.advance(step.n_accepted, (t.rows, lens))
        prev.copy_(torch.where(idle, prev, step.last_token))

    saved = [x.clone() for x in (prev, t.kv.cache_len)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        one()  # warm-up: attributes and library handles
    torch.cuda.current_stream().wait_stream(s)
    cg = torch.cuda.CUDAGraph()
    with torch.cuda.graph(cg):
        one()
    prev.copy_(saved[0])
    t.kv.cache_len.copy_(saved[1])
    for i in range(steps):
        for n, u in uni[i].items():
            cur[n].copy_(u)
        idle.copy_(pause[i])
        pages = {b: t.kv.k_cache[b * 16:(b + 1) * 16].clone() for b in range(B) if pause[i, b]}
        had_len, had_prev = t.kv.cache_len.clone(), prev.clone()
        cg.replay()
        torch.cuda.synchronize()
        assert all(f == 0 for f in t.kv.flags().values())
        assert D.dspark_get_device_flags(ws) == 0
        on = ~pause[i]
        assert torch.equal(lens < 0, pause[i])
        assert torch.equal(before, had_len) and torch.equal(prev[~on], had_prev[~on])
        assert torch.equal(t.kv.cache_len, had_len + torch.where(on, step.n_accepted + 1, 0))
        for b, x in pages.items():
            assert torch.equal(t.kv.k_cache[b * 16:(b + 1) * 16].view(torch.uint8), x.view(torch.uint8))
        check_layer(t, before, lens)
    assert int(t.kv.cache_len[5]) == 21 and int(t.kv.cache_len[1]) > 21
