"""A whole decode step with the target's attention in it: draft, prefix cut,
one target layer over the ragged verify rows (append, attention, output
projection), LM-head verify, the cache advanced by what was accepted; several
steps, eager and replayed from one CUDA graph.

The layer is checked against fp64 on the rows that the cut chose, and the
replayed steps give the eager ones' tokens bit for bit."""
import pytest
import torch

from speculative_decoding_05_b200 import dspark as D
from speculative_decoding_05_b200 import workloads as WL
from speculative_decoding_05_b200.kv import PagedKV, rope_frequencies
from speculative_decoding_05_b200.step import DSparkStep

from tests.kv_reference import append_rows, half_step

pytestmark = pytest.mark.gpu

BF, E4 = torch.bfloat16, torch.float8_e4m3fn
HQ, HKV, DH, DM = 8, 2, 64, 256


class Target:
    """Embedding, one attention layer, LM head (random weights)."""

    def __init__(self, V, B, K, cache, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def w(*s, scale=1.0):
            return (torch.randn(*s, generator=g, device="cuda") * scale).to(BF)

        self.emb = w(V, DM)
        self.qkv = w(DM, (HQ + 2 * HKV) * DH, scale=DM ** -0.5)
        self.out = w(HQ * DH, DM, scale=(HQ * DH) ** -0.5)
        self.head = w(V, DM, scale=3.0 * DM ** -0.5)
        self.norm = 1 + 0.1 * torch.randn(DH, generator=g, device="cuda")
        f, self.rope_scale = rope_frequencies(DH, 1e4, "yarn", 4.0, original_len=256)
        self.inv_freq = f.cuda()
        self.kv = PagedKV(B, HQ, HKV, DH, 16, 16, dtype=cache, max_len=K + 1)
        n = B * (K + 1)
        self.q_out = torch.zeros(n, HQ, DH, dtype=BF, device="cuda")
        self.att = torch.zeros(n, HQ, DH, dtype=BF, device="cuda")
        self.rows = torch.arange(B, device="cuda") * (K + 1)

    def prefill(self, tokens):
        """Sequences of equal length in chunks of rows, as a prompt is taken in."""
        B, n = tokens.shape
        x = (self.emb[tokens.reshape(-1).long()] @ self.qkv).view(B * n, -1, DH)
        q, k, v = x[:, :HQ], x[:, HQ:HQ + HKV], x[:, HQ + HKV:]
        rows = (torch.arange(B, device="cuda") * n,
                torch.full((B,), n - 1, dtype=torch.int32, device="cuda"))
        self.kv.append(q, k, v, rows, torch.empty(B * n, HQ, DH, dtype=BF, device="cuda"),
                       q_norm=self.norm, k_norm=self.norm, inv_freq=self.inv_freq,
                       rope_scale=self.rope_scale)
        self.kv.cache_len += n

    def hidden(self, prev, drafts, verify_len):
        """Final hidden states of the verify rows: the last token and the drafts."""
        tokens = torch.cat([prev[:, None], drafts], 1).reshape(-1).clamp_min(0).long()
        x = self.emb[tokens]
        p = (x @ self.qkv).view(len(tokens), -1, DH)
        q, k, v = p[:, :HQ], p[:, HQ:HQ + HKV], p[:, HQ + HKV:]
        rows = (self.rows, verify_len)
        self.kv.append(q, k, v, rows, self.q_out, q_norm=self.norm, k_norm=self.norm,
                       inv_freq=self.inv_freq, rope_scale=self.rope_scale)
        self.kv.attend(self.q_out, rows, self.att)
        self.projected = p
        return x + self.att.view(len(tokens), -1) @ self.out


def check_layer(t, before, lens, window=None):
    """The attention rows against fp64 on the layer's own projections and cache."""
    kv = t.kv
    for b in range(kv.B):
        n, past = int(lens[b]) + 1, int(before[b])
        r = slice(int(t.rows[b]), int(t.rows[b]) + n)
        pos = torch.arange(past, past + n, device="cuda")
        q = append_rows(t.projected[r, :HQ], t.norm, 1e-6, pos, t.inv_freq, False, t.rope_scale)
        # (q_out is one rounding of that, plus the fp32 arithmetic before it)
        size = q.abs().amax(-1, keepdim=True)
        assert bool(((t.q_out[r].double() - q).abs()
                     <= half_step(BF) * q.abs() + 2.0 ** -17 * size).all())
        q = t.q_out[r].double()
        at = torch.arange(past + n, device="cuda")
        pg, sl = kv.page_table[b, at // kv.page_size].long(), at % kv.page_size
        ks, vs = [], []
        for c, s, o in ((kv.k_cache, kv.k_scale, ks), (kv.v_cache, kv.v_scale, vs)):
            if s is None:
                o.append(c[pg, :, sl].double())
            else:
                o.append(c.view(torch.uint8)[pg, :, sl].view(E4).float().double()
                         * s[pg, :, sl].double()[..., None])
        for h in range(HQ):
            k, v = ks[0][:, h // (HQ // HKV)], vs[0][:, h // (HQ // HKV)]
            w = (q[:, h] @ k.T * DH ** -0.5).masked_fill(at[None] > pos[:, None], float("-inf"))
            w = torch.softmax(w, -1)
            want, size = w @ v, w @ v.abs()
            # weights and result rounded to 16 bits, fp32 sums (tests/kv_reference.py has
            # the full account): two half steps and 2^-10 for the rest
            assert bool(((t.att[r, h].double() - want).abs()
                         <= (2 * half_step(BF) + 2.0 ** -10) * size + 1e-6).all())


@pytest.mark.parametrize("cache", [BF, E4])
def test_steps_with_the_target_layer_eager_and_replayed(cache):
    B, K, steps = 12, 5, 6
    w = WL.get("serving", V=4096, r=64, B=B, K=K, seed=5)
    inp = WL.make_inputs(w, device="cuda")
    # a cost curve whose knee lies inside the batch's B + B K tokens
    inp["cost_tokens"], inp["cost_ms"] = (
        x.cuda() for x in WL.cost_table(step=6.0, knee=30.0, fixed_ms=2.0, slope=0.05))
    g = torch.Generator(device="cuda").manual_seed(9)
    prompt = torch.randint(0, w.V, (B, 37), generator=g, device="cuda")
    uni = [{n: torch.rand(inp[n].shape, generator=g, device="cuda")
            for n in ("u_draft", "u_accept", "u_res")} for _ in range(steps)]

    def run(graph):
        step = DSparkStep(w.V, w.r, B, K, B * (K + 1), inp["U"].dtype)
        t = Target(w.V, B, K, cache, 3)
        t.prefill(prompt)
        cur = dict(inp, **{n: u.clone() for n, u in uni[0].items()})
        prev = inp["prev_token"].clone()
        ws = D.workspace(D.dspark_verify_lmhead_workspace_size(w.V, w.r, B, K, DM, B * (K + 1)),
                         "cuda")

        def one():
            step.draft(cur, prev_token=prev)
            step.prefix(cur, True)
            hidden = t.hidden(prev, step.tokens, step.verify_len)
            D.dspark_verify_lmhead(hidden, t.head, t.rows, step.verify_len, cur["base"], cur["U"],
                                   cur["W"], prev, cur["inv_temp"], step.tokens, step.p_tok,
                                   step.ref_max, step.ref_sum, cur["u_accept"], cur["u_res"],
                                   step.n_accepted, step.out_tokens, ws,
                                   last_token=step.last_token, draft_bias=step.draft_bias)
            before.copy_(t.kv.cache_len)
            t.kv.advance(step.n_accepted)
            prev.copy_(step.last_token)

        before = torch.zeros_like(t.kv.cache_len)
        cg = None
        if graph:
            saved = [x.clone() for x in (prev, t.kv.cache_len)]
            s = torch.cuda.Stream()
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                one()  # warm-up: attributes and library handles
            torch.cuda.current_stream().wait_stream(s)
            prev.copy_(saved[0])
            t.kv.cache_len.copy_(saved[1])
            cg = torch.cuda.CUDAGraph()
            with torch.cuda.graph(cg):
                one()
            prev.copy_(saved[0])
            t.kv.cache_len.copy_(saved[1])
        trail = []
        for i in range(steps):
            for n, u in uni[i].items():
                cur[n].copy_(u)
            cg.replay() if graph else one()
            torch.cuda.synchronize()
            assert all(f == 0 for f in t.kv.flags().values())
            assert D.dspark_get_device_flags(ws) == 0
            if not graph:
                check_layer(t, before, step.verify_len)
            trail.append((step.tokens.clone(), step.verify_len.clone(), step.n_accepted.clone(),
                          step.out_tokens.clone(), t.kv.cache_len.clone()))
        return trail

    eager, replayed = run(False), run(True)
    for a, b in zip(eager, replayed):
        for x, y in zip(a, b):
            assert torch.equal(x, y)
    lens = torch.stack([s[1] for s in eager])
    assert int(lens.min()) < int(lens.max())  # the cut was ragged


def test_two_graphs_of_one_cache_replayed_in_turn():
    """Append and attention captured twice over the same buffers, with other row
    counts; replays in any order give the eager results."""
    g = torch.Generator(device="cuda").manual_seed(1)
    kv = PagedKV(3, 8, 2, 128, 8, 32, max_len=70)
    f = rope_frequencies(128)[0].cuda()
    runs = []
    for n in (1, 9, 70):
        q = torch.randn(3 * n, 8, 128, generator=g, device="cuda").to(BF)
        k, v = (torch.randn(3 * n, 2, 128, generator=g, device="cuda").to(BF) for _ in range(2))
        rows = (torch.arange(3, device="cuda") * n,
                torch.tensor([n - 1, -1, n // 2 - 1], dtype=torch.int32, device="cuda"))
        qo, out = torch.zeros_like(q), torch.zeros_like(q)

        def call(q=q, k=k, v=v, rows=rows, qo=qo, out=out):
            kv.append(q, k, v, rows, qo, inv_freq=f)
            kv.attend(qo, rows, out)

        runs.append((call, out))
    kv.cache_len.copy_(torch.tensor([100, 7, 33], dtype=torch.int32))
    want = []
    for call, out in runs:
        call()
        want.append(out.clone())
    graphs = []
    for call, out in runs:
        cg = torch.cuda.CUDAGraph()
        with torch.cuda.graph(cg):
            call()
        graphs.append(cg)
    for i in (0, 2, 1, 1, 0, 2):
        runs[i][1].zero_()
        graphs[i].replay()
        torch.cuda.synchronize()
        assert torch.equal(runs[i][1], want[i])
        assert all(x == 0 for x in kv.flags().values())
