"""dspark_attn_verify where it can go wrong in ways that random data of one size
do not show: loud rows beside quiet ones, one key far above the others, scores
that rise along the sequence, windows in every kernel, scales that are tiny or
not finite, parts that are lost in the join (bounds: tests/attn_bounds.py)."""
import pytest
import torch

from speculative_decoding_05_b200 import dspark as D

from tests.attn_bounds import attention_rows, put
from tests.kv_reference import Problem
from tests.test_gpu_attn import BF, E4, HF, TYPES, attend

pytestmark = pytest.mark.gpu


def worst(out, ref, skip=None):
    """The largest error over its bound; `skip`: (row, head) pairs left out."""
    most = 0.0
    for rows, want, tol in ref:
        err = (out[rows].double() - want).abs() / (tol + 1e-300)  # (zeros have no bound)
        for row, h in skip or []:
            if rows.start <= row < rows.stop:
                err[row - rows.start, h] = 0
        assert not bool(torch.isnan(err).any())
        most = max(most, float(err.max()))
    return most


def hold(*what):
    over = worst(*what)
    assert over <= 1.0, over


def run(p, **kw):
    out, ws = attend(p, **kw)
    torch.cuda.synchronize()
    assert D.dspark_get_device_flags(ws) == 0
    hold(out, attention_rows(p, kw.get("sm_scale"), kw.get("window", 0)))
    return out


# ---- rows beside each other --------------------------------------------------

@pytest.mark.parametrize("act,big", [(BF, 1e3), (BF, 1e5), (BF, 1e20), (HF, 1e3), (HF, 6e4)])
@pytest.mark.parametrize("D_", [64, 128])
@pytest.mark.parametrize("n", [3, 8, 40])
def test_a_loud_row_leaves_its_neighbours_their_bits(act, big, D_, n):
    """One large finite element in the queries of one token and head: every
    other row holds to the bound of its own elements."""
    p = Problem([n, 2], [300, 60], 8, 2, D_, act, E4, 64, seed=31)
    loud = p.start[0] + n // 2
    p.q[loud, 2, 5] = big
    p.q[loud, 6, 7] = -big
    out, ws = attend(p)
    torch.cuda.synchronize()
    assert D.dspark_get_device_flags(ws) == 0
    assert bool(torch.isfinite(out[loud].float()).all())
    hold(out, attention_rows(p), [(loud, 2), (loud, 6)])


@pytest.mark.parametrize("act", [BF, HF])
def test_rows_of_very_different_sizes(act):
    """Rows scaled by powers of two from 2^-12 to 2^3, each to its own bound."""
    p = Problem([16], [500], 8, 2, 128, act, E4, 32, seed=32)
    r = torch.arange(16, device="cuda")
    p.q[p.rows_of(0)] = (p.q[p.rows_of(0)].float() * torch.exp2(r - 12.0)[:, None, None]).to(act)
    run(p)


# ---- one key far above the others ----------------------------------------------

@pytest.mark.parametrize("act,cache", TYPES)
@pytest.mark.parametrize("n", [2, 100])
def test_many_light_keys_behind_a_heavy_first_one(act, cache, n):
    """The first key has all but 2^-14 of the weight, 4000 others 2^-26 each;
    they alone have values in the other channels."""
    B, L, D_ = 24, 4096, 64
    p = Problem([n] * B, [L - n] * B, 8, 8, D_, act, cache, 64, seed=33)
    p.q.fill_(1.0)
    g = torch.Generator(device="cuda").manual_seed(34)
    for b in range(B):
        k = -1.0 + 0.05 * torch.randn(L, 8, 1, generator=g, device="cuda").expand(L, 8, D_)
        v = 128.0 + 64.0 * torch.rand(L, 8, D_, generator=g, device="cuda")
        v[:, :, 0] = 0
        k, v = k.clone(), v
        k[0], v[0] = 1.25, 0.0
        v[0, :, 0] = 128.0
        put(p, "k", b, 0, k)
        put(p, "v", b, 0, v)
    run(p, sm_scale=0.125)


# ---- scores that rise ------------------------------------------------------------

@pytest.mark.parametrize("act,cache", TYPES)
@pytest.mark.parametrize("D_", [64, 128])
@pytest.mark.parametrize("n,G", [(1, 1), (5, 4), (60, 1), (70, 4)])
@pytest.mark.parametrize("down", [False, True])
def test_scores_that_rise_or_fall_along_the_sequence(act, cache, D_, n, G, down):
    """Keys grow (or shrink) by a factor of 40 over the sequence, so that the
    softmax reference moves again and again: behind the first tile too."""
    past = [1500, 700, 129]
    p = Problem([n, 1, n], past, 2 * G, 2, D_, act, cache, 64, seed=35)
    for b, m in enumerate(p.past):
        L = m + p.new[b]
        x = torch.linspace(0.2, 8.0, L, device="cuda")
        x = (x.flip(0) if down else x)[:, None, None]
        g = torch.Generator(device="cuda").manual_seed(36 + b)
        put(p, "k", b, 0, torch.randn(L, 2, D_, generator=g, device="cuda") * x)
    run(p, sm_scale=1.5 * D_ ** -0.5)


@pytest.mark.parametrize("act,cache", TYPES)
@pytest.mark.parametrize("n", [5, 100])
@pytest.mark.parametrize("at", [0, 127, 128, 300, 511, 700])
def test_one_key_far_above_at_any_place(act, cache, n, at):
    """A key 30 (natural units) above the rest in some tile: the first, a later
    one of either stream."""
    p = Problem([n, n], [800, 700], 4, 2, 128, act, cache, 32, seed=37)
    p.q.abs_()
    for b in range(2):
        size = float(p.q[p.rows_of(b)].float().sum(-1).mean()) * 128 ** -0.5
        put(p, "k", b, at, torch.full((1, 2, 128), 30.0 / size, device="cuda"))
    run(p)


# ---- windows -----------------------------------------------------------------------

@pytest.mark.parametrize("act,cache", TYPES)
@pytest.mark.parametrize("D_", [64, 128])
@pytest.mark.parametrize("window", [1, 2, 16, 100, 127, 128, 129, 300, 100000])
@pytest.mark.parametrize("n,G", [(1, 1), (17, 4), (33, 8)])
def test_windows_in_every_kernel(act, cache, D_, window, n, G):
    """Rows of a step (16-bit caches: up to 80 a head) and of a chunk."""
    run(Problem([n, 1, 0, n, 3], [500, 300, 8, 257, 9], 2 * G, 2, D_, act, cache, 16, seed=38),
        window=window)


@pytest.mark.parametrize("act,cache", TYPES)
def test_window_with_rising_scores(act, cache):
    for n, G in ((9, 4), (60, 4)):
        p = Problem([n, 2], [1500, 700], 2 * G, 2, 128, act, cache, 64, seed=39)
        for b, m in enumerate(p.past):
            L = m + p.new[b]
            x = torch.linspace(0.2, 8.0, L, device="cuda")[:, None, None]
            g = torch.Generator(device="cuda").manual_seed(40 + b)
            put(p, "k", b, 0, torch.randn(L, 2, 128, generator=g, device="cuda") * x)
        for window in (50, 400):
            run(p, window=window)


# ---- values and scales -------------------------------------------------------------

@pytest.mark.parametrize("power", [-40, -60, -75, -90, 60])
@pytest.mark.parametrize("n", [3, 50])
def test_small_and_large_values_keep_their_bits(power, n):
    """V as a whole tiny or huge (scales by 2^power): results are that much."""
    p = Problem([n, 1], [700, 90], 8, 2, 128, BF, E4, 64, seed=41)
    p.v_scale *= 2.0 ** power
    run(p)


@pytest.mark.parametrize("cache,act", [(HF, HF), (BF, BF), (E4, BF), (E4, HF)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n", [4, 70])
@pytest.mark.parametrize("where", ["cached", "new"])
def test_keys_and_values_that_are_not_finite(cache, act, bad, n, where):
    """K of key head 0 and V of key head 1, one element of a 16-bit cache or the
    scale of an e4m3 one, at a cached position that every row sees or at a new
    one that only the last rows see."""
    if cache == E4 and bad < 0:
        pytest.skip("a scale is not negative")
    past = 300
    p = Problem([n], [past], 8, 2, 64, act, cache, 32, seed=42)
    ref = attention_rows(p)[0]
    at = 130 if where == "cached" else past + n - 2
    pg, sl = p.places(0, at, at + 1)
    if cache == E4:
        p.k_scale[pg, 0, sl] = bad
        p.v_scale[pg, 1, sl] = bad
    else:
        p.k_cache[pg, 0, sl, 3] = bad
        p.v_cache[pg, 1, sl, 5] = bad
    out, ws = attend(p)
    torch.cuda.synchronize()
    assert D.dspark_get_device_flags(ws) == 0
    rows, want, tol = ref
    got = out[rows].double()
    sees = torch.arange(n, device="cuda") + past >= at
    ok = (got - want).abs() <= tol
    assert bool(ok[~sees].all())
    late = got[sees]
    if cache == E4:
        assert not bool(torch.isfinite(late[:, 4:]).any())
    else:
        others = torch.arange(64, device="cuda") != 5
        assert not bool(torch.isfinite(late[:, 4:, 5]).any())
        assert bool(ok[sees][:, 4:][..., others].all())
    if bad != bad:
        assert bool(torch.isnan(late[:, :4]).all())
    else:  # an infinite score one way makes a row no number, the other way a weight of 0
        whole = torch.isnan(late[:, :4]).all(-1)
        none = torch.isfinite(late[:, :4]).all(-1)
        assert bool((whole | none).all())
        if cache != E4:
            up = (p.q[rows][sees][:, :4, 3].float() * bad) > 0
            assert torch.equal(whole, up)


# ---- parts -----------------------------------------------------------------------

def mark_tiles(p, b):
    """V with one large value for each 128 keys, in a channel and of a size of
    their own: a tile that is lost, doubled or taken for another shows."""
    L = p.past[b] + p.new[b]
    g = torch.Generator(device="cuda").manual_seed(43)
    v = torch.randn(L, p.Hkv, p.D, generator=g, device="cuda")
    t = torch.arange(L, device="cuda") // 128
    v[torch.arange(L, device="cuda"), :, t % p.D] += (1000.0 + 500.0 * (t // p.D).float())[:, None]
    put(p, "v", b, 0, v)


@pytest.mark.parametrize("n,past,Hq,Hkv,D_,act,cache", [
    (1, 70001, 8, 2, 128, BF, BF), (17, 40000, 8, 1, 64, HF, HF), (9, 30000, 40, 2, 128, BF, E4),
    (2, 9000, 4, 4, 128, HF, E4), (90, 20000, 4, 1, 128, BF, BF), (1, 12800, 1, 1, 64, BF, BF)])
def test_every_part_of_a_long_sequence_counts(n, past, Hq, Hkv, D_, act, cache):
    p = Problem([n], [past], Hq, Hkv, D_, act, cache, 64, seed=44)
    p.q *= 0.25  # no key dominates
    mark_tiles(p, 0)
    out = run(p)
    # the bounds tell: without, or with twice, any whole tile of keys the first
    # row would be out of them
    rows, want, tol = attention_rows(p)[0]
    k, v = p.kv64(0, past + n)
    q = p.q[rows][0, 0].double()
    w = torch.exp(k[:past + 1, 0] @ q * D_ ** -0.5)
    wv = w[:, None] * v[:past + 1, 0]
    tiles = past // 128
    tv = wv[:tiles * 128].view(tiles, 128, D_).sum(1)
    tw = w[:tiles * 128].view(tiles, 128).sum(1, keepdim=True)
    for sign in (-1.0, 1.0):
        o = (wv.sum(0) + sign * tv) / (w.sum() + sign * tw)
        over = ((o - want[0, 0]).abs() / tol[0, 0]).amax(1)
        assert float(over.min()) > 2.0, float(over.min())
    assert bool(torch.isfinite(out[rows].float()).all())


# ---- rows formed one by one over a long sequence, in the step kernel ---------------

@pytest.mark.parametrize("cache,n", [(BF, 80), (E4, 64)])
def test_rows_formed_one_by_one_in_a_step(cache, n):
    """A NaN in V some 390000 positions before the new tokens, seen by all rows
    of two of many requests: their waits hold out (the documented limit is 2^19)."""
    B, page, reps, D_ = 200, 256, 1536, 128
    p = Problem([n] * 4, [page] * 4, 1, 1, D_, BF, cache, page, seed=46, stale=0.0)
    first = p.page_table[:, :2].clone()
    table = first[torch.arange(B, device="cuda") % 4][:, :1].repeat(1, reps)
    table = torch.cat([table, first[torch.arange(B, device="cuda") % 4][:, 1:2]], 1).int().contiguous()
    # request 3's first page again, with a NaN
    src = int(first[3, 0])
    extra = (set(range(p.n_pages)) - set(first.flatten().tolist())).pop()
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        t = getattr(p, name)
        if t is not None:
            t.view(torch.uint8)[extra] = t.view(torch.uint8)[src]
    if cache == E4:
        p.v_scale[extra, 0, 77] = float("nan")
    else:
        p.v_cache[extra, 0, 77, 5] = float("nan")
    poisoned = (43, 107)
    for b in poisoned:
        table[b, :reps] = extra
    q = torch.empty(B * n, 1, D_, dtype=BF, device="cuda")
    for b in range(B):
        q[b * n:(b + 1) * n] = p.q[p.rows_of(b % 4)]
    same = lambda x: torch.full((B,), x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.zeros(B * n, 1, D_, dtype=BF, device="cuda")
    ws = D.workspace(D.dspark_attn_workspace_size(B, 1, 1, D_, n), "cuda")
    D.dspark_attn_verify(q, p.k_cache, p.v_cache, torch.arange(B, device="cuda") * n, same(n - 1),
                         same(reps * page), table, out, ws, n, k_scale=p.k_scale,
                         v_scale=p.v_scale)
    torch.cuda.synchronize()
    assert D.dspark_get_device_flags(ws) == 0
    for b in (0, 42, *poisoned, 44, 108, B - 1):
        r = b % 4
        k, v = (x[:, 0] for x in p.kv64(r, page + n))
        w = torch.exp(q[b * n:(b + 1) * n, 0].double() @ k.T / D_ ** 0.5)
        w[:, :page] *= reps
        w[:, page:].tril_()
        w /= w.sum(1, keepdim=True)
        want, mass = w @ v, w @ v.abs()
        got = out[b * n:(b + 1) * n, 0].double()
        # half a step of bf16 for the result and the weights (fp16 ones of an
        # e4m3 cache have less); scores and sums in fp32, and Q's e4m3 parts:
        # below 2^-9 of the weighted |V|, as in the chunk's test of this kind
        tol = 2.0 ** -8 * (want.abs() + mass) + 2.0 ** -9 * mass
        if b in poisoned:
            if cache == E4:
                assert bool(torch.isnan(got).all())
                continue
            assert bool(torch.isnan(got[:, 5]).all())
            got[:, 5] = want[:, 5]
        assert bool(((got - want).abs() <= tol).all()), b


# ---- the holder --------------------------------------------------------------------

@pytest.mark.parametrize("cache", [BF, E4])
def test_holder_reads_back_and_windows(cache):
    """PagedKV.read of the last append, from a start of its own, and after
    advance; attend with a window."""
    from speculative_decoding_05_b200.kv import PagedKV
    g = torch.Generator(device="cuda").manual_seed(47)
    kv = PagedKV(2, 4, 2, 64, 6, 16, dtype=cache, max_len=20)
    k, v = (torch.randn(40, 2, 64, generator=g, device="cuda").to(BF) for _ in range(2))
    q = torch.randn(40, 4, 64, generator=g, device="cuda").to(BF)
    rows = (torch.tensor([0, 20], device="cuda"),
            torch.tensor([19, 10], dtype=torch.int32, device="cuda"))
    qo = torch.zeros_like(q)
    kv.append(q, k, v, rows, qo)
    out = [torch.full_like(k, 7.0) for _ in range(2)]
    kv.read(rows, *out)
    if cache == BF:
        for o, x in zip(out, (k, v)):
            assert torch.equal(o[:31], x[:31])
    else:
        for o, x in zip(out, (k, v)):
            size = x[:31].float().abs().amax(-1, keepdim=True)
            assert bool(((o[:31].float() - x[:31].float()).abs()
                         <= 2.0 ** -4 * x[:31].float().abs() + 2.0 ** -10 * size / 448
                         + 2.0 ** -8 * size).all())
    assert all(bool((o[31:] == 7.0).all()) for o in out)
    first = [o.clone() for o in out]
    kv.advance(torch.tensor([19, 10], dtype=torch.int32, device="cuda"), rows)
    assert kv.cache_len.tolist() == [20, 11]
    again = [torch.full_like(k, 7.0) for _ in range(2)]
    kv.read(rows, *again, start=torch.zeros(2, dtype=torch.int32, device="cuda"))
    part = (rows[0], torch.tensor([4, 2], dtype=torch.int32, device="cuda"))
    some = [torch.full_like(k, 7.0) for _ in range(2)]
    kv.read(part, *some, start=torch.tensor([3, 8], dtype=torch.int32, device="cuda"))
    for f, a, s in zip(first, again, some):
        assert torch.equal(f, a)
        assert torch.equal(s[:5], f[3:8]) and torch.equal(s[20:23], f[28:31])
        assert bool((s[5:20] == 7.0).all()) and bool((s[23:] == 7.0).all())
    assert all(x == 0 for x in kv.flags().values())
    # one more token a sequence, seen through a window of 4
    one = (torch.tensor([0, 1], device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda"))
    kv.append(q[:2], k[:2], v[:2], one, qo[:2])
    att = torch.zeros(2, 4, 64, dtype=BF, device="cuda")
    kv.attend(qo[:2], one, att, window=4)
    kv4 = [torch.zeros(8, 2, 64, dtype=BF, device="cuda") for _ in range(2)]
    back = (torch.tensor([0, 4], device="cuda"), torch.full((2,), 3, dtype=torch.int32, device="cuda"))
    kv.read(back, *kv4, start=kv.cache_len - 3)
    for b in range(2):
        kk, vv = (x[4 * b:4 * b + 4].double() for x in kv4)
        for h in range(4):
            w = torch.softmax(kk[:, h // 2] @ qo[b, h].double() / 8, 0)
            want, mass = w @ vv[:, h // 2], w @ vv[:, h // 2].abs()
            # weights and result rounded to 16 bits; read-back of e4m3 rounds K and
            # V to bf16 once more (2^-9 of a score of some units each way, and of V)
            tol = (2.0 ** -7 + (2.0 ** -5 if cache == E4 else 0.0)) * mass
            assert bool(((att[b, h].double() - want).abs() <= tol).all())


def test_few_keys_with_rounded_weights():
    """Seven keys of a sharp softmax in bf16: the roundings of the weights do not
    average out, in the product nor in their sum."""
    for seed in range(8):
        p = Problem([17, 6, 11, 17, 0, 1], [1180, 68, 146, 1077, 949, 1123], 4, 2, 64, BF, BF, 256,
                    seed=60 + seed)
        run(p, window=7, sm_scale=1.0)
