"""dspark_attn_verify against the fp64 statement of tests/kv_reference.py
(tolerances derived there): lengths from one token to chunks, odd sizes,
every type, page size and head layout, windows, idle slots, stale and
non-finite slots that no row may see."""
import pytest
import torch

from speculative_decoding_05_b200 import dspark as D

from tests.kv_reference import Problem, attention

pytestmark = pytest.mark.gpu

BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
MARK = 7.0


def attend(p, window=0, sm_scale=None, max_len=None, q=None, ws=None, stream=None):
    max_len = max_len or max(max(p.new), 1)
    out = torch.full((p.n_rows, p.Hq, p.D), MARK, dtype=p.act, device=p.dev)
    if ws is None:
        ws = D.workspace(D.dspark_attn_workspace_size(len(p.new), p.Hq, p.Hkv, p.D, max_len),
                         p.dev)
        ws.fill_(0xA5)
    D.dspark_attn_verify(p.q if q is None else q, p.k_cache, p.v_cache, *p.markers(), out, ws,
                         max_len, k_scale=p.k_scale, v_scale=p.v_scale, sm_scale=sm_scale,
                         window=window, stream=stream)
    return out, ws


def check(p, out, ref):
    left = torch.ones(p.n_rows, dtype=torch.bool, device=p.dev)
    for rows, want, tol in ref:
        got = out[rows].double()
        odd = ~torch.isfinite(want)
        assert torch.equal(odd, ~torch.isfinite(got)), "non-finite results at other places"
        err = torch.where(odd, torch.zeros_like(got), (got - want).abs())
        assert bool((err <= tol.nan_to_num(posinf=0.0)).logical_or(odd).all()), \
            (rows, float(err.max()), float((err / tol).nan_to_num().max()))
        left[rows] = False
    assert bool((out[left] == MARK).all()), "rows that no request claims were written"


def run(p, **kw):
    out, ws = attend(p, **kw)
    torch.cuda.synchronize()
    assert D.dspark_get_device_flags(ws) == 0
    check(p, out, attention(p, sm_scale=kw.get("sm_scale"), window=kw.get("window", 0)))
    return out


TYPES = [(BF, BF), (HF, HF), (BF, E4), (HF, E4)]


@pytest.mark.parametrize("act,cache", TYPES)
@pytest.mark.parametrize("D_", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 8), (8, 2), (10, 2), (7, 1), (48, 3)])
def test_verify_rows(act, cache, D_, Hq, Hkv):
    """A verify step's rows, lengths on both sides of tile and page borders."""
    run(Problem([1, 7, 3, 17, 2], [0, 63, 64, 700, 129], Hq, Hkv, D_, act, cache, 64, seed=1))


@pytest.mark.parametrize("act,cache", TYPES)
@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
def test_page_sizes(act, cache, page):
    run(Problem([5, 1, 9], [page - 2, 3 * page, 1000], 8, 2, 128, act, cache, page, seed=2))
    run(Problem([140, 33], [page + 1, 5], 4, 2, 64, act, cache, page, seed=3))


@pytest.mark.parametrize("past", [0, 1, 15, 16, 63, 64, 65, 127, 128, 129, 255, 257, 1023, 5000])
@pytest.mark.parametrize("cache", [BF, E4])
def test_one_token(past, cache):
    run(Problem([1], [past], 8, 2, 128, BF, cache, 32, seed=4))


@pytest.mark.parametrize("act,cache", TYPES)
@pytest.mark.parametrize("D_", [64, 128])
@pytest.mark.parametrize("n", [31, 64, 129, 400])
def test_chunks(act, cache, D_, n):
    """Chunks of a prompt next to single tokens and idle slots."""
    run(Problem([n, 0, 1, n // 2], [0, 40, 333, 777], 8, 2, D_, act, cache, 64, seed=5))


@pytest.mark.parametrize("G", [1, 3, 6, 16, 128])
def test_group_sizes_in_a_chunk(G):
    run(Problem([70, 9], [130, 2], 2 * G, 2, 128, BF, BF, 64, seed=6))


@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 100, 1000, 100000])
@pytest.mark.parametrize("cache", [BF, E4])
def test_window(window, cache):
    run(Problem([1, 17, 150, 0], [500, 300, 257, 9], 8, 2, 128, BF, cache, 16, seed=7),
        window=window)


def test_idle_batch_and_empty_problem():
    """Slots without rows: nothing is written, nothing is flagged."""
    p = Problem([0, 0, 0], [0, 64, 3], 8, 2, 128, seed=8)
    run(p)
    run(p, max_len=500)
    empty = Problem([0], [0], 8, 2, 128, seed=8)
    D.dspark_attn_verify(empty.q[:0], empty.k_cache, empty.v_cache, *empty.markers(),
                         empty.q[:0].clone(), ws := D.workspace(
                             D.dspark_attn_workspace_size(1, 8, 2, 128, 1), "cuda"), 1)
    assert D.dspark_get_device_flags(ws) == 0


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n", [6, 40, 200])
@pytest.mark.parametrize("D_", [64, 128])
def test_later_tokens_that_are_not_finite_do_not_reach_earlier_rows(bad, n, D_):
    """K and V of a later new token of the same tile may hold anything; rows
    that see it get what it makes of them."""
    p = Problem([n], [200], 8, 2, D_, seed=9)
    pg, sl = p.places(0, 200 + n - 3, 200 + n - 2)
    p.k_cache[pg, 0, sl, 3] = bad
    p.v_cache[pg, 1, sl, 5] = bad
    out, ws = attend(p)
    torch.cuda.synchronize()
    ref = attention(p)
    rows, want, tol = ref[0]
    got = out[rows].double()
    early = slice(0, n - 3)
    assert bool(torch.isfinite(got[early]).all())
    assert bool(((got - want)[early].abs() <= tol[early]).all())
    late_v = got[n - 3:, 4:, 5]          # heads of key head 1 see the V
    assert not bool(torch.isfinite(late_v).any())
    others = torch.arange(D_, device="cuda") != 5
    assert bool(((got - want)[n - 3:, 4:][..., others].abs() <= tol[n - 3:, 4:][..., others]).all())


def test_strided_queries_scale_and_wide_scores():
    """Rows of a fused projection; a scale of its own; scores far apart."""
    p = Problem([9, 140, 1], [100, 0, 1000], 8, 2, 128, seed=10, spread=6.0)
    wide = torch.zeros(p.n_rows, 12 * 128, dtype=BF, device="cuda")
    wide[:, 256:256 + 1024] = p.q.reshape(p.n_rows, -1)
    q = wide[:, 256:256 + 1024].view(p.n_rows, 8, 128)
    assert torch.equal(run(p, q=q, sm_scale=0.5), run(p, sm_scale=0.5))


def test_all_scores_equal_and_first_key_far_above():
    p = Problem([3, 130], [1000, 50], 8, 2, 128, seed=11)
    p.q.zero_()
    run(p)
    p = Problem([3, 130], [1000, 50], 8, 2, 128, seed=11)
    for b in range(2):
        pg, sl = p.places(b, 0, 1)
        p.k_cache[pg, :, sl] = 30.0
    p.q.abs_()
    run(p)


@pytest.mark.parametrize("new,past", [([1] * 40, None), ([5] * 40, None), ([300, 1, 2, 0] * 3, None)])
def test_same_bits_every_time(new, past):
    past = [(37 * i) % 900 for i in range(len(new))]
    p = Problem(new, past, 16, 2, 128, seed=12)
    first = run(p)
    for _ in range(5):
        assert torch.equal(attend(p)[0], first)


def test_one_long_sequence_split_over_the_device():
    run(Problem([1], [70001], 8, 2, 128, seed=13))
    run(Problem([17], [40000], 8, 1, 64, HF, HF, 16, seed=14))
    run(Problem([9], [30000], 40, 2, 128, BF, E4, 64, seed=15))


@pytest.mark.parametrize("max_len", [17, 18, 64, 129, 5000])
def test_bound_on_the_length_chooses_no_other_result(max_len):
    """Whatever kernel the bound chooses, the result holds."""
    run(Problem([17, 1, 0, 5], [90, 1500, 4, 700], 8, 2, 128, seed=16), max_len=max_len)


def test_many_requests():
    g = torch.Generator().manual_seed(3)
    for B, hi in ((700, 400), (4096, 20)):
        new = torch.randint(0, 4, (B,), generator=g).tolist()
        past = torch.randint(0, hi, (B,), generator=g).tolist()
        run(Problem(new, past, 4, 2, 64, page=16, seed=17))


@pytest.mark.parametrize("cache", [BF, E4])
def test_offsets_past_32_bits(cache):
    """Pages whose elements (and bytes) lie past 2^32."""
    Hkv, ps, Dh = 8, 64, 128
    n_pages = (1 << 32) // (Hkv * ps * Dh) + 40
    p = Problem([3, 150], [300, 100], 16, Hkv, Dh, BF, cache, ps, seed=18)
    big = {}
    shift = n_pages - p.n_pages
    for name in ("k_cache", "v_cache", "k_scale", "v_scale"):
        t = getattr(p, name)
        if t is None:
            continue
        b = torch.zeros(n_pages, *t.shape[1:], dtype=t.dtype, device="cuda")
        b.view(torch.uint8)[shift:] = t.view(torch.uint8)
        big[name] = b
    ref = attention(p)
    for name, b in big.items():
        setattr(p, name, b)
    p.page_table += shift
    out, ws = attend(p)
    torch.cuda.synchronize()
    assert D.dspark_get_device_flags(ws) == 0
    check(p, out, ref)


def test_bad_markers_are_flagged_and_idle():
    """Lengths, rows and positions out of range: the request is left out, the
    others hold; the next call's status is clean."""
    def fresh():
        return Problem([5, 3, 9, 2, 4], [100, 30, 64, 0, 7], 8, 2, 128, seed=19)

    def bad(change):
        p = fresh()
        ref = attention(p)
        change(p)
        out, ws = attend(p, max_len=9)
        torch.cuda.synchronize()
        assert D.dspark_get_device_flags(ws) == D.FLAG_BAD_LENGTH
        assert D.dspark_get_device_status(ws) == 5
        check(p, out, [r for i, r in enumerate(ref) if i != 2])
        p = fresh()
        out, ws = attend(p, max_len=9, ws=ws)
        torch.cuda.synchronize()
        assert D.dspark_get_device_flags(ws) == 0
        check(p, out, ref)

    bad(lambda p: p.verify_len.__setitem__(2, 9))
    bad(lambda p: p.verify_len.__setitem__(2, -2))
    bad(lambda p: p.row_start.__setitem__(2, -1))
    bad(lambda p: p.row_start.__setitem__(2, p.n_rows - 8))
    bad(lambda p: p.cache_len.__setitem__(2, -1))
    bad(lambda p: p.cache_len.__setitem__(2, p.page_table.shape[1] * 64 - 8))
    bad(lambda p: p.cache_len.__setitem__(2, 2 ** 31 - 1))


@pytest.mark.parametrize("n,past", [(5, 300), (150, 300)])
@pytest.mark.parametrize("cache", [BF, E4])
def test_bad_pages_read_page_zero(n, past, cache):
    p = Problem([n, 2], [past, 50], 8, 2, 128, BF, cache, 64, seed=20, stale=0.5)
    p.page_table[0, 1] = 0
    ref = attention(p)
    for bad in (-1, p.n_pages, 2 ** 31 - 1, -2 ** 31):
        p.page_table[0, 1] = bad
        out, ws = attend(p)
        torch.cuda.synchronize()
        assert D.dspark_get_device_flags(ws) == D.FLAG_BAD_PAGE
        check(p, out, ref)


def test_other_stream_and_two_calls_at_once():
    p1 = Problem([5] * 20, [37 * i for i in range(20)], 8, 2, 128, seed=21)
    p2 = Problem([200, 3], [50, 2000], 8, 2, 128, seed=22)
    r1, r2 = attention(p1), attention(p2)
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(10):
        with torch.cuda.stream(s1):
            o1, w1 = attend(p1)
        with torch.cuda.stream(s2):
            o2, w2 = attend(p2)
        o3, w3 = attend(p2)
        torch.cuda.synchronize()
        check(p1, o1, r1)
        check(p2, o2, r2)
        check(p2, o3, r2)


@pytest.mark.parametrize("cache", [BF, E4])
@pytest.mark.parametrize("D_", [64, 128])
@pytest.mark.parametrize("G,n", [(1, 9), (4, 7), (5, 9), (4, 17), (4, 90)])
def test_many_short_items_back_to_back(cache, D_, G, n):
    """Items of one to a few key tiles, calls behind each other without a
    pause: the rings pass from item to item and from call to call."""
    g = torch.Generator().manual_seed(G + n)
    B = 250 if n < 90 else 40
    new = torch.randint(0, n + 1, (B,), generator=g).tolist()
    new[0] = n
    past = torch.randint(0, 500, (B,), generator=g).tolist()
    p = Problem(new, past, 4 * G, 4, D_, BF, cache, 32, seed=23)
    first = run(p)
    outs = [attend(p)[0] for _ in range(20)]
    torch.cuda.synchronize()
    for o in outs:
        assert torch.equal(o, first)


@pytest.mark.parametrize("cache", [BF, E4])
@pytest.mark.parametrize("n", [5, 150])
def test_queries_that_are_not_finite_spoil_their_own_rows_only(cache, n):
    """A NaN or an infinity in a query head: that row and head is not a number,
    every other result holds."""
    p = Problem([n, 2], [300, 60], 8, 2, 128, BF, cache, 64, seed=24)
    ref = attention(p)
    bad = [(p.start[0] + 1, 3, float("nan")), (p.start[0] + 2, 6, float("inf")),
           (p.start[1], 0, -float("inf"))]
    for row, h, x in bad:
        p.q[row, h, 17] = x
    out, ws = attend(p)
    torch.cuda.synchronize()
    assert D.dspark_get_device_flags(ws) == 0
    for row, h, _ in bad:
        assert bool(torch.isnan(out[row, h].float()).all())
    for rows, want, tol in ref:
        got = out[rows].double()
        err = (got - want).abs() <= tol
        for row, h, _ in bad:
            if rows.start <= row < rows.stop:
                err[row - rows.start, h] = True
        # (the e4m3 parts of the other rows formed with a bad one: rows one by one)
        assert bool(err.all())


def test_positions_past_the_limit_are_flagged():
    """A table that repeats one page reaches positions that no tile end can hold."""
    p = Problem([3, 2], [40, 50], 8, 2, 128, page=256, seed=25, max_pages=(1 << 22) + 4)
    ref = attention(p)
    p.page_table[0] = 0
    p.cache_len[0] = (1 << 30) - 2
    out, ws = attend(p)
    torch.cuda.synchronize()
    assert D.dspark_get_device_flags(ws) == D.FLAG_BAD_LENGTH
    check(p, out, ref[1:])


def test_rows_formed_one_by_one_over_a_long_sequence():
    """A NaN in V that the rows of a few requests see, 393216 positions before
    their new tokens: such a row is formed by itself, a CTA's for seconds, and
    its waits hold out.  (Every position before the new ones is in one page, so
    that the weights of its keys count 1536 times.)"""
    B, n, D_, reps = 300, 256, 128, 1536
    page, poisoned = n, (40, 41, 42)
    g = torch.Generator(device="cuda").manual_seed(26)
    k = torch.randn(6, 1, page, D_, generator=g, device="cuda").to(BF)
    v = torch.randn(6, 1, page, D_, generator=g, device="cuda").to(BF)
    q = torch.randn(B * n, 1, D_, generator=g, device="cuda").to(BF)
    k[1], v[1] = k[0], v[0]
    v[1, 0, 77, 5] = float("nan")
    table = torch.zeros(B, reps + 1, dtype=torch.int32, device="cuda")
    table[poisoned[0]:poisoned[-1] + 1] = 1
    last = 2 + torch.arange(B, device="cuda") % 4
    table[:, reps] = last.int()
    row_start = torch.arange(B, device="cuda") * n
    same = lambda x: torch.full((B,), x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = torch.full((B * n, 1, D_), MARK, dtype=BF, device="cuda")
    ws = D.workspace(D.dspark_attn_workspace_size(B, 1, 1, D_, n), "cuda")
    D.dspark_attn_verify(q, k, v, row_start, same(n - 1), same(reps * page), table, out, ws, n)
    torch.cuda.synchronize()
    assert D.dspark_get_device_flags(ws) == 0
    for b in (0, 39, *poisoned, 43, 150, B - 1):
        got = out[b * n:(b + 1) * n, 0].double()
        kk = torch.cat([k[0, 0], k[2 + b % 4, 0]]).double()
        vv = torch.cat([v[0, 0], v[2 + b % 4, 0]]).double()
        w = torch.exp(q[b * n:(b + 1) * n, 0].double() @ kk.T / D_ ** 0.5)
        w[:, :page] *= reps
        w[:, page:].tril_()
        w /= w.sum(1, keepdim=True)
        want, mass = w @ vv, w @ vv.abs()
        # half a step of bf16 for the result and, in the tiled kernel, the
        # weights; fp32: scores (128 products, below 8e-5), the weights' and the
        # results' sums (256 + 1537 additions of half a step, 1.1e-4 each),
        # together below 2^-9 of the weighted |V|
        tol = 2.0 ** -8 * (want.abs() + mass) + 2.0 ** -9 * mass
        if b in poisoned:
            assert bool(torch.isnan(got[:, 5]).all())
            got[:, 5] = want[:, 5]
        assert bool(((got - want).abs() <= tol).all()), b
