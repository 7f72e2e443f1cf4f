"""dspark_kv_append and dspark_kv_read against the fp64 statement of
tests/kv_reference.py."""
import pytest
import torch

from speculative_decoding_05_b200 import dspark as D

from tests.kv_reference import Problem, append_rows, half_step, quantise

pytestmark = pytest.mark.gpu

BF, HF, E4 = torch.bfloat16, torch.float16, torch.float8_e4m3fn
TYPES = [(BF, BF), (HF, HF), (BF, E4), (HF, E4)]


def ws_new():
    ws = D.workspace(D.dspark_kv_workspace_size(), "cuda")
    ws.fill_(0xA5)
    return ws


def rows_for(p, seed, size=2.0):
    """q, k, v as slices of one fused projection."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = (torch.randn(p.n_rows, (p.Hq + 2 * p.Hkv) * p.D, generator=g, device="cuda") * size).to(p.act)
    a, b = p.Hq * p.D, (p.Hq + p.Hkv) * p.D
    return (x[:, :a].view(p.n_rows, p.Hq, p.D), x[:, a:b].view(p.n_rows, p.Hkv, p.D),
            x[:, b:].view(p.n_rows, p.Hkv, p.D))


def append(p, q, k, v, q_out=None, ws=None, **kw):
    q_out = torch.full((p.n_rows, p.Hq, p.D), 7.0, dtype=p.act, device="cuda") if q_out is None \
        else q_out
    ws = ws_new() if ws is None else ws
    D.dspark_kv_append(q, k, v, *p.markers(), p.k_cache, p.v_cache, q_out, ws, k_scale=p.k_scale,
                       v_scale=p.v_scale, **kw)
    torch.cuda.synchronize()
    return q_out, ws


def close(got, want, x_abs, act):
    """One rounding to act; fp32 arithmetic before it: the norm's sum of D
    squares, root and products, the angle's cosine and sine (each within
    2^-21 of 1) on the row's two elements: 2^-17 of their size covers them."""
    tol = half_step(act) * want.abs() + 2.0 ** -17 * x_abs + (2.0 ** -25 if act == HF else 0)
    return bool(((got.double() - want).abs() <= tol).all())


def run(p, seed=0, q_norm=None, k_norm=None, eps=1e-6, inv_freq=None, interleaved=False,
        rope_scale=1.0):
    q, k, v = rows_for(p, seed)
    before = {n: getattr(p, n).clone() for n in ("k_cache", "v_cache", "k_scale", "v_scale")
              if getattr(p, n) is not None}
    q_out, ws = append(p, q, k, v, q_norm=q_norm, k_norm=k_norm, eps=eps, inv_freq=inv_freq,
                       interleaved=interleaved, rope_scale=rope_scale)
    assert D.dspark_get_device_flags(ws) == 0
    left = torch.ones(p.n_rows, dtype=torch.bool, device="cuda")
    free = torch.ones(p.n_pages, p.page, dtype=torch.bool, device="cuda")
    for b in range(len(p.new)):
        if p.new[b] == 0:
            continue
        rows = p.rows_of(b)
        left[rows] = False
        pos = torch.arange(p.past[b], p.past[b] + p.new[b], device="cuda")
        args = (eps, pos, inv_freq, interleaved, rope_scale)
        want_q = append_rows(q[rows], q_norm, *args)
        want_k = append_rows(k[rows], k_norm, *args)
        size_q, size_k = (w.abs().amax(-1, keepdim=True) + 1e-30 for w in (want_q, want_k))
        assert close(q_out[rows], want_q, size_q, p.act)
        pg, sl = p.places(b, p.past[b], p.past[b] + p.new[b])
        free[pg, sl] = False
        for name, want, size in (("k", want_k, size_k), ("v", v[rows].double(), None)):
            c, s = getattr(p, name + "_cache"), getattr(p, name + "_scale")
            if s is None:
                got = c[pg, :, sl]
                if size is None:
                    assert torch.equal(got, v[rows])
                else:
                    assert close(got, want, size, p.act)
                continue
            got_s = s[pg, :, sl].double()
            top = want.abs().amax(-1)
            assert bool(((got_s - (top / 448).clamp_min(2.0 ** -126)).abs()
                         <= 2.0 ** -16 * got_s).all())
            code = c.view(torch.uint8)[pg, :, sl].view(E4).float().double()
            # to the nearest code: half a step of the value (relative 2^-4, at
            # least half of 2^-9 scales), plus the fp32 arithmetic before it
            tol = 2.0 ** -4 * want.abs() + 2.0 ** -10 * got_s[..., None] \
                + 2.0 ** -16 * top[..., None]
            assert bool(((code * got_s[..., None] - want).abs() <= tol).all())
            if size is None:
                wc, wsc = quantise(v[rows].float())
                assert torch.equal(code, wc.float().double()) and torch.equal(got_s, wsc.double())
    assert bool((q_out[left] == 7.0).all())
    for n, t in before.items():  # places that no new token has stay as they were
        x, y = getattr(p, n).transpose(1, 2)[free], t.transpose(1, 2)[free]
        assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), n


def freqs(rot, base=1e4):
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)


@pytest.mark.parametrize("act,cache", TYPES)
@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("rot,inter", [(0, False), (16, False), (48, False), (64, False),
                                       (64, True), (32, True), (-1, False), (-1, True)])
def test_append(act, cache, Dh, rot, inter):
    rot = Dh if rot < 0 else rot
    p = Problem([1, 7, 0, 17, 65], [0, 63, 5, 700, 30], 6, 2, Dh, act, cache, 32, seed=rot)
    g = torch.Generator(device="cuda").manual_seed(5)
    w = [1 + 0.2 * torch.randn(Dh, generator=g, device="cuda") for _ in range(2)]
    f = freqs(rot) if rot else None
    run(p, 1, inv_freq=f, interleaved=inter)
    run(p, 2, q_norm=w[0], k_norm=w[1], inv_freq=f, interleaved=inter, rope_scale=1.25)
    run(p, 3, k_norm=w[1], eps=0.1)
    run(p, 4, q_norm=w[0], eps=0.0)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (32, 8), (7, 7), (128, 1), (5, 5), (1024, 2)])
@pytest.mark.parametrize("page", [16, 256])
def test_append_head_counts(Hq, Hkv, page):
    run(Problem([3, 1, 20], [0, 100, 255], Hq, Hkv, 128, BF, BF, page, seed=1),
        q_norm=torch.ones(128, device="cuda"), inv_freq=freqs(128))
    run(Problem([3, 1, 20], [0, 100, 255], Hq, Hkv, 64, BF, E4, page, seed=1),
        k_norm=torch.ones(64, device="cuda"), inv_freq=freqs(64))


def test_far_positions_keep_their_angles():
    """Positions near 2^21: an angle formed in fp32 would be off by 0.1 rad."""
    page = 256
    p = Problem([40], [0], 4, 2, 128, page=page, seed=2, max_pages=(1 << 21) // page + 8)
    far = (1 << 21) + 100
    p.page_table[0, far // page:far // page + 1] = p.page_table[0, 0]
    p.past[0] = far
    p.cache_len[0] = far
    run(p, inv_freq=freqs(128, 1e6))


def test_many_requests_and_long_rows():
    g = torch.Generator().manual_seed(3)
    new = torch.randint(0, 4, (4096,), generator=g).tolist()
    past = torch.randint(0, 20, (4096,), generator=g).tolist()
    run(Problem(new, past, 4, 2, 64, page=16, seed=4), inv_freq=freqs(64))
    run(Problem([5000, 0, 1], [10, 0, 0], 8, 2, 128, BF, E4, 64, seed=5), inv_freq=freqs(128))


def test_query_rows_in_place():
    p = Problem([9, 2], [10, 0], 8, 2, 128, seed=6)
    q, k, v = rows_for(p, 1)
    out, _ = append(p, q, k, v, inv_freq=freqs(128))
    own = q.contiguous()
    append(p, own, k, v, q_out=own, inv_freq=freqs(128))
    for b in range(2):
        assert torch.equal(own[p.rows_of(b)], out[p.rows_of(b)])


def test_e4m3_rows_of_zeros_tiny_and_not_finite_values():
    """A row of zeros, one of subnormal fp32 size, one with an infinity (its
    scale is NaN, its codes 0), in bf16 where such values exist."""
    p = Problem([5], [0], 2, 1, 64, BF, E4, 16, seed=7)
    q, k, v = (t.clone() for t in rows_for(p, 1))
    r = p.start[0]
    v[r + 1] = 0
    v[r + 2] = 2.0 ** -130
    v[r + 3, 0, 5] = float("inf")
    v[r + 4, 0, 6] = float("nan")
    _, ws = append(p, q, k, v)
    pg, sl = p.places(0, 0, 5)
    s = p.v_scale[pg, :, sl][:, 0]
    c = p.v_cache.view(torch.uint8)[pg, :, sl][:, 0]
    assert torch.equal(s[1:3], torch.full((2,), 2.0 ** -126, device="cuda"))
    assert int(c[1].max()) == 0
    val = c[2].view(E4).float() * s[2]
    assert bool(((val - 2.0 ** -130).abs() <= 2.0 ** -135).all())
    assert bool(torch.isnan(s[3:]).all()) and int(c[3:].max()) == 0


def test_append_flags_bad_markers_and_pages():
    p = Problem([5, 3, 9], [100, 30, 64], 8, 2, 128, seed=8)
    ref = Problem([5, 3, 9], [100, 30, 64], 8, 2, 128, seed=8)
    q, k, v = rows_for(p, 1)
    append(ref, q, k, v)
    p.verify_len[1] = p.n_rows
    p.page_table[2, 1] = -5
    before = p.k_cache.clone()
    _, ws = append(p, q, k, v)
    assert D.dspark_get_device_flags(ws) == D.FLAG_BAD_LENGTH | D.FLAG_BAD_PAGE
    pg, sl = p.places(0, 100, 105)
    assert torch.equal(p.k_cache[pg, :, sl], ref.k_cache[pg, :, sl])
    changed = (p.k_cache.view(torch.int16) != before.view(torch.int16)).any(-1).any(1)
    want = torch.zeros_like(changed)
    want[pg, sl] = True
    assert not bool((changed & ~want).any())
    p = Problem([5, 3, 9], [100, 30, 64], 8, 2, 128, seed=8)
    append(p, q, k, v, ws=ws)
    assert D.dspark_get_device_flags(ws) == 0


@pytest.mark.parametrize("act,cache", TYPES)
@pytest.mark.parametrize("Dh", [64, 128])
@pytest.mark.parametrize("page", [16, 128])
def test_read(act, cache, Dh, page):
    p = Problem([1, 300, 0, 17], [0, 63, 9, 200], 4, 2, Dh, act, cache, page, seed=9)
    for whole in (False, True):
        new, past = p.new, p.past
        if whole:  # each sequence from its start
            p2 = Problem([n + q for n, q in zip(new, past)], [0] * 4, 4, 2, Dh, act, cache, page,
                         seed=9)
        else:
            p2 = p
        out = [torch.full((p2.n_rows, 2, Dh), 7.0, dtype=act, device="cuda") for _ in range(2)]
        ws = ws_new()
        D.dspark_kv_read(p2.k_cache, p2.v_cache, *p2.markers(), *out, ws, k_scale=p2.k_scale,
                         v_scale=p2.v_scale)
        torch.cuda.synchronize()
        assert D.dspark_get_device_flags(ws) == 0
        left = torch.ones(p2.n_rows, dtype=torch.bool, device="cuda")
        for b in range(4):
            if p2.new[b] == 0:
                continue
            left[p2.rows_of(b)] = False
            pg, sl = p2.places(b, p2.past[b], p2.past[b] + p2.new[b])
            for o, c, s in ((out[0], p2.k_cache, p2.k_scale), (out[1], p2.v_cache, p2.v_scale)):
                if s is None:
                    want = c[pg, :, sl]
                else:
                    want = (c.view(torch.uint8)[pg, :, sl].view(E4).float()
                            * s[pg, :, sl][..., None]).to(act)
                assert torch.equal(o[p2.rows_of(b)], want)
        for o in out:
            assert bool((o[left] == 7.0).all())


def test_read_gives_back_what_append_wrote():
    p = Problem([9, 0, 130], [10, 4, 33], 8, 2, 128, seed=10)
    q, k, v = rows_for(p, 1)
    append(p, q, k, v)
    out = [torch.zeros(p.n_rows, 2, 128, dtype=BF, device="cuda") for _ in range(2)]
    D.dspark_kv_read(p.k_cache, p.v_cache, *p.markers(), *out, ws_new())
    for b in (0, 2):
        assert torch.equal(out[0][p.rows_of(b)], k[p.rows_of(b)])
        assert torch.equal(out[1][p.rows_of(b)], v[p.rows_of(b)])


def test_read_flags_bad_pages():
    p = Problem([70, 3], [0, 30], 8, 2, 128, seed=11, stale=0.25)
    p.page_table[0, 1] = p.n_pages
    out = [torch.zeros(p.n_rows, 2, 128, dtype=BF, device="cuda") for _ in range(2)]
    ws = ws_new()
    D.dspark_kv_read(p.k_cache, p.v_cache, *p.markers(), *out, ws)
    torch.cuda.synchronize()
    assert D.dspark_get_device_flags(ws) == D.FLAG_BAD_PAGE
    assert torch.equal(out[0][p.start[0] + 64:p.start[0] + 70], p.k_cache[0, :, :6].transpose(0, 1))
