"""What is measured of the target-side operators of a verify step: the paged
K/V cache's append (norms, rotation, write), its read-back, and the attention
of the flattened verify rows over it.

`run` computes them in plain torch (fp32) where `own` is false and calls the
library where it is true; `exact` states them in fp64, written apart.
"""
import math

import torch

own = False

E4M3_MAX = 448.0
TINY = 2.0 ** -126


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------

def _case(name, kind, B, new, ragged, past, past_min, Hq, Hkv, D, act, cache, page, window=0,
          layout="half", rot=0, norm=False, far=0):
    c = dict(kind=kind, B=B, new=new, ragged=ragged, past=past, past_min=past_min, Hq=Hq, Hkv=Hkv,
             D=D, act=act, cache=cache, page=page, window=window, layout=layout, rot=rot,
             norm=norm, far=far)
    if name:
        c["name"] = name
    return c


def listed():
    return [
        # one new token of one short sequence: the latency of a call
        _case("attend one token", "attend", 1, 1, False, 512, 512, 32, 8, 128, "bf16", "bf16", 64),
        # the single-request step: a full block of K = 16 drafts and the last committed token
        _case("attend single block", "attend", 1, 17, False, 8191, 8191, 32, 8, 128, "bf16",
              "bf16", 64),
        # one new token far into a long sequence: one row per head, a long axis to split
        _case("attend long token", "attend", 1, 1, False, 131071, 131071, 32, 8, 128, "bf16",
              "bf16", 64),
        # the batched step (K = 8), cache lengths of a mixed load, five query heads to a kv head
        _case("attend batched", "attend", 64, 9, False, 4000, 300, 40, 8, 128, "bf16", "bf16", 32),
        # the serving step: verify lengths of the prefix cut (0..6 drafts), 8-bit cache
        _case("attend serving e4m3", "attend", 256, 7, True, 4096, 1, 32, 8, 128, "bf16", "e4m3",
              64),
        # plain decoding of small heads without grouping, fp16
        _case("attend decode f16", "attend", 128, 1, False, 3000, 1, 16, 16, 64, "f16", "f16", 16),
        # a prompt's chunk over what earlier chunks left
        _case("attend chunk", "attend", 2, 2048, False, 6001, 2000, 32, 8, 128, "bf16", "bf16",
              64),
        # the single-request step's writes
        _case("append single block", "append", 1, 17, False, 9000, 9000, 32, 8, 128, "bf16",
              "bf16", 64, rot=128, norm=True, far=0),
        # the stress step's writes (K = 16, lengths of the prefix cut), far positions
        _case("append stress", "append", 512, 17, True, 3000, 1, 32, 8, 128, "bf16", "bf16", 64,
              rot=128, norm=True, far=120000),
        # a long prompt's chunk, quantised as it is written, then read back
        _case("append chunk e4m3", "append", 3, 4099, False, 4000, 1, 32, 8, 128, "bf16", "e4m3",
              64, layout="interleaved", rot=64),
        # one short sequence read back
        _case("read one", "read", 1, 1000, False, 0, 0, 32, 8, 128, "bf16", "bf16", 64),
        # a batch of quantised sequences read back
        _case("read batch e4m3", "read", 64, 3000, True, 0, 0, 32, 8, 128, "bf16", "e4m3", 64),
    ]


def _spread(rng, lo, hi):
    """An integer of [lo, hi], even over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    kind = rng.choice(["attend", "attend", "attend", "append", "read"])
    D = rng.choice([64, 128, 128])
    Hkv = rng.choice([1, 2, 4, 8, 8, 16])
    G = rng.choice([1, 2, 3, 4, 4, 5, 7, 8])
    act = rng.choice(["bf16", "bf16", "f16"])
    cache = rng.choice([act, act, "e4m3"])
    page = rng.choice([16, 32, 64, 128])
    window = 0
    if kind == "attend":
        if rng.random() < 0.7:  # decode and verify steps
            new = rng.randint(1, 17)
            B = _spread(rng, 1, 256)
            past = _spread(rng, 1, max(64, min(100000, 600000 // B)))
        else:                   # chunks of a prompt
            new = _spread(rng, 32, 2500)
            B = rng.randint(1, 3)
            past = _spread(rng, 1, 5000)
        # no dearer than the largest listed ones: products of a chunk, bytes of a cache
        while new > 64 and B * new * (past + new) * Hkv * G * D > 2 * 2048 * 5000 * 32 * 128:
            past, new, B = past // 2 + 1, new * 2 // 3, max(1, B - 1)
        while past > 1 and B * (past + new) * Hkv * D > 256 * 2048 * 8 * 128:
            past //= 2
        if rng.random() < 0.2:
            window = _spread(rng, 1, 4096)
    else:
        B = _spread(rng, 1, 256)
        heads = Hkv if kind == "read" else (G + 2) * Hkv
        most = (64 * 1500 * 8 if kind == "read" else 3 * 4099 * 48) * 128 // (heads * D)
        new = _spread(rng, 1, max(2, min(20000, most // B)))
        past = _spread(rng, 1, 4000)
    return _case("", kind, B, new, rng.random() < 0.5, past, rng.choice([1, past]), Hkv * G, Hkv, D,
                 act, cache, page, window, rng.choice(["half", "interleaved"]),
                 rng.choice([0, 16, 32, D // 2, D, D]), rng.random() < 0.6,
                 rng.choice([0, 0, 100000]))


# --------------------------------------------------------------------------
# what a program has in hand
# --------------------------------------------------------------------------

_DT = {"bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def _lengths(c):
    """(new tokens, tokens in the cache before them) of every request."""
    g = torch.Generator().manual_seed(c["B"] * 1000003 + c["new"] * 101 + c["past"])
    new = [c["new"]] * c["B"]
    if c["ragged"]:
        new = torch.randint(1, c["new"] + 1, (c["B"],), generator=g).tolist()
        new[0] = c["new"]
    lo, hi = min(c["past_min"], c["past"]), c["past"]
    past = torch.randint(lo, hi + 1, (c["B"],), generator=g).tolist()
    past[-1] = hi
    return new, past


def _quantised(x):
    """e4m3 codes and one scale for each row of the last axis."""
    s = (x.abs().amax(-1) / E4M3_MAX).clamp_min(TINY)
    return (x / s[..., None]).to(torch.float8_e4m3fn), s


def prepare(case, seed):
    c = dict(case)
    dev = "cuda"
    g = torch.Generator(device=dev).manual_seed(seed)
    Hq, Hkv, D, ps, B = c["Hq"], c["Hkv"], c["D"], c["page"], c["B"]
    act, cdt = _DT[c["act"]], _DT[c["cache"]]
    new, past = _lengths(c)
    # an append needs only the pages that it writes; attention and reads need all of them
    first = [p // ps if c["kind"] == "append" else 0 for p in past]
    last = [(p + n - 1) // ps for p, n in zip(past, new)]
    far = [c["far"] // ps if c["kind"] == "append" else 0] * B  # positions shifted by whole pages
    used = sum(l - f + 1 for f, l in zip(first, last))
    n_pages = used + used // 8 + 1
    max_pages = max(l + s for l, s in zip(last, far)) + 1
    perm = torch.randperm(n_pages, generator=g, device=dev)[:used].to(torch.int32).cpu()
    table = torch.zeros(B, max_pages, dtype=torch.int32)
    at = 0
    for b in range(B):
        k = last[b] - first[b] + 1
        table[b, first[b] + far[b]:last[b] + far[b] + 1] = perm[at:at + k]
        at += k
    past = [p + f * ps for p, f in zip(past, far)]
    rows = sum(new)
    n_rows = rows + 3  # rows behind the last sequence stay as they are
    start = [0]
    for n in new[:-1]:
        start.append(start[-1] + n)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device=dev)

    st = dict(case=c, new=new, past=past, start=start, act=act, cdt=cdt)
    st["page_table"] = table.to(dev)
    st["row_start"] = torch.tensor(start, dtype=torch.int64, device=dev)
    st["verify_len"] = torch.tensor([n - 1 for n in new], dtype=torch.int32, device=dev)
    st["cache_len"] = torch.tensor(past, dtype=torch.int32, device=dev)
    st["sm_scale"] = 1.0 / math.sqrt(D)
    # keys with a few strong channels, as the norms' weights leave them
    gain = torch.ones(D, device=dev)
    gain[torch.randperm(D, generator=g, device=dev)[:4]] = 3.0
    pool = (n_pages, Hkv, ps, D)
    st["k_scale"] = st["v_scale"] = None
    if c["cache"] == "e4m3":
        st["k_cache"], st["k_scale"] = _quantised(randn(*pool) * gain)
        st["v_cache"], st["v_scale"] = _quantised(randn(*pool))
    else:
        st["k_cache"], st["v_cache"] = (randn(*pool) * gain).to(cdt), randn(*pool).to(cdt)
    if c["kind"] == "attend":
        st["q"] = (randn(n_rows, Hq, D) * 1.5 / gain.sqrt()).to(act)
        st["out"] = torch.zeros(n_rows, Hq, D, dtype=act, device=dev)
    if c["kind"] == "append":
        # the rows of one fused projection
        qkv = (randn(n_rows, (Hq + 2 * Hkv) * D) * 1.7).to(act)
        st["q"] = qkv[:, :Hq * D].view(n_rows, Hq, D)
        st["k"] = qkv[:, Hq * D:(Hq + Hkv) * D].view(n_rows, Hkv, D)
        st["v"] = qkv[:, (Hq + Hkv) * D:].view(n_rows, Hkv, D)
        st["q_out"] = torch.zeros(n_rows, Hq, D, dtype=act, device=dev)
        st["q_norm"] = 1 + 0.1 * randn(D) if c["norm"] else None
        st["k_norm"] = gain + 0.1 * randn(D) if c["norm"] else None
        r = c["rot"]
        st["inv_freq"] = None
        if r:
            i = torch.arange(r // 2, dtype=torch.float64, device=dev)
            st["inv_freq"] = 1e6 ** (-2.0 * i / r)
        st["rope_scale"] = 1.0 if c["layout"] == "half" else 1.125
        st["eps"] = 1e-6
    if c["kind"] == "read" or (c["kind"] == "append" and c["cache"] == "e4m3"):
        st["k_out"] = torch.zeros(n_rows, Hkv, D, dtype=act, device=dev)
        st["v_out"] = torch.zeros(n_rows, Hkv, D, dtype=act, device=dev)
    if own:
        from speculative_decoding_05_b200 import dspark as lib
        st["lib"] = lib
        st["ws"] = lib.workspace(lib.dspark_kv_workspace_size(), dev)
        if c["kind"] == "attend":
            st["ws"] = lib.workspace(
                lib.dspark_attn_workspace_size(B, Hq, Hkv, D, max(new)), dev)
    return st


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------

def _slots(st, b):
    """(page, place in it) of request b's new tokens."""
    ps = st["case"]["page"]
    pos = torch.arange(st["past"][b], st["past"][b] + st["new"][b], device="cuda")
    return st["page_table"][b, pos // ps].long(), pos % ps


def _normed(x, w, eps):
    if w is None:
        return x
    return x * torch.rsqrt((x * x).mean(-1, keepdim=True) + eps) * w


def _rotated(x, cos, sin, rot, interleaved):
    if not rot:
        return x
    if interleaved:
        x1, x2 = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2)
    else:
        x1, x2 = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
    return torch.cat([y, x[..., rot:]], -1)


def _plain_append(st):
    c = st["case"]
    for b in range(c["B"]):
        r0, n = st["start"][b], st["new"][b]
        q, k, v = (st[t][r0:r0 + n].float() for t in ("q", "k", "v"))
        q, k = _normed(q, st["q_norm"], st["eps"]), _normed(k, st["k_norm"], st["eps"])
        if c["rot"]:
            pos = torch.arange(st["past"][b], st["past"][b] + n, device="cuda")
            a = pos.double()[:, None] * st["inv_freq"]  # far angles: in 64 bits
            cos = (a.cos().float() * st["rope_scale"])[:, None, :]
            sin = (a.sin().float() * st["rope_scale"])[:, None, :]
            q = _rotated(q, cos, sin, c["rot"], c["layout"] == "interleaved")
            k = _rotated(k, cos, sin, c["rot"], c["layout"] == "interleaved")
        st["q_out"][r0:r0 + n] = q.to(st["act"])
        page, at = _slots(st, b)
        for x, cache, scale in ((k, "k_cache", "k_scale"), (v, "v_cache", "v_scale")):
            if c["cache"] == "e4m3":
                x, s = _quantised(x)
                st[scale][page, :, at] = s
                st[cache].view(torch.uint8)[page, :, at] = x.view(torch.uint8)
            else:
                st[cache][page, :, at] = x.to(st["cdt"])


def _plain_read(st):
    c = st["case"]
    for b in range(c["B"]):
        r0, n = st["start"][b], st["new"][b]
        page, at = _slots(st, b)
        for cache, scale, out in (("k_cache", "k_scale", "k_out"), ("v_cache", "v_scale", "v_out")):
            if c["cache"] == "e4m3":
                x = st[cache].view(torch.uint8)[page, :, at].view(torch.float8_e4m3fn).float()
                x = x * st[scale][page, :, at][..., None]
            else:
                x = st[cache][page, :, at]
            st[out][r0:r0 + n] = x.to(st["act"])


def _plain_attend(st):
    c = st["case"]
    Hq, Hkv, D, ps = c["Hq"], c["Hkv"], c["D"], c["page"]
    G = Hq // Hkv
    for b in range(c["B"]):
        r0, n, past = st["start"][b], st["new"][b], st["past"][b]
        L = past + n
        pages = st["page_table"][b, :(L + ps - 1) // ps].long()
        k, v = st["k_cache"][pages].float(), st["v_cache"][pages].float()
        if c["cache"] == "e4m3":
            k = k * st["k_scale"][pages][..., None]
            v = v * st["v_scale"][pages][..., None]
        k = k.transpose(0, 1).reshape(Hkv, -1, D)[:, :L]
        v = v.transpose(0, 1).reshape(Hkv, -1, D)[:, :L]
        q = st["q"][r0:r0 + n].float().view(n, Hkv, G, D).permute(1, 2, 0, 3)  # [Hkv, G, n, D]
        s = torch.matmul(q, k[:, None].transpose(-1, -2)) * st["sm_scale"]
        pos = torch.arange(past, L, device="cuda")[:, None]
        key = torch.arange(L, device="cuda")[None, :]
        hidden = key > pos
        if c["window"]:
            hidden = hidden | (key <= pos - c["window"])
        s = s.masked_fill(hidden, float("-inf"))
        p = (s - s.amax(-1, keepdim=True)).exp()
        o = torch.matmul(p, v[:, None]) / p.sum(-1, keepdim=True)
        st["out"][r0:r0 + n] = o.permute(2, 0, 1, 3).reshape(n, Hq, D).to(st["act"])


def run(st):
    c = st["case"]
    kind = c["kind"]
    if own:
        lib = st["lib"]
        if kind == "attend":
            lib.dspark_attn_verify(st["q"], st["k_cache"], st["v_cache"], st["row_start"],
                                   st["verify_len"], st["cache_len"], st["page_table"], st["out"],
                                   st["ws"], max_len=c["new"], k_scale=st["k_scale"],
                                   v_scale=st["v_scale"], sm_scale=st["sm_scale"],
                                   window=c["window"])
        if kind == "append":
            lib.dspark_kv_append(st["q"], st["k"], st["v"], st["row_start"], st["verify_len"],
                                 st["cache_len"], st["page_table"], st["k_cache"], st["v_cache"],
                                 st["q_out"], st["ws"], k_scale=st["k_scale"],
                                 v_scale=st["v_scale"], q_norm=st["q_norm"], k_norm=st["k_norm"],
                                 eps=st["eps"], inv_freq=st["inv_freq"],
                                 interleaved=c["layout"] == "interleaved",
                                 rope_scale=st["rope_scale"])
        if "k_out" in st:
            lib.dspark_kv_read(st["k_cache"], st["v_cache"], st["row_start"], st["verify_len"],
                               st["cache_len"], st["page_table"], st["k_out"], st["v_out"],
                               st["ws"], k_scale=st["k_scale"], v_scale=st["v_scale"])
    else:
        if kind == "attend":
            _plain_attend(st)
        if kind == "append":
            _plain_append(st)
        if "k_out" in st:
            _plain_read(st)
    if kind == "attend":
        return {"out": st["out"]}
    if kind == "read":
        return {"k": st["k_out"], "v": st["v_out"]}
    if c["cache"] == "e4m3":  # the written rows, as the values that their codes stand for
        return {"q": st["q_out"], "k": st["k_out"], "v": st["v_out"]}
    return {"q": st["q_out"], "k_cache": st["k_cache"], "v_cache": st["v_cache"]}


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------

def _codes64(x):
    """The value that x (fp64, one row on the last axis) has in the e4m3 cache: the
    nearest of the format's values (3 bits of mantissa, smallest step 2^-9, ties to
    even) times the row's scale."""
    s = torch.clamp_min(x.abs().amax(-1, keepdim=True) / E4M3_MAX, TINY).float().double()
    y = x / s
    e = torch.floor(torch.log2(y.abs().clamp_min(2.0 ** -20))).clamp_min(-6.0)
    step = torch.exp2(e - 3.0)
    return (torch.round(y / step) * step).clamp(-E4M3_MAX, E4M3_MAX) * s


def exact(case, seed):
    st = prepare(case, seed)
    c = st["case"]
    Hq, Hkv, D, ps, B = c["Hq"], c["Hkv"], c["D"], c["page"], c["B"]
    G = Hq // Hkv
    # request and position of every row, then its place in the pool
    req = torch.cat([torch.full((n,), b) for b, n in enumerate(st["new"])]).cuda()
    pos = torch.cat([torch.arange(p, p + n) for p, n in zip(st["past"], st["new"])]).cuda()
    rows = len(req)
    page = st["page_table"][req, pos // ps].long()
    slot = pos % ps
    if c["kind"] == "read":
        res = {}
        for name in "kv":
            o = torch.zeros(st[name + "_out"].shape, dtype=torch.float64, device="cuda")
            x = st[name + "_cache"].to(torch.float32)[page, :, slot].double()
            if st[name + "_scale"] is not None:
                x = x * st[name + "_scale"][page, :, slot].double()[..., None]
            o[:rows] = x
            res[name] = o
        return res
    if c["kind"] == "append":
        def turned(x, w):
            x = x[:rows].double()
            if w is not None:
                x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / D + st["eps"]) * w.double()
            if c["rot"]:
                h = c["rot"] // 2
                i = torch.arange(h, device="cuda")
                first, second = (2 * i, 2 * i + 1) if c["layout"] == "interleaved" else (i, i + h)
                z = torch.polar(torch.full((rows, h), float(st["rope_scale"]), dtype=torch.float64,
                                           device="cuda"),
                                pos.double()[:, None] * st["inv_freq"])
                z = torch.complex(x[..., first], x[..., second]) * z[:, None]
                x = x.clone()
                x[..., first], x[..., second] = z.real, z.imag
            return x

        q = torch.zeros(st["q_out"].shape, dtype=torch.float64, device="cuda")
        q[:rows] = turned(st["q"], st["q_norm"])
        k, v = turned(st["k"], st["k_norm"]), st["v"][:rows].double()
        if c["cache"] == "e4m3":
            ko = torch.zeros(st["k_out"].shape, dtype=torch.float64, device="cuda")
            vo = ko.clone()
            ko[:rows], vo[:rows] = _codes64(k), _codes64(v)
            return {"q": q, "k": ko, "v": vo}
        kc, vc = st["k_cache"].double(), st["v_cache"].double()
        kc[page, :, slot], vc[page, :, slot] = k, v
        return {"q": q, "k_cache": kc, "v_cache": vc}
    out = torch.zeros(st["out"].shape, dtype=torch.float64, device="cuda")
    for b in range(B):
        L = st["past"][b] + st["new"][b]
        j = torch.arange(L, device="cuda")
        pages = st["page_table"][b, :(L + ps - 1) // ps].long()
        mine = (req == b).nonzero()[:, 0]
        for h in range(Hkv):
            kv = {}
            for name in "kv":
                if c["cache"] == "e4m3":
                    x = st[name + "_cache"].view(torch.uint8)[pages, h]
                    x = x.view(torch.float8_e4m3fn).float().double()
                    x = x * st[name + "_scale"][pages, h].double()[..., None]
                else:
                    x = st[name + "_cache"][pages, h].double()
                kv[name] = x.flatten(0, 1)[:L]
            k, v = kv["k"], kv["v"]
            far = pos[mine][:, None] - j[None, :]
            seen = (far >= 0) & (far < c["window"]) if c["window"] else far >= 0
            for x in range(h * G, (h + 1) * G):
                s = torch.einsum("id,jd->ij", st["q"][mine, x].double(), k) * st["sm_scale"]
                s = torch.where(seen, s, torch.full_like(s, -math.inf))
                out[mine, x] = torch.softmax(s, -1) @ v
    return {"out": out}


# --------------------------------------------------------------------------
# what a pass cannot do without
# --------------------------------------------------------------------------

def work(case):
    c = case
    new, past = _lengths(c)
    D, Hq, Hkv = c["D"], c["Hq"], c["Hkv"]
    one = 1 if c["cache"] == "e4m3" else 2
    token = 2 * Hkv * (D * one + (4 if c["cache"] == "e4m3" else 0))  # K and V of one token
    rows = sum(new)
    if c["kind"] == "attend":
        pairs, seen = 0, 0
        for n, p in zip(new, past):
            w = c["window"] or p + n
            pairs += sum(min(p + i + 1, w) for i in range(n))
            seen += min(p + n, w + n - 1)
        return {"bytes": 2 * rows * Hq * D * 2 + seen * token, "flops": 4.0 * D * Hq * pairs}
    if c["kind"] == "read":
        return {"bytes": rows * (token + 2 * Hkv * D * 2), "flops": 2.0 * rows * Hkv * D}
    move = rows * (Hq + 2 * Hkv) * D * 2 + rows * Hq * D * 2 + rows * token
    if c["cache"] == "e4m3":  # and read back
        move += rows * (token + 2 * Hkv * D * 2)
    return {"bytes": move, "flops": 12.0 * rows * (Hq + 2 * Hkv) * D}
