"""Plain fp64 statements of the paged-cache calls, and seeded problems for
them (test infrastructure; shares no code with the library)."""
import math

import torch

F64 = torch.float64


def half_step(dtype):
    """Largest relative error of one rounding to dtype."""
    return torch.finfo(dtype).eps / 2


class Problem:
    """Ragged requests over a paged cache.  new[b] tokens (0: an idle slot)
    behind past[b] cached ones; rows of the requests in a shuffled order with
    gaps between them; pages in a random order.  Slots that no request owns
    hold `stale` (NaN by default)."""

    def __init__(self, new, past, Hq, Hkv, D, act=torch.bfloat16, cache=None, page=64, seed=0,
                 device="cuda", stale=float("nan"), gap=1, spread=1.0, max_pages=None):
        g = torch.Generator(device=device).manual_seed(seed)
        self.new, self.past = list(new), list(past)
        self.Hq, self.Hkv, self.D, self.act, self.page = Hq, Hkv, D, act, page
        self.cache = cache or act
        self.dev = device
        B = len(new)
        need = [(p + n + page - 1) // page for p, n in zip(past, new)]
        self.n_pages = sum(need) + 2
        ids = torch.randperm(self.n_pages, generator=torch.Generator().manual_seed(seed))
        table = torch.full((B, max(max_pages or 0, max(need + [1])) + 1), self.n_pages - 1,
                           dtype=torch.int32)
        at = 0
        for b in range(B):
            table[b, :need[b]] = ids[at:at + need[b]].to(torch.int32)
            at += need[b]
        order = torch.randperm(B, generator=torch.Generator().manual_seed(seed + 1)).tolist()
        start, row = [0] * B, gap
        for b in order:
            start[b] = row
            row += self.new[b] + gap
        self.start, self.n_rows = start, row
        self.row_start = torch.tensor(start, dtype=torch.int64, device=device)
        self.verify_len = torch.tensor([n - 1 for n in new], dtype=torch.int32, device=device)
        self.cache_len = torch.tensor(past, dtype=torch.int32, device=device)
        self.page_table = table.to(device)

        def randn(*s):
            return torch.randn(*s, generator=g, device=device)

        shape = (self.n_pages, Hkv, page, D)
        self.q = (randn(self.n_rows, Hq, D) * spread).to(act)
        k, v = randn(*shape) * spread, randn(*shape)
        owned = torch.zeros(self.n_pages, page, dtype=torch.bool, device=device)
        for b in range(B):
            pg, sl = self.places(b, 0, past[b] + new[b])
            owned[pg, sl] = True
        hole = ~owned[:, None, :].expand(self.n_pages, Hkv, page)
        self.k_scale = self.v_scale = None
        if self.cache == torch.float8_e4m3fn:
            self.k_cache, self.k_scale = quantise(k)
            self.v_cache, self.v_scale = quantise(v)
            self.k_scale[hole] = stale
            self.v_scale[hole] = stale
        else:
            k[hole], v[hole] = stale, stale
            self.k_cache, self.v_cache = k.to(self.cache), v.to(self.cache)

    def places(self, b, lo, hi):
        pos = torch.arange(lo, hi, device=self.dev)
        return self.page_table[b, pos // self.page].long(), pos % self.page

    def rows_of(self, b):
        return slice(self.start[b], self.start[b] + self.new[b])

    def kv64(self, b, hi):
        """K and V of request b's first hi positions, [hi, Hkv, D] fp64."""
        pg, sl = self.places(b, 0, hi)
        out = []
        for c, s in ((self.k_cache, self.k_scale), (self.v_cache, self.v_scale)):
            if s is None:
                out.append(c[pg, :, sl].to(F64))
            else:
                x = c.view(torch.uint8)[pg, :, sl].view(torch.float8_e4m3fn).float().to(F64)
                out.append(x * s[pg, :, sl].to(F64)[..., None])
        return out

    def markers(self):
        return self.row_start, self.verify_len, self.cache_len, self.page_table


def quantise(x):
    # torch divides by a Python number through its reciprocal: a true division
    # of the definition goes through fp64
    s = (x.abs().amax(-1).to(F64) / 448.0).float().clamp_min(2.0 ** -126)
    return (x.float() / s[..., None]).to(torch.float8_e4m3fn), s


def attention(p, sm_scale=None, window=0):
    """[(rows, out, tolerance)] per request, in fp64.

    Tolerance, per element d of a row, from the definition's roundings:
    the weights are rounded once to 16 bits (u_p relative each; fp16 also
    absolutely by half its smallest step, 2^-25, against a largest weight of
    at least 1), the sums run in fp32 over n keys (a step of at most 2^-23
    relative to A_d = sum_j w_j |v_jd| each, truncating adders included), a
    score is a fp32 sum of D products (error at most D 2^-23 S, S the largest
    sum of |q k| scale) scaled and turned into 2^x (relative 2^-21 and, of
    |score| <= S, 2^-22 S), which moves weight and normaliser: twice.  Then
    one rounding of the result.

    e4m3: the weights are fp16 with V's scale on them, the largest such product
    at least 1, so half the smallest step is against max|v| again.  Queries are
    sums of e4m3 parts, off by at most 2^-17 of the largest element of the rows
    formed together (at most the request's for the key head): a score by 2^-17
    max|q| sum|k| scale."""
    sm_scale = p.D ** -0.5 if sm_scale is None else sm_scale
    u_p = half_step(torch.bfloat16 if p.cache == torch.bfloat16 else torch.float16)
    u_o = half_step(p.act)
    res = []
    for b in range(len(p.new)):
        n, past = p.new[b], p.past[b]
        if n == 0:
            continue
        L = past + n
        k, v = p.kv64(b, L)
        pos = torch.arange(past, L, device=p.dev)[:, None]
        key = torch.arange(L, device=p.dev)[None, :]
        seen = key <= pos
        if window:
            seen &= key > pos - window
        q = p.q[p.rows_of(b)].to(F64)
        out = torch.empty(n, p.Hq, p.D, dtype=F64, device=p.dev)
        tol = torch.empty_like(out)
        G = p.Hq // p.Hkv
        for h in range(p.Hq):
            kh, vh = k[:, h // G], v[:, h // G]
            s = (q[:, h] @ kh.T) * sm_scale
            S = ((q[:, h].abs() @ kh.abs().T) * sm_scale).masked_fill(~seen, 0).amax(-1, True)
            w = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
            w = torch.where(seen, w, torch.zeros_like(w))  # unseen V may be anything
            vz = torch.where(seen.any(0)[:, None], vh, torch.zeros_like(vh))
            finite = torch.isfinite(vz)
            va = torch.where(finite, vz, torch.zeros_like(vz))
            o = w @ va
            for j in (~finite).any(-1).nonzero()[:, 0].tolist():  # rows that do see such a value
                rows = seen[:, j]
                bad = torch.where(finite[j], torch.zeros_like(vz[j]), vz[j])
                o[rows] = o[rows] + bad
            A = w @ va.abs()
            if p.cache == torch.float8_e4m3fn:
                most = q[:, h // G * G:(h // G + 1) * G].abs().amax()
                part = 2.0 ** -17 * sm_scale * most * kh.abs().sum(-1).expand(n, -1)
                S8 = part.masked_fill(~seen, 0).amax(-1, True)
            else:
                S8 = 0.0
            eps = 2 * S8 + u_p + L * 2.0 ** -23 + 2 * (p.D * 2.0 ** -23 * S + 2.0 ** -21 + 2.0 ** -22 * S)
            t = A * eps
            if p.cache != torch.bfloat16:
                t = t + L * 2.0 ** -25 * va.abs().amax()
            out[:, h] = o
            tol[:, h] = t + u_o * (o.abs() + t) + 1e-30
            if p.act == torch.float16:
                tol[:, h] += 2.0 ** -25
        res.append((p.rows_of(b), out, tol))
    return res


def rotation(pos, inv_freq, rope_scale):
    a = pos.to(F64)[:, None] * inv_freq
    return a.cos() * rope_scale, a.sin() * rope_scale


def append_rows(x, w, eps, pos, inv_freq, interleaved, rope_scale):
    """Norm and rotation of x [n, H, D] in fp64."""
    x = x.to(F64)
    if w is not None:
        x = x / torch.sqrt(x.square().mean(-1, keepdim=True) + eps) * w.to(F64)
    if inv_freq is not None:
        h = inv_freq.numel()
        cos, sin = (t[:, None] for t in rotation(pos, inv_freq, rope_scale))
        i = torch.arange(h, device=x.device)
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + h)
        y = x.clone()
        y[..., a] = x[..., a] * cos - x[..., b] * sin
        y[..., b] = x[..., b] * cos + x[..., a] * sin
        x = y
    return x
