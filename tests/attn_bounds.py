"""A second fp64 statement of dspark_attn_verify with bounds that hold for every
row by itself (test infrastructure): what stands in the rows beside it, or in
keys of little weight, widens none of them."""
import torch

from tests.kv_reference import F64, half_step, quantise

E4 = torch.float8_e4m3fn
# fp16 weights keep 2^-25 (half their smallest step) against a largest weight of
# at least 2^LIFT
LIFT = 8


def put(p, name, b, lo, x):
    """Overwrites positions lo .. of request b in one of p's caches by x
    [n, Hkv, D] (fp32)."""
    pg, sl = p.places(b, lo, lo + x.shape[0])
    cache, scale = getattr(p, name + "_cache"), getattr(p, name + "_scale")
    if scale is None:
        cache[pg, :, sl] = x.to(cache.dtype)
    else:
        c, s = quantise(x)
        cache.view(torch.uint8)[pg, :, sl] = c.view(torch.uint8)
        scale[pg, :, sl] = s


def attention_rows(p, sm_scale=None, window=0):
    """[(rows, out, tolerance)] per request in fp64, for finite inputs among the
    keys that are seen.

    For element d of a row with weights w_j and A = sum_j w_j |v_jd|:
      weights rounded once, p_j = w_j (1 + d_j), |d_j| <= u_p: the product is off by
        u_p A; where their sum is formed from the rounded ones, o = sum p v / sum p
        moves by sum_j w_j d_j (v_jd - o), at most u_p (A + |o|);
      fp16 weights also by 2^-25 each where the largest (16-bit cache: w_j; e4m3: w_j
        with V's scale, times a code of at most 448, which makes it w_j max_d |v_jd|)
        is at least 2^LIFT: L 2^(-25 - LIFT) times the largest of these products, for
        product and sum;
      sums in fp32 over L keys: L 2^-23 A;
      a score: D products in fp32, D 2^-23 S for S the largest sum of |q k| scale of
        the row, its factor and 2^x (2^-21 and 2^-22 S); weight and normaliser, so
        twice.  e4m3: Q as a sum of e4m3 parts, off by half the format's
        smallest step, 2^-10, where the largest element of THIS row and head is in
        [128, 256): 2^-17 max|q| sum|k| scale;
      the result rounded once."""
    sm_scale = p.D ** -0.5 if sm_scale is None else sm_scale
    u_p = half_step(torch.bfloat16 if p.cache == torch.bfloat16 else torch.float16)
    u_o = half_step(p.act)
    res = []
    for b in range(len(p.new)):
        n, L = p.new[b], p.past[b] + p.new[b]
        if n == 0:
            continue
        k, v = p.kv64(b, L)
        back = torch.arange(p.past[b], L, device=p.dev)[:, None] - torch.arange(L, device=p.dev)
        seen = (back >= 0) & (back < window) if window else back >= 0
        q = p.q[p.rows_of(b)].to(F64)
        out = torch.empty(n, p.Hq, p.D, dtype=F64, device=p.dev)
        tol = torch.empty_like(out)
        G = p.Hq // p.Hkv
        for h in range(p.Hq):
            kh, vh = k[:, h // G], v[:, h // G]
            s = torch.where(seen, q[:, h] @ kh.T * sm_scale, -torch.inf)
            w = torch.exp(s - s.amax(1, keepdim=True))
            w = w / w.sum(1, keepdim=True)
            o, A = w @ vh, w @ vh.abs()
            S = torch.where(seen, q[:, h].abs() @ kh.abs().T * sm_scale, 0).amax(1, keepdim=True)
            eps = u_p + L * 2.0 ** -23 + 2 * (p.D * 2.0 ** -23 * S + 2.0 ** -21 + 2.0 ** -22 * S)
            if p.cache == E4:
                part = 2.0 ** -17 * sm_scale * q[:, h].abs().amax(1, keepdim=True) * kh.abs().sum(1)
                eps = eps + 2 * torch.where(seen, part, 0).amax(1, keepdim=True)
            t = A * eps + u_p * o.abs()
            if p.cache != torch.bfloat16:
                top = (w * vh.abs().amax(1)).amax(1, keepdim=True) if p.cache == E4 else \
                    w.amax(1, keepdim=True) * vh.abs().amax()
                t = t + 2 * L * 2.0 ** (-25 - LIFT) * top
            out[:, h] = o
            tol[:, h] = t + u_o * (o.abs() + t) + (2.0 ** -25 if p.act == torch.float16 else 0)
        res.append((p.rows_of(b), out, tol))
    return res
