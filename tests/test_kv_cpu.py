"""Host-side checks of the paged-cache calls that need no GPU: sizes and
pointers are refused before anything is enqueued, and the binding refuses
tensors that do not fit together."""
import ctypes

import pytest
import torch

from speculative_decoding_05_b200 import build
from speculative_decoding_05_b200 import dspark as D

P = ctypes.c_void_p
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 4, 6


@pytest.fixture(scope="module")
def lib():
    build.build()
    return D.load()


def base():
    """Arguments of a valid call (addresses never touched: every case below
    is refused first)."""
    a = 1 << 24
    return dict(q=a, k=a, v=a, q_stride=1024, k_stride=256, v_stride=256, act=1, n_rows=10, B=2,
                Hq=8, Hkv=2, D=128, max_len=4, row_start=a, verify_len=a, cache_len=a, table=a,
                max_pages=4, kc=a, vc=a, ks=0, vs=0, cache=1, n_pages=9, ps=64, qn=0, kn=0,
                eps=1e-6, freq=a, rot=128, inter=0, rs=1.0, out=a, vout=a, ws=a, bytes=1 << 26,
                scale=0.1, window=0)


def append(lib, **kw):
    c = dict(base(), **kw)
    return lib.dspark_kv_append(
        P(c["q"]), P(c["k"]), P(c["v"]), c["q_stride"], c["k_stride"], c["v_stride"], c["act"],
        c["n_rows"], c["B"], c["Hq"], c["Hkv"], c["D"], P(c["row_start"]), P(c["verify_len"]),
        P(c["cache_len"]), P(c["table"]), c["max_pages"], P(c["kc"]), P(c["vc"]), P(c["ks"]),
        P(c["vs"]), c["cache"], c["n_pages"], c["ps"], P(c["qn"]), P(c["kn"]), c["eps"],
        P(c["freq"]), c["rot"], c["inter"], c["rs"], P(c["out"]), P(c["ws"]), c["bytes"], None)


def read(lib, **kw):
    c = dict(base(), **kw)
    return lib.dspark_kv_read(
        P(c["kc"]), P(c["vc"]), P(c["ks"]), P(c["vs"]), c["cache"], c["n_pages"], c["ps"],
        P(c["row_start"]), P(c["verify_len"]), P(c["cache_len"]), P(c["table"]), c["max_pages"],
        c["n_rows"], c["B"], c["Hkv"], c["D"], P(c["out"]), P(c["vout"]), c["act"], P(c["ws"]),
        c["bytes"], None)


def attend(lib, **kw):
    c = dict(base(), **kw)
    return lib.dspark_attn_verify(
        P(c["q"]), c["q_stride"], c["act"], c["n_rows"], c["B"], c["Hq"], c["Hkv"], c["D"],
        c["max_len"], P(c["row_start"]), P(c["verify_len"]), P(c["cache_len"]), P(c["table"]),
        c["max_pages"], P(c["kc"]), P(c["vc"]), P(c["ks"]), P(c["vs"]), c["cache"], c["n_pages"],
        c["ps"], c["scale"], c["window"], P(c["out"]), P(c["ws"]), c["bytes"], None)


@pytest.mark.parametrize("call", [append, read, attend])
def test_shared_refusals(lib, call):
    assert call(lib, act=3) == INVALID           # rows are never e4m3
    assert call(lib, act=0) == INVALID
    assert call(lib, act=1, cache=2) == INVALID  # a 16-bit cache has its rows' type
    assert call(lib, cache=4) == INVALID
    assert call(lib, B=-1) == INVALID
    assert call(lib, n_rows=-1) == INVALID
    assert call(lib, Hkv=0) == INVALID
    assert call(lib, n_pages=-1) == INVALID
    assert call(lib, n_pages=0) == INVALID
    assert call(lib, max_pages=0) == INVALID
    assert call(lib, ps=0) == INVALID
    assert call(lib, D=96) == UNSUPPORTED
    assert call(lib, ps=8) == UNSUPPORTED
    assert call(lib, ps=48) == UNSUPPORTED
    assert call(lib, ps=512) == UNSUPPORTED
    assert call(lib, B=4097) == UNSUPPORTED
    assert call(lib, n_rows=1 << 31) == UNSUPPORTED
    assert call(lib, n_pages=1 << 24, ps=64) == UNSUPPORTED  # 2^31 places
    assert call(lib, ws=0) == WORKSPACE
    assert call(lib, ws=(1 << 24) + 16) == WORKSPACE
    assert call(lib, bytes=4096) == WORKSPACE
    for name in ("row_start", "verify_len", "cache_len", "table", "kc", "vc", "out"):
        assert call(lib, **{name: 0}) == INVALID, name
    for name in ("kc", "vc", "out"):
        assert call(lib, **{name: (1 << 24) + 8}) == INVALID, name
    assert call(lib, row_start=(1 << 24) + 4) == INVALID
    assert call(lib, table=(1 << 24) + 2) == INVALID
    # e4m3 needs its scales
    assert call(lib, cache=3) == INVALID
    assert call(lib, cache=3, ks=1 << 24) == INVALID
    assert call(lib, cache=3, ks=1 << 24, vs=(1 << 24) + 4) == INVALID


def test_append_refusals(lib):
    assert append(lib, Hq=9) == INVALID          # not a multiple of Hkv
    assert append(lib, Hq=1026, q_stride=1 << 20) == UNSUPPORTED
    assert append(lib, rot=144) == INVALID       # more than the head
    assert append(lib, rot=24) == UNSUPPORTED
    assert append(lib, rot=-16) == INVALID
    assert append(lib, freq=0) == INVALID
    assert append(lib, eps=-1.0) == INVALID
    assert append(lib, eps=float("nan")) == INVALID
    assert append(lib, rs=float("inf")) == INVALID
    assert append(lib, q_stride=1023) == INVALID
    assert append(lib, q_stride=1028) == UNSUPPORTED
    assert append(lib, k_stride=128) == INVALID
    assert append(lib, v_stride=260) == UNSUPPORTED
    for name in ("q", "k", "v"):
        assert append(lib, **{name: 0}) == INVALID
        assert append(lib, **{name: (1 << 24) + 2}) == INVALID


def test_attend_refusals(lib):
    assert attend(lib, Hq=9) == INVALID
    assert attend(lib, max_len=0) == INVALID
    assert attend(lib, window=-1) == INVALID
    assert attend(lib, scale=0.0) == INVALID
    assert attend(lib, scale=-1.0) == INVALID
    assert attend(lib, scale=float("nan")) == INVALID
    assert attend(lib, q=0) == INVALID
    assert attend(lib, q=(1 << 24) + 8) == INVALID
    assert attend(lib, q_stride=1016) == INVALID
    assert attend(lib, q_stride=1025) == UNSUPPORTED
    need = lib.dspark_attn_workspace_size(2, 8, 2, 128, 4)
    assert attend(lib, bytes=need - 1) == WORKSPACE


def test_workspace_sizes(lib):
    """Bounded whatever the lengths, 0 for sizes that no call takes."""
    assert lib.dspark_kv_workspace_size() >= 2048
    assert lib.dspark_attn_workspace_size(1, 8, 3, 128, 1) == 0
    assert lib.dspark_attn_workspace_size(1, 8, 2, 128, 0) == 0
    assert lib.dspark_attn_workspace_size(-1, 8, 2, 128, 1) == 0
    for B, Hq, n in ((1, 8, 1), (512, 64, 17), (4096, 1024, 1 << 20)):
        size = lib.dspark_attn_workspace_size(B, Hq, 8, 128, n)
        assert lib.dspark_kv_workspace_size() <= size < 256 << 20 and size % 256 == 0


def tensors(**kw):
    t = dict(q=torch.zeros(5, 8, 64, dtype=torch.bfloat16),
             k=torch.zeros(5, 2, 64, dtype=torch.bfloat16),
             v=torch.zeros(5, 2, 64, dtype=torch.bfloat16),
             row_start=torch.zeros(3, dtype=torch.int64),
             verify_len=torch.zeros(3, dtype=torch.int32),
             cache_len=torch.zeros(3, dtype=torch.int32),
             page_table=torch.zeros(3, 4, dtype=torch.int32),
             k_cache=torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16),
             v_cache=torch.zeros(6, 2, 16, 64, dtype=torch.bfloat16),
             q_out=torch.zeros(5, 8, 64, dtype=torch.bfloat16))
    t.update(kw)
    return t


def test_binding_refuses_tensors_that_do_not_fit(lib):
    ws = torch.zeros(1 << 16, dtype=torch.uint8)
    bf = torch.bfloat16

    def bad(**kw):
        t = tensors(**{n: x for n, x in kw.items() if n not in ("inv_freq", "q_norm", "k_scale",
                                                                "v_scale")})
        more = {n: x for n, x in kw.items() if n not in t}
        with pytest.raises(ValueError):
            D.dspark_kv_append(t["q"], t["k"], t["v"], t["row_start"], t["verify_len"],
                               t["cache_len"], t["page_table"], t["k_cache"], t["v_cache"],
                               t["q_out"], ws, **more)

    bad(q=torch.zeros(5, 8, 64))                            # fp32 rows
    bad(q=torch.zeros(5, 8, 128, dtype=bf)[..., ::2])       # elements apart
    bad(q=torch.zeros(8, 5, 64, dtype=bf).transpose(0, 1))  # heads apart
    bad(k=torch.zeros(5, 3, 64, dtype=bf))
    bad(k=torch.zeros(4, 2, 64, dtype=bf))
    bad(v=torch.zeros(5, 2, 64, dtype=torch.float16))
    bad(row_start=torch.zeros(3, dtype=torch.int32))
    bad(verify_len=torch.zeros(2, dtype=torch.int32))
    bad(cache_len=torch.zeros(6, dtype=torch.int32)[::2])
    bad(page_table=torch.zeros(3, 8, dtype=torch.int32)[:, ::2])
    bad(page_table=torch.zeros(12, dtype=torch.int32))
    bad(v_cache=torch.zeros(7, 2, 16, 64, dtype=bf))
    bad(k_cache=torch.zeros(6, 2, 16, 64, dtype=bf).transpose(1, 2))
    bad(q_out=torch.zeros(5, 8, 128, dtype=bf)[..., :64])
    bad(inv_freq=torch.zeros(32))                           # fp32 frequencies
    bad(q_norm=torch.zeros(64, dtype=bf))
    bad(k_scale=torch.zeros(6, 2, 16))                      # scales of a 16-bit cache
    f8 = torch.float8_e4m3fn
    bad(k_cache=torch.zeros(6, 2, 16, 64).to(f8), v_cache=torch.zeros(6, 2, 16, 64).to(f8))
    t = tensors()
    with pytest.raises(ValueError):
        D.dspark_attn_verify(t["q"], t["k_cache"], t["v_cache"], t["row_start"], t["verify_len"],
                             t["cache_len"], t["page_table"], t["q_out"][:4], ws, 1)
    with pytest.raises(D.DSparkError) as err:               # refused by the library
        D.dspark_attn_verify(t["q"], t["k_cache"], t["v_cache"], t["row_start"], t["verify_len"],
                             t["cache_len"], t["page_table"], t["q_out"], ws, 0)
    assert err.value.code == INVALID
    with pytest.raises(D.DSparkError) as err:
        D.dspark_kv_read(t["k_cache"], t["v_cache"], t["row_start"], t["verify_len"],
                         t["cache_len"], t["page_table"], t["k"], t["v"], ws[:256])
    assert err.value.code == WORKSPACE
