"""The target's paged K/V cache beside a decode step (include/dspark_kv.h).

PagedKV owns one layer's pages, the sequences' page table and lengths, and the
workspaces of its calls (one stream at a time), so that a layer of the target's verify forward launches
only library kernels and captures into the step's CUDA graph:

    kv.append(q, k, v, rows, q_out)      # norms, rotation, cache write
    kv.attend(q_out, rows, out)          # attention of the new rows
    ...                                  # the rest of the target, dspark_verify*
    kv.advance(n_accepted, rows)         # the accepted tokens and the emitted one

`rows` are the row markers of the verify: (row_start [B] int64, verify_len [B]
int32), which dspark_confidence_prefix writes on the device.  A slot without a
request has verify_len = -1 here and 0 in dspark_verify* (include/dspark_kv.h,
"Idle slots").
"""
from __future__ import annotations

import math

import torch

from . import dspark as D


def rope_frequencies(rot_dim: int, theta: float = 1e4, scaling: str = "none", factor: float = 1.0,
                     original_len: int = 0, beta_fast: float = 32.0, beta_slow: float = 1.0):
    """(inv_freq [rot_dim / 2] fp64 on the CPU, rope_scale) for dspark_kv_append.

    scaling  "none"
             "linear": positions divided by factor
             "ntk":    theta enlarged so that the lowest frequency is divided by
                       factor and the highest stays
             "yarn":   frequencies that turn more than beta_fast times over
                       original_len positions stay, those that turn less than
                       beta_slow times are divided by factor, linear between
                       (over the index); rope_scale 0.1 ln(factor) + 1, at least 1
    """
    if rot_dim <= 0 or rot_dim % 2:
        raise ValueError(f"rot_dim: want a positive even number, got {rot_dim}")
    half = rot_dim // 2
    i = torch.arange(half, dtype=torch.float64)
    if scaling == "ntk":
        theta = theta * factor ** (rot_dim / max(rot_dim - 2, 1))
    f = theta ** (-2.0 * i / rot_dim)
    if scaling in ("none", "ntk"):
        return f, 1.0
    if scaling == "linear":
        return f / factor, 1.0
    if scaling == "yarn":
        if original_len <= 0:
            raise ValueError("yarn needs original_len")

        def index_of(turns):  # where a frequency turns that often over original_len
            return half * math.log(original_len / (2 * math.pi * turns)) / math.log(theta)

        # (high may lie beyond the last frequency: the ramp then ends beyond it too)
        low = max(math.floor(index_of(beta_fast)), 0)
        high = min(math.ceil(index_of(beta_slow)), rot_dim - 1)
        ramp = ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        return f * (1.0 - ramp) + f / factor * ramp, 0.1 * math.log(max(factor, 1.0)) + 1.0
    raise ValueError(f"scaling: {scaling!r} is not one of none, linear, ntk, yarn")


class PagedKV:
    """One layer's paged cache for B sequences of up to max_pages pages each.

    dtype: the rows' type (bfloat16 or float16) or float8_e4m3fn (quantised, one
    scale for each token and head).  page_table [B, max_pages] int32 may be
    shared between layers; by default sequence b owns pages b * max_pages .., so
    that n_pages (default B * max_pages) can not be less.

    max_len: the longest run of new rows that attend takes; it chooses the kernel,
    and a longer run is flagged and left out.  K + 1 for the steps of a decode; a
    prompt's chunk wants a bound of its own (a step under a chunk's bound is right
    but slower): dspark_attn_verify over the same tensors takes one.  append and
    read have no such bound.  ws_attn (39 MB at 128 elements) may be another
    layer's, where both run on one stream.
    """

    def __init__(self, B: int, Hq: int, Hkv: int, head_dim: int, max_pages: int,
                 page_size: int = 64, dtype=torch.bfloat16, n_pages: int | None = None,
                 max_len: int = 1, page_table=None, device="cuda"):
        self.B, self.Hq, self.Hkv, self.D = B, Hq, Hkv, head_dim
        self.page_size, self.max_len = page_size, max_len
        dev = torch.device(device)
        n_pages = B * max_pages if n_pages is None else n_pages
        if page_table is None and n_pages < B * max_pages:
            raise ValueError(f"n_pages: {n_pages} pages do not hold {B} sequences of {max_pages}; "
                             "fewer need a page_table")
        shape = (n_pages, Hkv, page_size, head_dim)
        self.k_cache = torch.zeros(shape, dtype=dtype, device=dev)
        self.v_cache = torch.zeros(shape, dtype=dtype, device=dev)
        self.k_scale = self.v_scale = None
        if dtype == torch.float8_e4m3fn:
            self.k_scale = torch.zeros(shape[:3], dtype=torch.float32, device=dev)
            self.v_scale = torch.zeros(shape[:3], dtype=torch.float32, device=dev)
        if page_table is None:
            page_table = torch.arange(B * max_pages, dtype=torch.int32, device=dev).view(B, -1)
        self.page_table = page_table
        self.cache_len = torch.zeros(B, dtype=torch.int32, device=dev)
        self.ws = D.workspace(D.dspark_kv_workspace_size(), dev)
        self.ws_attn = D.workspace(D.dspark_attn_workspace_size(B, Hq, Hkv, head_dim, max_len), dev)
        for ws in (self.ws, self.ws_attn):  # flags() may come before a call
            ws[:256].zero_()

    def _markers(self, rows):
        row_start, verify_len = rows
        return row_start, verify_len, self.cache_len, self.page_table

    def append(self, q, k, v, rows, q_out, stream=None, **how):
        """dspark_kv_append of the new rows; `how`: q_norm, k_norm, eps,
        inv_freq, interleaved, rope_scale."""
        D.dspark_kv_append(q, k, v, *self._markers(rows), self.k_cache, self.v_cache, q_out,
                           self.ws, k_scale=self.k_scale, v_scale=self.v_scale, stream=stream,
                           **how)

    def attend(self, q, rows, out, sm_scale=None, window=0, stream=None):
        """dspark_attn_verify of the new rows, after their append."""
        D.dspark_attn_verify(q, self.k_cache, self.v_cache, *self._markers(rows), out,
                             self.ws_attn, self.max_len, k_scale=self.k_scale,
                             v_scale=self.v_scale, sm_scale=sm_scale, window=window, stream=stream)

    def read(self, rows, k_out, v_out, start=None, stream=None):
        """dspark_kv_read: verify_len[b] + 1 positions from start[b] (None: the
        rows of the last append)."""
        row_start, verify_len = rows
        D.dspark_kv_read(self.k_cache, self.v_cache, row_start, verify_len,
                         self.cache_len if start is None else start, self.page_table, k_out, v_out,
                         self.ws, k_scale=self.k_scale, v_scale=self.v_scale, stream=stream)

    def advance(self, n_accepted, rows=None):
        """The sequences grow by the accepted tokens and the one the verify
        emitted before them (whose row the step computed).  With the step's
        `rows`, slots that were idle in it (verify_len < 0) stay as they are,
        whatever n_accepted says of them: dspark_verify* knows no idle slots and
        counts one as a request without drafts.  Without `rows` an idle slot
        needs n_accepted = -1."""
        if rows is None:
            self.cache_len.add_(n_accepted).add_(1)
        else:
            self.cache_len.add_((n_accepted + 1) * (rows[1] >= 0))

    def flags(self, stream=None):
        return {"kv": D.dspark_get_device_flags(self.ws, stream),
                "attn": D.dspark_get_device_flags(self.ws_attn, stream)}
