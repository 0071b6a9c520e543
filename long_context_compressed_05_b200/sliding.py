"""Layer helpers of the uncompressed sliding-window layers: grouped heads over the recent window and the first tokens,
a paged cache, and the norm between the layers of a residual-chained stack.

Nothing here computes: every step is a call into libhcsa.so.
"""
from __future__ import annotations

import dataclasses

import torch

from . import _lib as L
from .layer import params_for, torch_dtype

__all__ = ["SlidingSpec", "SlidingPrefillLayer", "SlidingDecodeLayer", "new_pages"]


@dataclasses.dataclass(frozen=True)
class SlidingSpec:
    """One sliding-window layer; the fields have the meaning of the call parameters of the same names."""
    D: int
    H: int
    Hkv: int
    dh: int
    window: int = 128
    sinks: int = 0
    scale: float = 0.125
    dtype: str = "bf16"
    eps: float = 1e-6
    T: int = 0

    kind = "swa"
    m = 1
    width = 1

    @property
    def C(self) -> int:
        return 2 * self.dh

    @property
    def ncols(self) -> int:
        """Columns of the projection [k | v | q]."""
        return (self.H + 2 * self.Hkv) * self.dh

    def views(self, y):
        """(k, v, q) column views of the projection y [rows, ncols]."""
        n = self.Hkv * self.dh
        return y[:, :n], y[:, n:2 * n], y[:, 2 * n:]


def new_pages(spec: SlidingSpec, p: L.Params, page_table, device="cuda") -> L.Pages:
    """Zeroed page arrays of the size p asks for (FP8 byte arrays with p.lowprec) around `page_table`."""
    if p.lowprec:
        kv = [torch.zeros(L.hcsa_page_bytes(p), dtype=torch.uint8, device=device) for _ in range(2)]
    else:
        kv = [torch.zeros((p.n_pages, p.Hkv, p.page, p.dh), dtype=torch_dtype(spec.dtype), device=device)
              for _ in range(2)]
    return L.make_pages(*kv, page_table)


class _Normed:
    """The norm before the layer (its input is the residual stream, or the stream and what was added to it)."""

    def norm(self, x, w, delta=None, x_out=None):
        """self.h = rmsnorm(x + delta) * w; x_out (may be x): the updated stream."""
        L.hcsa_add_rmsnorm(self.p, x, delta, w, self.spec.eps, x_out, self.h)
        return self.h

    def out_project(self, x, W_o):
        """Residual update of a chained stack: x += out W_o, in place (bf16)."""
        L.hcsa_out_project(self.p, self.out, W_o, x, self.ws_proj)
        return x

    def _buffers(self, rows, device):
        dt = torch_dtype(self.spec.dtype)
        self.h = torch.empty((rows, self.spec.D), dtype=dt, device=device)
        self.y = torch.empty((rows, self.spec.ncols), dtype=dt, device=device)
        self.out = torch.empty((rows, self.spec.H * self.spec.dh), dtype=dt, device=device)
        n = L.hcsa_workspace_bytes(self.p, L.OP_PROJECT)
        self.ws_proj = torch.empty(max(n, 16), dtype=torch.uint8, device=device) if n else None


class SlidingPrefillLayer(_Normed):
    """One sliding-window layer over a sequence of spec.T tokens, buffers allocated once."""

    def __init__(self, spec: SlidingSpec, device="cuda"):
        self.spec = spec
        self.p = params_for(spec)
        self._buffers(spec.T, device)

    def forward(self, h, W_cat):
        """Attention of the (normed) input h [T, D]; W_cat [D, ncols] = [W_k | W_v | W_q]."""
        L.hcsa_project(self.p, L.KIND_SWA, h, W_cat, self.y, self.ws_proj)
        k, v, q = self.spec.views(self.y)
        L.swa_attend(self.p, q, k, v, self.out)
        return self.out

    def to_pages(self, p: L.Params, pages: L.Pages, seq: int):
        """Write the keys and values of the last forward() to tokens 0 .. T - 1 of sequence `seq` (p: the decode
        layer's parameters)."""
        T, dev = self.spec.T, self.y.device
        pos = torch.arange(T, dtype=torch.int32, device=dev)
        k, v, _ = self.spec.views(self.y)
        L.swa_page_append(p, pages, pos, k, v, torch.full((T,), seq, dtype=torch.int32, device=dev))


class SlidingDecodeLayer(_Normed):
    """One sliding-window layer's decode step for B sequences over a paged cache."""

    def __init__(self, spec: SlidingSpec, B, page, n_pages, page_table, lowprec=False, pages=None, device="cuda"):
        """page_table [B, max_pages] int32; pages: an existing handle (make_pages), else zeroed arrays are made.
        lowprec: the pages in FP8."""
        self.spec = spec
        self.p = params_for(spec, T=0, B=B, lowprec=lowprec, page=page, n_pages=n_pages,
                            max_pages=page_table.shape[1])
        self.pages = new_pages(spec, self.p, page_table, device) if pages is None else pages
        self._buffers(B, device)
        self.ws = torch.empty(L.hcsa_workspace_bytes(self.p, L.OP_SWA_DECODE_ATTEND), dtype=torch.uint8,
                              device=device)

    def step(self, h, W_cat, pos):
        """Attention of the new tokens h [B, D] at positions pos [B] (-1: empty slot)."""
        L.hcsa_project(self.p, L.KIND_SWA, h, W_cat, self.y, self.ws_proj)
        k, v, q = self.spec.views(self.y)
        L.swa_page_append(self.p, self.pages, pos, k, v)
        L.swa_decode_attend(self.p, self.pages, pos, q, self.out, self.ws)
        return self.out
