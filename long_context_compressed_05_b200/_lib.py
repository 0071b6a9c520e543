"""ctypes binding of libhcsa.so: same names as the C ABI (include/hca_csa.h).

Argument marshalling only: tensors become (pointer, leading dimension) pairs and
the current torch CUDA stream is passed along.  Every step runs in the CUDA
library; if it is missing the first call raises.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhcsa.so")

HCSA_F32, HCSA_BF16 = 0, 1
KIND_CSA, KIND_HCA, KIND_SWA = 0, 1, 2
OP_PROJECT, OP_CSA_INDEX_TOPK, OP_CSA_ATTEND, OP_HCA_ATTEND = 0, 1, 2, 3
OP_CSA_DECODE_INDEX_TOPK, OP_CSA_DECODE_ATTEND, OP_HCA_DECODE_ATTEND = 4, 5, 6
OP_CSA_DECODE_INDEX_TOPK_SHARD, OP_CSA_DECODE_ATTEND_SHARD, OP_HCA_DECODE_ATTEND_SHARD = 7, 8, 9
OP_SWA_DECODE_ATTEND = 10
NO_WINDOW = 2 ** 31 - 1   # window of a sliding-window layer that sees every earlier token

STATUS = {0: "HCSA_OK", 1: "HCSA_ERR_NULL", 2: "HCSA_ERR_SHAPE", 3: "HCSA_ERR_DTYPE", 4: "HCSA_ERR_ALIGN",
          5: "HCSA_ERR_WORKSPACE", 6: "HCSA_ERR_CUDA", 7: "HCSA_ERR_TIMEOUT", 8: "HCSA_ERR_UNSUPPORTED",
          9: "HCSA_ERR_DEVICE"}

# every entry point the header declares (checked by the CPU export test)
EXPORTS = ["hcsa_version", "hcsa_status_string", "hcsa_workspace_bytes", "hcsa_proj_cols", "hcsa_project",
           "hcsa_out_project",
           "csa_compress", "hca_compress", "csa_index_topk", "csa_attend", "hca_attend", "hcsa_cache_append",
           "csa_decode_index_topk", "csa_decode_attend", "hca_decode_attend", "csa_decode_index_topk_noalloc",
           "hcsa_get_device_status", "hcsa_selftest_wait_timeout",
           "hcsa_launch_count", "hcsa_entry_bytes", "hcsa_key_bytes", "hcsa_quantize_rows",
           "csa_decode_index_topk_shard", "csa_topk_merge", "csa_decode_attend_shard", "hca_decode_attend_shard",
           "hcsa_merge_partials", "hcsa_project_append", "hcsa_project_compress",
           "hcsa_page_bytes", "swa_attend", "swa_page_append", "swa_decode_attend", "hcsa_add_rmsnorm"]
STORE_ENTRIES, STORE_KEYS = 0, 1


class HcsaError(RuntimeError):
    def __init__(self, fn, code):
        self.code = code
        super().__init__(f"{fn} failed: {STATUS.get(code, code)}")


class Params(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int32) for n in ("B", "T", "D", "m", "width", "C", "di", "Hi", "topk", "window",
                                              "H", "dh")] + [("scale", ctypes.c_float), ("dtype", ctypes.c_int32),
                                                             ("n_cap", ctypes.c_int32), ("row0", ctypes.c_int32),
                                                             ("row1", ctypes.c_int32), ("lowprec", ctypes.c_int32),
                                                             ("ent0", ctypes.c_int32), ("ent_shard", ctypes.c_int32),
                                                             ("Hkv", ctypes.c_int32), ("sinks", ctypes.c_int32),
                                                             ("page", ctypes.c_int32), ("n_pages", ctypes.c_int32),
                                                             ("max_pages", ctypes.c_int32)]


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("entries", "idx_keys", "win_kv", "ring_g", "ring_ki")]


class Pages(ctypes.Structure):
    _fields_ = [(n, ctypes.c_void_p) for n in ("k_pages", "v_pages", "page_table")]


_lib = None


def load():
    """Load libhcsa.so (raises if it has not been built)."""
    global _lib
    if _lib is not None:
        return _lib
    if not os.path.exists(LIB_PATH):
        raise RuntimeError(f"CUDA library {LIB_PATH} is missing: build it with __graft_entry__.build()")
    lib = ctypes.CDLL(LIB_PATH)
    V, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    P = ctypes.POINTER(Params)
    CP = ctypes.POINTER(Cache)
    PG = ctypes.POINTER(Pages)
    sig = {
        "hcsa_version": (I32, []),
        "hcsa_status_string": (ctypes.c_char_p, [I32]),
        "hcsa_workspace_bytes": (SZ, [P, I32]),
        "hcsa_proj_cols": (I64, [P, I32]),
        "hcsa_project": (I32, [P, I32, I64, V, V, V, V, SZ, V]),
        "hcsa_out_project": (I32, [P, I64, V, I64, V, V, I64, V, SZ, V]),
        "csa_compress": (I32, [P, V, I64, V, I64, V, I64, V, V, V, V]),
        "hca_compress": (I32, [P, V, I64, V, I64, V, V, V]),
        "csa_index_topk": (I32, [P, V, I64, V, I64, V, V, V, SZ, V]),
        "csa_attend": (I32, [P, V, I64, V, I64, V, V, V, V, SZ, V]),
        "hca_attend": (I32, [P, V, I64, V, I64, V, V, V, SZ, V]),
        "hcsa_cache_append": (I32, [P, CP, V, V, I64, V, I64, V, I64, V, V]),
        "csa_decode_index_topk": (I32, [P, CP, V, V, I64, V, I64, V, V, SZ, V]),
        "csa_decode_attend": (I32, [P, CP, V, V, I64, V, V, V, SZ, V]),
        "hca_decode_attend": (I32, [P, CP, V, V, I64, V, V, SZ, V]),
        "csa_decode_index_topk_noalloc": (I32, [P, CP, V, V, I64, V, I64, V, V]),
        "hcsa_get_device_status": (I32, [V]),
        "hcsa_selftest_wait_timeout": (I32, [V]),
        "hcsa_launch_count": (I64, [I32]),
        "hcsa_entry_bytes": (SZ, [P, I64]),
        "hcsa_key_bytes": (SZ, [P, I64]),
        "hcsa_quantize_rows": (I32, [P, I32, V, I64, V, V]),
        "csa_decode_index_topk_shard": (I32, [P, CP, V, V, I64, V, I64, V, V, V, SZ, V]),
        "csa_topk_merge": (I32, [P, V, V, I32, V, V]),
        "csa_decode_attend_shard": (I32, [P, CP, V, V, I64, V, I32, V, V, SZ, V]),
        "hca_decode_attend_shard": (I32, [P, CP, V, V, I64, I32, V, V, SZ, V]),
        "hcsa_merge_partials": (I32, [P, V, I32, V, I64, V]),
        "hcsa_project_append": (I32, [P, I32, CP, V, V, V, V, V, V, SZ, V]),
        "hcsa_project_compress": (I32, [P, I32, V, V, V, V, V, V, V, SZ, V]),
        "hcsa_page_bytes": (SZ, [P]),
        "swa_attend": (I32, [P, V, I64, V, I64, V, I64, V, I64, V]),
        "swa_page_append": (I32, [P, PG, I64, V, V, V, I64, V, I64, V]),
        "swa_decode_attend": (I32, [P, PG, V, V, I64, V, I64, V, SZ, V]),
        "hcsa_add_rmsnorm": (I32, [P, I64, V, I64, V, I64, V, ctypes.c_float, V, I64, V, I64, V, V]),
    }
    for name, (res, args) in sig.items():
        f = getattr(lib, name)
        f.restype = res
        f.argtypes = args
    _lib = lib
    return lib


def _check(fn, code):
    if code != 0:
        raise HcsaError(fn, code)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _ld(t):
    return 0 if t is None else (t.stride(0) if t.dim() >= 2 else t.shape[-1])


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def make_params(*, T=0, D=0, m=4, width=8, C=0, di=0, Hi=0, topk=0, window=128, H=1, dh=0, scale=1.0,
                dtype="bf16", B=1, n_cap=0, row0=0, row1=0, lowprec=0, ent0=0, ent_shard=0, Hkv=0, sinks=0, page=0,
                n_pages=0, max_pages=0) -> Params:
    return Params(B=B, T=T, D=D, m=m, width=width, C=C, di=di, Hi=Hi, topk=topk, window=window, H=H, dh=dh,
                  scale=scale, dtype=HCSA_BF16 if dtype == "bf16" else HCSA_F32, n_cap=n_cap, row0=row0,
                  row1=row1, lowprec=int(lowprec), ent0=ent0, ent_shard=int(ent_shard), Hkv=Hkv, sinks=sinks,
                  page=page, n_pages=n_pages, max_pages=max_pages)


def make_cache(entries, win_kv, ring_g, idx_keys=None, ring_ki=None) -> Cache:
    return Cache(entries=_ptr(entries), idx_keys=_ptr(idx_keys), win_kv=_ptr(win_kv), ring_g=_ptr(ring_g),
                 ring_ki=_ptr(ring_ki))


# ---------------------------------------------------------------- entry points (same names as the C ABI)

def hcsa_version():
    return load().hcsa_version()


def hcsa_status_string(code):
    return load().hcsa_status_string(code).decode()


def hcsa_workspace_bytes(p: Params, op: int) -> int:
    return int(load().hcsa_workspace_bytes(ctypes.byref(p), op))


def hcsa_proj_cols(p: Params, kind: int) -> int:
    return int(load().hcsa_proj_cols(ctypes.byref(p), kind))


def hcsa_project(p, kind, x, W_cat, y, ws=None, stream=None):
    _check("hcsa_project", load().hcsa_project(ctypes.byref(p), kind, x.shape[0], _ptr(x), _ptr(W_cat), _ptr(y),
                                               _ptr(ws), 0 if ws is None else ws.numel() * ws.element_size(),
                                               _stream(stream)))


def hcsa_out_project(p, out, W_o, x, ws=None, stream=None):
    """x += out W_o in place (the residual update of a chained stack; bf16)."""
    _check("hcsa_out_project", load().hcsa_out_project(ctypes.byref(p), x.shape[0], _ptr(out), _ld(out), _ptr(W_o),
                                                       _ptr(x), _ld(x), _ptr(ws), _wsz(ws), _stream(stream)))


def csa_compress(p, kv, g, ki, bias, entries, idx_keys, stream=None):
    _check("csa_compress", load().csa_compress(ctypes.byref(p), _ptr(kv), _ld(kv), _ptr(g), _ld(g), _ptr(ki),
                                               _ld(ki), _ptr(bias), _ptr(entries), _ptr(idx_keys),
                                               _stream(stream)))


def hca_compress(p, kv, g, bias, entries, stream=None):
    _check("hca_compress", load().hca_compress(ctypes.byref(p), _ptr(kv), _ld(kv), _ptr(g), _ld(g), _ptr(bias),
                                               _ptr(entries), _stream(stream)))


def _wsz(ws):
    return 0 if ws is None else ws.numel() * ws.element_size()


def csa_index_topk(p, qi, w, idx_keys, sel, ws, stream=None):
    _check("csa_index_topk", load().csa_index_topk(ctypes.byref(p), _ptr(qi), _ld(qi), _ptr(w), _ld(w),
                                                   _ptr(idx_keys), _ptr(sel), _ptr(ws), _wsz(ws),
                                                   _stream(stream)))


def csa_attend(p, q, kv, entries, sel, out, ws=None, stream=None):
    _check("csa_attend", load().csa_attend(ctypes.byref(p), _ptr(q), _ld(q), _ptr(kv), _ld(kv), _ptr(entries),
                                           _ptr(sel), _ptr(out), _ptr(ws), _wsz(ws), _stream(stream)))


def hca_attend(p, q, kv, entries, out, ws=None, stream=None):
    _check("hca_attend", load().hca_attend(ctypes.byref(p), _ptr(q), _ld(q), _ptr(kv), _ld(kv), _ptr(entries),
                                           _ptr(out), _ptr(ws), _wsz(ws), _stream(stream)))


def hcsa_cache_append(p, cache: Cache, pos, kv, g, ki, bias, stream=None):
    _check("hcsa_cache_append", load().hcsa_cache_append(ctypes.byref(p), ctypes.byref(cache), _ptr(pos),
                                                         _ptr(kv), _ld(kv), _ptr(g), _ld(g), _ptr(ki), _ld(ki),
                                                         _ptr(bias), _stream(stream)))


def csa_decode_index_topk(p, cache: Cache, pos, qi, w, sel, ws, stream=None):
    _check("csa_decode_index_topk", load().csa_decode_index_topk(
        ctypes.byref(p), ctypes.byref(cache), _ptr(pos), _ptr(qi), _ld(qi), _ptr(w), _ld(w), _ptr(sel), _ptr(ws),
        _wsz(ws), _stream(stream)))


def csa_decode_attend(p, cache: Cache, pos, q, sel, out, ws=None, stream=None):
    _check("csa_decode_attend", load().csa_decode_attend(ctypes.byref(p), ctypes.byref(cache), _ptr(pos), _ptr(q),
                                                         _ld(q), _ptr(sel), _ptr(out), _ptr(ws), _wsz(ws),
                                                         _stream(stream)))


def hca_decode_attend(p, cache: Cache, pos, q, out, ws=None, stream=None):
    _check("hca_decode_attend", load().hca_decode_attend(ctypes.byref(p), ctypes.byref(cache), _ptr(pos), _ptr(q),
                                                         _ld(q), _ptr(out), _ptr(ws), _wsz(ws), _stream(stream)))


def csa_decode_index_topk_noalloc(p, cache: Cache, pos, qi, w, sel, stream=None):
    """csa_decode_index_topk with the scores in the library's fixed scratch array (no workspace)."""
    _check("csa_decode_index_topk_noalloc", load().csa_decode_index_topk_noalloc(
        ctypes.byref(p), ctypes.byref(cache), _ptr(pos), _ptr(qi), _ld(qi), _ptr(w), _ld(w), _ptr(sel),
        _stream(stream)))


def hcsa_get_device_status(stream=None) -> int:
    return int(load().hcsa_get_device_status(_stream(stream)))


def hcsa_selftest_wait_timeout(stream=None) -> None:
    """Enqueue the bounded-wait self-test kernel (see include/hca_csa.h)."""
    _check("hcsa_selftest_wait_timeout", load().hcsa_selftest_wait_timeout(_stream(stream)))


def hcsa_entry_bytes(p: Params, rows: int) -> int:
    return int(load().hcsa_entry_bytes(ctypes.byref(p), rows))


def hcsa_key_bytes(p: Params, rows: int) -> int:
    return int(load().hcsa_key_bytes(ctypes.byref(p), rows))


def hcsa_quantize_rows(p, what, src, dst, stream=None):
    """src: [rows, C] (entries) or [rows, di] (keys) bf16; dst: a byte buffer of the matching size."""
    _check("hcsa_quantize_rows", load().hcsa_quantize_rows(ctypes.byref(p), what, _ptr(src), src.shape[0],
                                                           _ptr(dst), _stream(stream)))


def hcsa_project_compress(p, kind, x, W_cat, bias, y, entries, idx_keys, ws=None, stream=None):
    _check("hcsa_project_compress", load().hcsa_project_compress(
        ctypes.byref(p), kind, _ptr(x), _ptr(W_cat), _ptr(bias), _ptr(y), _ptr(entries), _ptr(idx_keys), _ptr(ws),
        _wsz(ws), _stream(stream)))


def hcsa_project_append(p, kind, cache: Cache, pos, x, W_cat, bias, y, ws=None, stream=None):
    _check("hcsa_project_append", load().hcsa_project_append(
        ctypes.byref(p), kind, ctypes.byref(cache), _ptr(pos), _ptr(x), _ptr(W_cat), _ptr(bias), _ptr(y), _ptr(ws),
        _wsz(ws), _stream(stream)))


def csa_decode_index_topk_shard(p, cache: Cache, pos, qi, w, sel, sel_scores, ws, stream=None):
    _check("csa_decode_index_topk_shard", load().csa_decode_index_topk_shard(
        ctypes.byref(p), ctypes.byref(cache), _ptr(pos), _ptr(qi), _ld(qi), _ptr(w), _ld(w), _ptr(sel),
        _ptr(sel_scores), _ptr(ws), _wsz(ws), _stream(stream)))


def csa_topk_merge(p, cand_sel, cand_scores, sel, stream=None):
    """cand_sel / cand_scores: [B, n_cand] (one row per sequence); sel: [B, topk]."""
    _check("csa_topk_merge", load().csa_topk_merge(ctypes.byref(p), _ptr(cand_sel), _ptr(cand_scores),
                                                   cand_sel.shape[1], _ptr(sel), _stream(stream)))


def csa_decode_attend_shard(p, cache: Cache, pos, q, sel, with_window, part, ws=None, stream=None):
    _check("csa_decode_attend_shard", load().csa_decode_attend_shard(
        ctypes.byref(p), ctypes.byref(cache), _ptr(pos), _ptr(q), _ld(q), _ptr(sel), int(with_window), _ptr(part),
        _ptr(ws), _wsz(ws), _stream(stream)))


def hca_decode_attend_shard(p, cache: Cache, pos, q, with_window, part, ws=None, stream=None):
    _check("hca_decode_attend_shard", load().hca_decode_attend_shard(
        ctypes.byref(p), ctypes.byref(cache), _ptr(pos), _ptr(q), _ld(q), int(with_window), _ptr(part), _ptr(ws),
        _wsz(ws), _stream(stream)))


def hcsa_merge_partials(p, parts, n_parts, out, stream=None):
    """parts: n_parts consecutive partial blocks of B * H * (dh + 2) floats; out: [B, H * dh]."""
    _check("hcsa_merge_partials", load().hcsa_merge_partials(ctypes.byref(p), _ptr(parts), n_parts, _ptr(out),
                                                             _ld(out), _stream(stream)))


def hcsa_launch_count(reset: bool = False) -> int:
    return int(load().hcsa_launch_count(1 if reset else 0))


# ---------------------------------------------------------------- sliding-window layers

_TORCH = {HCSA_F32: torch.float32, HCSA_BF16: torch.bfloat16}


def make_pages(k_pages, v_pages, page_table) -> Pages:
    """The two page arrays ([n_pages, Hkv, page, dh], or FP8 byte arrays) and the [B, max_pages] int32 table.  The
    handle keeps the tensors alive."""
    if page_table.dtype != torch.int32 or not (page_table.is_contiguous() and k_pages.is_contiguous()
                                               and v_pages.is_contiguous()):
        raise HcsaError("make_pages", 2)
    pages = Pages(k_pages=_ptr(k_pages), v_pages=_ptr(v_pages), page_table=_ptr(page_table))
    pages.tensors = (k_pages, v_pages, page_table)
    # what the calls check: element type, bytes of the smaller array, entries and row length of the table, device
    pages.dtype = k_pages.dtype if k_pages.dtype == v_pages.dtype else None
    pages.bytes = min(t.numel() * t.element_size() for t in (k_pages, v_pages))
    pages.entries = page_table.numel()
    pages.row = page_table.shape[1] if page_table.dim() == 2 and page_table.shape[0] > 1 else 0   # 0: any
    dev = {t.get_device() for t in pages.tensors}
    pages.device = dev.pop() if len(dev) == 1 else -1
    return pages


# These calls check what the C library cannot see (element types, extents, strides, devices).  A decode step makes many
# of them, so the checks are few attribute reads each and the stream comes from torch's raw accessors (looked up when
# called: a torch without CUDA has none): about 9 us a call on the host instead of 15, the launch included.


def _rows2d(fn, t, dtype, rows, cols):
    """A [rows, cols] tensor of the call's type whose columns are contiguous; a single row's stride does not matter.
    Returns its leading dimension."""
    if t.dtype is not dtype:
        raise HcsaError(fn, 3)
    shape, stride = t.shape, t.stride()
    if len(shape) != 2 or shape[0] < rows or shape[1] != cols or (stride[1] != 1 and cols > 1):
        raise HcsaError(fn, 2)
    return stride[0] if rows > 1 else cols


def _vec32(fn, t, n):
    if t.dtype is not torch.int32:
        raise HcsaError(fn, 3)
    if t.dim() != 1 or t.shape[0] < n or (n > 1 and t.stride(0) != 1):
        raise HcsaError(fn, 2)


def _check_pages(fn, p, pages):
    dt = torch.uint8 if p.lowprec else _TORCH.get(p.dtype)
    if pages.dtype is not dt:
        raise HcsaError(fn, 3)
    rows, dh = p.n_pages * p.Hkv * p.page, p.dh
    if (pages.bytes < rows * (dh + dh // 32 if p.lowprec else dh * dt.itemsize)
            or pages.entries < p.B * p.max_pages or (p.B > 1 and pages.row not in (0, p.max_pages))):
        raise HcsaError(fn, 2)


def _call(fn, dev, stream, tensors, call, *args):
    """The call on the tensors' device (which need not be the current one); its stream there unless one is given."""
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise HcsaError(fn, 2)
    if dev < 0:
        raise HcsaError(fn, 2)
    at = torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream
    if dev == torch._C._cuda_getDevice():
        code = call(*args, at)
    else:
        with torch.cuda.device(dev):
            code = call(*args, at)
    if code:
        raise HcsaError(fn, code)


def hcsa_page_bytes(p: Params) -> int:
    return int(load().hcsa_page_bytes(ctypes.byref(p)))


def swa_attend(p, q, k, v, out, stream=None):
    """q, out: [T, H * dh]; k, v: [T, Hkv * dh] (column views of one projection are fine)."""
    fn, dt, T, dh = "swa_attend", _TORCH.get(p.dtype), p.T, p.dh
    n, nkv = p.H * dh, p.Hkv * dh
    lq, lk, lv, lo = _rows2d(fn, q, dt, T, n), _rows2d(fn, k, dt, T, nkv), _rows2d(fn, v, dt, T, nkv), \
        _rows2d(fn, out, dt, T, n)
    _call(fn, q.get_device(), stream, (k, v, out), load().swa_attend, ctypes.byref(p), q.data_ptr(), lq, k.data_ptr(),
          lk, v.data_ptr(), lv, out.data_ptr(), lo)


def swa_page_append(p, pages: Pages, pos, k, v, seq=None, stream=None):
    """Write k, v [rows, Hkv * dh] to tokens pos[r] of sequences seq[r] (default: sequence r); pos[r] < 0: skipped."""
    fn, dt, nkv, rows = "swa_page_append", _TORCH.get(p.dtype), p.Hkv * p.dh, k.shape[0]
    lk, lv = _rows2d(fn, k, dt, rows, nkv), _rows2d(fn, v, dt, rows, nkv)
    _vec32(fn, pos, rows)
    if seq is not None:
        _vec32(fn, seq, rows)
    _check_pages(fn, p, pages)
    _call(fn, pages.device, stream, (k, v, pos, seq), load().swa_page_append, ctypes.byref(p), ctypes.byref(pages), rows,
          pos.data_ptr(), _ptr(seq), k.data_ptr(), lk, v.data_ptr(), lv)


def swa_decode_attend(p, pages: Pages, pos, q, out, ws=None, stream=None):
    """q, out: [B, H * dh]; pos[b]: position of the new token (already in the pages), -1 for an empty slot."""
    fn, dt, n, B = "swa_decode_attend", _TORCH.get(p.dtype), p.H * p.dh, p.B
    lq, lo = _rows2d(fn, q, dt, B, n), _rows2d(fn, out, dt, B, n)
    _vec32(fn, pos, B)
    _check_pages(fn, p, pages)
    _call(fn, pages.device, stream, (q, out, pos, ws), load().swa_decode_attend, ctypes.byref(p), ctypes.byref(pages),
          pos.data_ptr(), q.data_ptr(), lq, out.data_ptr(), lo, _ptr(ws), _wsz(ws))


def hcsa_add_rmsnorm(p, x, delta, w, eps, x_out, y, y8=None, stream=None):
    """x_out = x + delta, y = rmsnorm(x + delta) * w ([rows, D]); delta, x_out, y or y8 (a byte buffer of
    rows * (D + D / 32), FP8 layout) may be None."""
    fn, dt, D, rows = "hcsa_add_rmsnorm", _TORCH.get(p.dtype), p.D, x.shape[0]
    lx = _rows2d(fn, x, dt, rows, D)
    ld = 0 if delta is None else _rows2d(fn, delta, dt, rows, D)
    lo = 0 if x_out is None else _rows2d(fn, x_out, dt, rows, D)
    ly = 0 if y is None else _rows2d(fn, y, dt, rows, D)
    if w.dtype is not dt or (y8 is not None and y8.dtype is not torch.uint8):
        raise HcsaError(fn, 3)
    if w.dim() != 1 or w.shape[0] != D or not w.is_contiguous() or (
            y8 is not None and (y8.numel() < rows * (D + D // 32) or not y8.is_contiguous())):
        raise HcsaError(fn, 2)
    _call(fn, x.get_device(), stream, (delta, w, x_out, y, y8), load().hcsa_add_rmsnorm, ctypes.byref(p), rows,
          x.data_ptr(), lx, _ptr(delta), ld, w.data_ptr(), eps, _ptr(x_out), lo, _ptr(y), ly, _ptr(y8))
