"""The sliding-window calls without a GPU: every bad argument is refused on the host, with its code, before anything
is launched."""
import ctypes

import pytest
import torch

FAKE = 0x10000   # an aligned address that is never dereferenced
V = ctypes.c_void_p


@pytest.fixture(scope="module")
def h():
    import long_context_compressed_05_b200 as h
    from long_context_compressed_05_b200 import build
    build.build()
    return h


def params(h, **kw):
    base = dict(T=300, B=4, H=8, Hkv=2, dh=64, C=128, m=1, width=1, window=128, sinks=4, scale=0.125, page=16,
                n_pages=10, max_pages=4, dtype="bf16")
    dtype_code = kw.pop("dtype_code", None)
    p = h.make_params(**{**base, **kw})
    if dtype_code is not None:
        p.dtype = dtype_code
    return p


def attend(h, p, q=FAKE, ld_q=512, k=FAKE, ld_k=128, v=FAKE, ld_v=128, out=FAKE, ld_out=512):
    return h.load().swa_attend(ctypes.byref(p), V(q), ld_q, V(k), ld_k, V(v), ld_v, V(out), ld_out, None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype_code=7), 3), (dict(dh=63, C=126), 2), (dict(dh=32), 2), (dict(Hkv=3), 2), (dict(Hkv=0), 2),
    (dict(window=0), 2), (dict(sinks=-1), 2), (dict(T=-1), 2), (dict(H=258, Hkv=2), 8), (dict(dh=520, C=1040), 8),
    (dict(lowprec=1), 8), (dict(row0=64, row1=256), 2), (dict(row0=0, row1=301), 2), (dict(T=(1 << 30) + 1), 8)])
def test_attend_refuses_bad_parameters(h, kw, code):
    assert attend(h, params(h, **kw), ld_q=1 << 17, ld_k=1 << 17, ld_v=1 << 17, ld_out=1 << 17) == code


@pytest.mark.parametrize("kw,code", [
    (dict(q=0), 1), (dict(k=0), 1), (dict(v=0), 1), (dict(out=0), 1), (dict(q=FAKE + 2), 4), (dict(out=FAKE + 8), 4),
    (dict(ld_q=511), 4), (dict(ld_k=120), 4), (dict(ld_v=129), 4), (dict(ld_out=508), 4)])
def test_attend_refuses_bad_tensors(h, kw, code):
    assert attend(h, params(h), **kw) == code


def test_attend_of_nothing_is_no_error(h):
    assert attend(h, params(h, T=0)) == 0
    assert attend(h, params(h, T=256, row0=128, row1=128)) == 0


def pages(h, k=FAKE, v=FAKE, table=FAKE):
    return h.Pages(k_pages=k, v_pages=v, page_table=table)


def append(h, p, g, rows=4, pos=FAKE, seq=0, k=FAKE, ld_k=128, v=FAKE, ld_v=128):
    return h.load().swa_page_append(ctypes.byref(p), ctypes.byref(g), rows, V(pos), V(seq) if seq else None, V(k), ld_k,
                                    V(v), ld_v, None)


def decode(h, p, g, pos=FAKE, q=FAKE, ld_q=512, out=FAKE, ld_out=512, ws=FAKE, n=1 << 40):
    return h.load().swa_decode_attend(ctypes.byref(p), ctypes.byref(g), V(pos), V(q), ld_q, V(out), ld_out, V(ws), n,
                                      None)


@pytest.mark.parametrize("kw,code", [
    (dict(B=0), 2), (dict(page=8), 2), (dict(page=24), 2), (dict(page=0), 2), (dict(n_pages=0), 2),
    (dict(max_pages=0), 2), (dict(lowprec=1, dh=48, C=96), 8), (dict(lowprec=1, dtype="f32"), 8),
    (dict(n_pages=1 << 28), 8), (dict(max_pages=1 << 27), 8), (dict(H=258, Hkv=2), 8)])
def test_paged_calls_refuse_bad_parameters(h, kw, code):
    p = params(h, **kw)
    assert append(h, p, pages(h), rows=0, ld_k=1 << 17, ld_v=1 << 17) == code
    assert decode(h, p, pages(h), ld_q=1 << 17, ld_out=1 << 17) == code


def test_paged_calls_refuse_bad_tensors(h):
    p, g = params(h), pages(h)
    for bad, code in ((pages(h, k=None), 1), (pages(h, table=None), 1), (pages(h, v=FAKE + 4), 4),
                      (pages(h, table=FAKE + 2), 4)):
        assert append(h, p, bad) == code and decode(h, p, bad) == code
    assert append(h, p, g, pos=0) == 1 and append(h, p, g, k=0) == 1
    assert append(h, p, g, rows=5) == 2                       # more rows than sequences, and no seq
    assert append(h, p, g, rows=-1) == 2
    assert append(h, p, g, ld_k=127) == 4 and append(h, p, g, v=FAKE + 2) == 4 and append(h, p, g, seq=FAKE + 2) == 4
    assert append(h, p, g, rows=0) == 0
    assert decode(h, p, g, q=0) == 1 and decode(h, p, g, out=0) == 1 and decode(h, p, g, pos=0) == 1
    assert decode(h, p, g, ld_q=500) == 4 and decode(h, p, g, pos=FAKE + 2) == 4
    assert decode(h, p, g, ws=0) == 5
    assert decode(h, p, g, n=h.hcsa_workspace_bytes(p, h.OP_SWA_DECODE_ATTEND) - 1) == 5


def norm(h, p, rows=3, x=FAKE, ld_x=256, delta=FAKE, ld_d=256, w=FAKE, eps=1e-6, xo=FAKE, ld_xo=256, y=FAKE, ld_y=256,
         y8=0):
    return h.load().hcsa_add_rmsnorm(ctypes.byref(p), rows, V(x), ld_x, V(delta), ld_d, V(w), eps, V(xo), ld_xo, V(y),
                                     ld_y, V(y8), None)


def test_norm_refuses_bad_arguments(h):
    p = h.make_params(D=256)
    for kw, code in ((dict(x=0), 1), (dict(w=0), 1), (dict(y=0), 1), (dict(rows=-1), 2), (dict(eps=-1.0), 2),
                     (dict(eps=float("nan")), 2), (dict(x=FAKE + 2), 4), (dict(ld_x=255), 4), (dict(ld_y=257), 4),
                     (dict(ld_d=8), 4), (dict(ld_xo=8), 4), (dict(y8=FAKE + 8), 4)):
        assert norm(h, p, **kw) == code, kw
    assert norm(h, h.make_params(D=0)) == 2
    assert norm(h, h.make_params(D=252)) == 4                 # rows of 16-byte vectors
    assert norm(h, h.make_params(D=264), ld_x=264, ld_d=264, ld_xo=264, ld_y=264, y8=FAKE) == 8
    assert norm(h, h.make_params(D=256, dtype="f32"), y8=FAKE) == 8
    assert norm(h, h.make_params(D=16392), ld_x=16392, ld_d=16392, ld_xo=16392, ld_y=16392) == 8
    bad = h.make_params(D=256)
    bad.dtype = 5
    assert norm(h, bad) == 3
    assert norm(h, p, rows=0) == 0


def test_sizes_and_projection_columns(h):
    p = params(h)
    assert h.hcsa_page_bytes(p) == 10 * 2 * 16 * 64 * 2
    assert h.hcsa_page_bytes(params(h, lowprec=1)) == 10 * 2 * 16 * (64 + 2)
    assert h.hcsa_proj_cols(p, h.KIND_SWA) == (8 + 4) * 64
    spec = h.SlidingSpec(D=256, H=8, Hkv=2, dh=64)
    assert spec.ncols == h.hcsa_proj_cols(h.params_for(spec), h.KIND_SWA)
    assert h.hcsa_workspace_bytes(p, h.OP_SWA_DECODE_ATTEND) > 0


def test_python_wrappers_check_what_the_library_cannot_see(h):
    """Element types, row counts and strides of the tensors (CPU tensors: refused before the library is called)."""
    bf = torch.bfloat16
    p = params(h, T=8)
    q, kv = torch.zeros(8, 512, dtype=bf), torch.zeros(8, 128, dtype=bf)
    for args, code in (((q.float(), kv, kv, q), 3), ((q[:7], kv, kv, q), 2), ((q, kv[:, :64], kv, q), 2),
                       ((q, kv, torch.zeros(128, 8, dtype=bf).t(), q), 2), ((q, kv, kv, q.half()), 3)):
        with pytest.raises(h.HcsaError) as e:
            h.swa_attend(p, *args)
        assert e.value.code == code
    kp = torch.zeros(10, 2, 16, 64, dtype=bf)
    table = torch.zeros(4, 4, dtype=torch.int32)
    with pytest.raises(h.HcsaError):
        h.make_pages(kp, kp, table.long())
    g = h.make_pages(kp, kp, table)
    pos = torch.zeros(4, dtype=torch.int32)
    q4, kv4, ws = torch.zeros(4, 512, dtype=bf), torch.zeros(4, 128, dtype=bf), torch.zeros(16, dtype=torch.uint8)
    for call, code in ((lambda: h.swa_decode_attend(p, g, pos.long(), q4, q4, ws), 3),
                       (lambda: h.swa_decode_attend(p, g, pos[:3], q4, q4, ws), 2),
                       (lambda: h.swa_decode_attend(p, g, pos, q4[:3], q4, ws), 2),
                       (lambda: h.swa_page_append(p, g, pos[:2], kv4, kv4), 2),
                       (lambda: h.swa_page_append(p, h.make_pages(kp[:9].clone(), kp, table), pos, kv4, kv4), 2),
                       (lambda: h.swa_page_append(p, h.make_pages(kp.float(), kp, table), pos, kv4, kv4), 3),
                       (lambda: h.swa_decode_attend(p, h.make_pages(kp, kp, table[:3].clone()), pos, q4, q4, ws), 2)):
        with pytest.raises(h.HcsaError) as e:
            call()
        assert e.value.code == code
    pn = h.make_params(D=64)
    x, w = torch.zeros(3, 64, dtype=bf), torch.ones(64, dtype=bf)
    for call, code in ((lambda: h.hcsa_add_rmsnorm(pn, x, None, w.float(), 1e-6, x, x), 3),
                       (lambda: h.hcsa_add_rmsnorm(pn, x, None, w[:32], 1e-6, x, x), 2),
                       (lambda: h.hcsa_add_rmsnorm(pn, x, x[:2], w, 1e-6, x, x), 2),
                       (lambda: h.hcsa_add_rmsnorm(pn, x, None, w, 1e-6, None, None,
                                                   torch.zeros(3 * 65, dtype=torch.uint8)), 2)):
        with pytest.raises(h.HcsaError) as e:
            call()
        assert e.value.code == code


def test_norm_refuses_outputs_over_what_it_reads_again(h):
    p = h.make_params(D=256)
    other = 0x20000
    assert norm(h, p, xo=other, y=other) == 8
    assert norm(h, p, delta=0x30000, xo=0, y=FAKE, y8=0x40000) == 8          # y over x
    assert norm(h, p, delta=other, xo=0, y=other, y8=0x40000) == 8           # y over delta


def test_calls_of_no_rows_take_tensors_without_an_address(h):
    assert attend(h, params(h, T=0), q=0, k=0, v=0, out=0) == 0
    assert append(h, params(h), pages(h), rows=0, pos=0, k=0, v=0) == 0
    assert norm(h, h.make_params(D=256), rows=0, x=0, delta=0, xo=0, y=0) == 0


def test_the_package_works_on_a_torch_without_cuda(h):
    """Import, host-side checks and refusals where torch has none of its CUDA accessors."""
    import os
    import subprocess
    import sys
    code = """
import torch
for n in [n for n in dir(torch._C) if n.startswith("_cuda_get")]:
    delattr(torch._C, n)
import long_context_compressed_05_b200 as h
p = h.make_params(D=64)
x = torch.zeros(3, 64, dtype=torch.bfloat16)
try:
    h.hcsa_add_rmsnorm(p, x, None, torch.ones(64, dtype=torch.bfloat16), 1e-6, None, x.clone())
except h.HcsaError as e:
    assert e.code == 2
else:
    raise SystemExit("CPU tensors were taken")
"""
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True,
                       cwd=os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
    assert r.returncode == 0, r.stderr[-2000:]


def test_a_page_table_of_another_row_length_is_refused(h):
    """Its entries would be read as other sequences' pages."""
    p = params(h)                                             # B 4, max_pages 4
    kp = torch.zeros(10, 2, 16, 64, dtype=torch.bfloat16)
    pos = torch.zeros(4, dtype=torch.int32)
    kv, q = torch.zeros(4, 128, dtype=torch.bfloat16), torch.zeros(4, 512, dtype=torch.bfloat16)
    ws = torch.zeros(16, dtype=torch.uint8)
    for shape, refused in (((4, 5), True), ((8, 2), True), ((4, 4), False), ((6, 4), False), ((16,), False)):
        pages = h.make_pages(kp, kp, torch.zeros(shape, dtype=torch.int32))
        from long_context_compressed_05_b200 import _lib
        if not refused:
            _lib._check_pages("test", p, pages)
            continue
        for call in (lambda: h.swa_page_append(p, pages, pos, kv, kv), lambda: h.swa_decode_attend(p, pages, pos, q, q, ws),
                     lambda: _lib._check_pages("test", p, pages)):
            with pytest.raises(h.HcsaError) as e:
                call()
            assert e.value.code == 2
    one = params(h, B=1)                                      # a single sequence's table may be longer than it needs
    _lib._check_pages("test", one, h.make_pages(kp, kp, torch.zeros(1, 9, dtype=torch.int32)))


def test_norm_in_place_needs_the_same_leading_dimension(h):
    """Rows of an output over an input's address that start elsewhere would be written before they are read."""
    p = h.make_params(D=256)
    other = 0x20000
    assert norm(h, p, xo=FAKE, ld_xo=512, y=other) == 8                          # x_out over x
    assert norm(h, p, delta=other, ld_d=512, xo=other, y=0x30000) == 8           # x_out over delta
    assert norm(h, p, delta=0x30000, xo=0, y=FAKE, ld_y=264) == 8                # y over x
    assert norm(h, p, delta=other, ld_d=512, xo=0, y=other) == 8                 # y over delta


def test_attend_refuses_an_output_over_its_inputs(h):
    """Rows may be computed again after others are stored, so the inputs have to last."""
    far = dict(q=0x20000, k=0x30000, v=0x40000)
    for name in ("q", "k", "v"):
        assert attend(h, params(h), **{**far, name: FAKE}) == 8
