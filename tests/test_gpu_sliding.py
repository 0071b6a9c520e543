"""The sliding-window layer's calls against a plain computation in 64 bits: norm, prefill attention, paged cache
writes, one-token attention, and a run of them together.

Tolerances, from the arithmetic of the kernels (u = half a step of the storage type: 2^-8 bf16, 2^-24 fp32;
v = 2^-24, of the fp32 sums; A = sum_j w_j |v_j| of the output element, which bounds every partial sum):
  stored result          u |out|
  weights as bf16        2^-8 A  (tensor-core paths only: each weight is rounded once, the sum of the weights is not)
  scores                 a dot product of dh terms in fp32 is off by (dh + 2) v S, S = scale sum_d |q_d k_d|, and so
                         is the weight, relatively; once in the numerator and once in the sum of the weights.
                         The tensor core's adder may drop the bits that do not fit instead of rounding: 2 v a term
  sums over n keys       (n + 8) 2 v A, numerator and sum of the weights: twice
  exponential            2^-22 relative, and the rounding of its argument (|s| v log2 e twice): below (S + 4) 4 v
"""
import math

import pytest
import torch

pytestmark = pytest.mark.gpu

NO_WINDOW = 2 ** 31 - 1
HCSA_ERR_DEVICE = 9


@pytest.fixture(scope="module")
def h():
    import long_context_compressed_05_b200 as h
    torch.cuda.set_device(0)
    assert h.hcsa_get_device_status() == 0
    yield h
    torch.cuda.synchronize()
    assert h.hcsa_get_device_status() == 0


def dt(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape, dtype=torch.bfloat16):
    return torch.randn(shape, generator=g, device="cuda").to(dtype)


def seen_mask(t, n, window, sinks):
    """[len(t), n] truth: query at position t[i] sees key j."""
    j = torch.arange(n, device="cuda")
    t = t[:, None]
    return (j <= t) & ((j > t - window) | (j < sinks))


def attend64(q, k, v, mask, scale):
    """q [R, H, dh], k / v [n, Hkv, dh], mask [R, n] -> (out, bound of |error| per element without the stored
    rounding and without rounded weights, A), all [R, H, dh] in 64 bits.  Keys that are not seen take no part."""
    R, H, dh = q.shape
    G = H // k.shape[1]
    q, k, v = q.double(), k.double(), v.double()
    out, A, rel = (torch.zeros(R, H, dh, dtype=torch.float64, device="cuda") for _ in range(3))
    for hq in range(H):
        kh, vh = k[:, hq // G], v[:, hq // G]
        used = mask.any(0)
        kk, vv, m = kh[used], vh[used], mask[:, used]
        kk, vv = torch.nan_to_num(kk, 0, 0, 0), vv
        s = (q[:, hq] @ kk.T * scale).masked_fill(~m, -math.inf)
        S = ((q[:, hq].abs() @ kk.abs().T) * abs(scale)).masked_fill(~m, 0).amax(1, keepdim=True)
        w = torch.nan_to_num(torch.softmax(s, 1), 0.0)
        out[:, hq], A[:, hq] = w @ vv, w @ vv.abs()
        n = m.sum(1, keepdim=True)
        rel[:, hq] = 2.0 ** -24 * (2 * 2 * (dh + 2) * S + 2 * 2 * (n + 8) + 4 * (S + 4) * 2)
    return out, rel * A, A


def check(got, q, k, v, mask, scale, dtype, what=""):
    """Every element of got [R, H dh] within the bounds above."""
    want, err, A = attend64(q, k, v, mask, scale)
    u = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -24
    err = err + (2.0 ** -8 * A if dtype == "bf16" else 0)
    tol = err + u * (want.abs() + err) + 1e-30
    diff = (got.double().view_as(want) - want).abs()
    bad = ~(diff <= tol)
    assert not bad.any(), f"{what}: {int(bad.sum())} of {bad.numel()} off, first at {bad.nonzero()[0].tolist()}, " \
        f"worst ratio {float((diff / tol).nan_to_num(math.inf).max()):.3g}"


# ---------------------------------------------------------------- norm

@pytest.mark.parametrize("dtype,fp8", [("bf16", False), ("bf16", True), ("f32", False)])
@pytest.mark.parametrize("rows,D", [(1, 32), (3, 64), (5, 2048), (33, 96), (1100, 416), (1, 16384), (2, 8224)])
def test_norm(h, rows, D, dtype, fp8):
    g = gen(rows * 131 + D)
    x, d = randn(g, rows, D, dtype=dt(dtype)), randn(g, rows, D, dtype=dt(dtype))
    w = (1 + 0.3 * torch.randn(D, generator=g, device="cuda")).to(dt(dtype))
    x[rows // 2, : D // 2] *= 64
    p = h.make_params(D=D, dtype=dtype)
    xo, y = torch.empty_like(x), torch.empty_like(x)
    y8 = torch.full((rows * (D + D // 32) + 16,), 0x77, dtype=torch.uint8, device="cuda") if fp8 else None
    h.hcsa_add_rmsnorm(p, x, d, w, 1e-5, xo, y, y8)
    s = x.double() + d.double()
    want = s / (s.square().mean(-1, keepdim=True) + 1e-5).sqrt() * w.double()
    # the sum's one rounding in fp32, then the storage's
    assert torch.equal(xo, (x.float() + d.float()).to(x.dtype))
    # mean of D squares: a thread's at most 32 in a row, then a tree (log2 1024 + 32 roundings of v), halved by the
    # root; x + delta, 1 / sqrt, the two products: 6 more; all below 64 v
    rel = (2.0 ** -8 if dtype == "bf16" else 2.0 ** -24) + 64 * 2.0 ** -24
    assert ((y.double() - want).abs() <= rel * 1.01 * want.abs() + 1e-38).all()
    if not fp8:
        return
    codes = y8[:rows * D].view(torch.float8_e4m3fn).double().view(rows, D // 32, 32)
    exps = y8[rows * D:rows * (D + D // 32)].view(torch.int8).double().view(rows, D // 32)
    assert (y8[rows * (D + D // 32):] == 0x77).all()
    b = want.view(rows, D // 32, 32)
    amax = b.abs().amax(-1)
    e = torch.ceil(torch.log2(amax / 448))
    e = torch.where(amax > 448 * torch.exp2(e), e + 1, torch.where(amax <= 224 * torch.exp2(e), e - 1, e))
    assert torch.equal(exps, e)
    scaled = b / torch.exp2(e)[..., None]
    # half a step: 2^-4 of the value, or half the subnormal step 2^-9; the value itself within 64 v
    tol = torch.maximum(scaled.abs() * 2.0 ** -4, torch.full_like(scaled, 2.0 ** -10)) + 64 * 2.0 ** -24 * scaled.abs()
    assert ((codes - scaled).abs() <= tol).all()


def test_norm_in_place_without_delta_and_strided(h):
    g = gen(5)
    wide = randn(g, 7, 3 * 256)
    x, d, y = wide[:, :256], wide[:, 256:512], wide[:, 512:]
    w = randn(g, 256)
    p = h.make_params(D=256)
    x0, d0 = x.clone(), d.clone()
    h.hcsa_add_rmsnorm(p, x, None, w, 0.0, None, y)
    want = x0.double() / x0.double().square().mean(-1, keepdim=True).sqrt() * w.double()
    assert torch.equal(x, x0)
    assert ((y.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -17) * want.abs()).all()
    h.hcsa_add_rmsnorm(p, x, d, w, 1e-6, x, y)                     # the stream updated in place
    assert torch.equal(x, x0 + d0) and torch.equal(d, d0)


def test_norm_of_zeros_and_block_borders(h):
    p = h.make_params(D=64)
    x = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    x[1] = 1.0                                                     # y = w exactly with eps 0
    w = torch.full((64,), 1.75, dtype=torch.bfloat16, device="cuda")
    w[32:] = 448.0
    y8 = torch.zeros(3 * 66, dtype=torch.uint8, device="cuda")
    h.hcsa_add_rmsnorm(p, x, None, w, 1e-12, None, None, y8)
    exps = y8[3 * 64:].view(torch.int8).view(3, 2)
    assert exps[0].tolist() == [0, 0] and (y8[:64] == 0).all()
    # y is just below 1.75 and 448 (eps), so 2^-8 and 1 hold them
    assert exps[1].tolist() == [-8, 0]
    h.hcsa_add_rmsnorm(p, x[1:2], None, w, 0.0, None, None, y8)    # exactly on the border: still held
    assert y8[64:66].view(torch.int8).tolist() == [-8, 0]


# ---------------------------------------------------------------- prefill attention

SHAPES = [  # T, H, Hkv, dh, window, sinks
    (1, 1, 1, 64, 1, 0), (2, 4, 1, 128, 1, 1), (3, 6, 2, 64, 2, 0), (127, 8, 8, 128, 128, 4), (128, 8, 2, 64, 64, 0),
    (129, 8, 1, 128, NO_WINDOW, 0), (300, 16, 1, 64, 7, 3), (517, 8, 2, 64, 128, 4), (640, 5, 1, 128, 200, 129),
    (1000, 14, 2, 128, NO_WINDOW, 5), (777, 3, 3, 64, 33, 200), (700, 128, 1, 64, 50, 1), (260, 128, 2, 128, 31, 40),
    (1500, 6, 1, 128, 700, 2), (400, 4, 2, 72, 100, 3), (200, 2, 1, 256, 60, 2), (90, 2, 2, 512, 40, 1),
    (150, 2, 1, 8, 40, 1), (2100, 16, 2, 64, NO_WINDOW, 0), (1300, 8, 2, 128, 1024, 1000), (1200, 4, 4, 64, 512, 0)]


def attend_params(h, T, H, Hkv, dh, window, sinks, dtype, scale=None, **kw):
    return h.make_params(T=T, H=H, Hkv=Hkv, dh=dh, C=2 * dh, m=1, width=1, window=window, sinks=sinks, dtype=dtype,
                         scale=dh ** -0.5 if scale is None else scale, **kw)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("T,H,Hkv,dh,window,sinks", SHAPES)
def test_attend(h, T, H, Hkv, dh, window, sinks, dtype):
    g = gen(T + dh)
    y = randn(g, T, (H + 2 * Hkv) * dh, dtype=dt(dtype))
    n = Hkv * dh
    k, v, q = y[:, :n], y[:, n:2 * n], y[:, 2 * n:]
    wide = torch.full((T, H * dh + 64), 7.0, dtype=y.dtype, device="cuda")
    out = wide[:, 32:32 + H * dh]
    p = attend_params(h, T, H, Hkv, dh, window, sinks, dtype)
    h.swa_attend(p, q, k, v, out)
    mask = seen_mask(torch.arange(T, device="cuda"), T, window, sinks)
    check(out, q.reshape(T, H, dh), k.reshape(T, Hkv, dh), v.reshape(T, Hkv, dh), mask, p.scale, dtype)
    assert (wide[:, :32] == 7).all() and (wide[:, 32 + H * dh:] == 7).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 4.0])
def test_attend_scales(h, scale):
    """Equal weights, a negative scale, and one that leaves a few keys most of the weight."""
    T, H, Hkv, dh = 333, 8, 2, 64
    g = gen(9)
    q, k, v = randn(g, T, H * dh), randn(g, T, Hkv * dh), randn(g, T, Hkv * dh)
    out = torch.empty_like(q)
    p = attend_params(h, T, H, Hkv, dh, 150, 2, "bf16", scale=scale)
    h.swa_attend(p, q, k, v, out)
    mask = seen_mask(torch.arange(T, device="cuda"), T, 150, 2)
    check(out, q.view(T, H, dh), k.view(T, Hkv, dh), v.view(T, Hkv, dh), mask, p.scale, "bf16")


@pytest.mark.parametrize("dtype,dh", [("bf16", 128), ("bf16", 64), ("f32", 64), ("bf16", 72)])
def test_attend_rising_scores(h, dtype, dh):
    """Each key scores far above all earlier ones, so that the running maximum rises at every tile."""
    T, H, Hkv = 700, 4, 1
    g = gen(10)
    q = randn(g, T, H * dh, dtype=dt(dtype)) * 0.1
    k, v = randn(g, T, dh, dtype=dt(dtype)) * 0.1, randn(g, T, dh, dtype=dt(dtype))
    q.view(T, H, dh)[:, :, 0] = 4.0
    k[:, 0] = torch.arange(T, device="cuda").to(k.dtype) * 0.25
    out = torch.empty_like(q)
    p = attend_params(h, T, H, Hkv, dh, NO_WINDOW, 0, dtype, scale=1.0)
    h.swa_attend(p, q, k, v, out)
    mask = seen_mask(torch.arange(T, device="cuda"), T, NO_WINDOW, 0)
    check(out, q.view(T, H, dh), k.view(T, Hkv, dh), v.view(T, Hkv, dh), mask, p.scale, dtype)


@pytest.mark.parametrize("dtype,H,Hkv,dh,window,sinks", [("bf16", 8, 2, 64, 128, 4), ("f32", 4, 4, 64, 100, 0),
                                                         ("bf16", 8, 1, 128, NO_WINDOW, 0), ("bf16", 4, 1, 72, 30, 3)])
def test_attend_row_range(h, dtype, H, Hkv, dh, window, sinks):
    """A row range gives the rows of the whole call and writes no other row."""
    T = 900
    g = gen(11)
    q, k, v = (randn(g, T, n * dh, dtype=dt(dtype)) for n in (H, Hkv, Hkv))
    full = torch.empty_like(q)
    h.swa_attend(attend_params(h, T, H, Hkv, dh, window, sinks, dtype), q, k, v, full)
    mask = seen_mask(torch.arange(T, device="cuda"), T, window, sinks)
    for r0, r1 in ((0, 128), (128, 640), (640, 900), (896, 900)):
        part = torch.full_like(q, 3.0)
        k2, v2 = k.clone(), v.clone()                  # rows that the range may not read
        lo = max(0, r0 - window + 1)
        for t in (k2, v2):
            t[r1:] = math.nan
            t[min(sinks, lo):lo] = math.nan
        h.swa_attend(attend_params(h, T, H, Hkv, dh, window, sinks, dtype, row0=r0, row1=r1), q, k2, v2, part)
        assert (part[:r0] == 3).all() and (part[r1:] == 3).all()
        check(part[r0:r1], q[r0:r1].reshape(-1, H, dh), k.view(T, Hkv, dh), v.view(T, Hkv, dh), mask[r0:r1],
              dh ** -0.5, dtype)
    assert torch.isfinite(full.float()).all()


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf, "lowest"])
@pytest.mark.parametrize("dtype,dh,window,sinks", [("bf16", 64, 40, 2), ("bf16", 128, NO_WINDOW, 0), ("bf16", 128, 128, 4),
                                                   ("f32", 64, 100, 0), ("bf16", 72, 30, 0)])
def test_attend_unseen_values_do_not_reach_a_row(h, dtype, dh, window, sinks, bad):
    """Keys and values that are infinite, NaN or the type's lowest value: rows that do not see them are as without
    them, rows that see a NaN or an infinite value are not finite."""
    T, H, Hkv = 450, 4, 2
    g = gen(12)
    q, k, v = (randn(g, T, n * dh, dtype=dt(dtype)) for n in (H, Hkv, Hkv))
    x = torch.finfo(dt(dtype)).min if bad == "lowest" else bad
    at = [77, 130, 301, 302]
    k2, v2 = k.clone(), v.clone()
    k2[at[::2]] = x
    v2[at] = x
    out, clean = torch.empty_like(q), torch.empty_like(q)
    p = attend_params(h, T, H, Hkv, dh, window, sinks, dtype)
    h.swa_attend(p, q, k, v, clean)
    h.swa_attend(p, q, k2, v2, out)
    mask = seen_mask(torch.arange(T, device="cuda"), T, window, sinks)
    hit = mask[:, at].any(1)
    check(out[~hit], q.view(T, H, dh)[~hit], k.view(T, Hkv, dh), v.view(T, Hkv, dh), mask[~hit], p.scale, dtype)
    if bad != "lowest":
        assert not torch.isfinite(out[mask[:, 130] | mask[:, 302]].float()).any()


def test_attend_all_values_nan_ends(h):
    T, H, dh = 3000, 2, 128
    q = torch.ones(T, H * dh, dtype=torch.bfloat16, device="cuda")
    kv = torch.full((T, dh), math.nan, dtype=torch.bfloat16, device="cuda")
    out = torch.zeros_like(q)
    h.swa_attend(attend_params(h, T, H, 1, dh, NO_WINDOW, 0, "bf16"), q, kv, kv, out)
    assert torch.isnan(out.float()).all()


def test_attend_is_deterministic_on_a_side_stream_and_in_a_graph(h):
    T, H, Hkv, dh = 1111, 8, 2, 128
    g = gen(13)
    q, k, v = (randn(g, T, n * dh) for n in (H, Hkv, Hkv))
    p = attend_params(h, T, H, Hkv, dh, 300, 4, "bf16")
    ref, out = torch.empty_like(q), torch.empty_like(q)
    h.swa_attend(p, q, k, v, ref)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        h.swa_attend(p, q, k, v, out)
    side.synchronize()
    assert torch.equal(out, ref)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        h.swa_attend(p, q, k, v, out)
    q.copy_(randn(g, T, H * dh))
    graph.replay()
    h.swa_attend(p, q, k, v, ref)
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


# ---------------------------------------------------------------- paged cache

def rows_of(pool, n_pages, Hkv, page, dh, lowprec):
    """The pool's values in 64 bits, [n_pages, Hkv, page, dh]."""
    if not lowprec:
        return pool.double().view(n_pages, Hkv, page, dh)
    n = n_pages * Hkv * page
    codes = pool[:n * dh].view(torch.float8_e4m3fn).double().view(n, dh // 32, 32)
    exps = pool[n * dh:n * (dh + dh // 32)].view(torch.int8).double().view(n, dh // 32, 1)
    return (codes * torch.exp2(exps)).view(n_pages, Hkv, page, dh)


class Paged:
    """A paged cache of random keys and values with shuffled pages; what no sequence holds is NaN."""

    def __init__(self, h, pos, H, Hkv, dh, window, sinks, page, dtype, lowprec=False, seed=0, spare=2):
        g = gen(seed)
        self.h, self.pos_h = h, pos
        B, P = len(pos), max(max(pos) + 1, 1)
        most = -(-P // page) + 1
        need = [-(-(x + 1) // page) for x in pos]
        self.n_pages = n_pages = sum(need) + spare
        order = torch.randperm(n_pages, generator=g, device="cuda").tolist()
        table = torch.full((B, most), -1, dtype=torch.int32)
        for b, n in enumerate(need):
            table[b, :n] = torch.tensor([order.pop() for _ in range(n)], dtype=torch.int32)
        self.table = table.cuda()
        self.p = h.make_params(B=B, H=H, Hkv=Hkv, dh=dh, C=2 * dh, m=1, width=1, window=window, sinks=sinks,
                               scale=dh ** -0.5, page=page, n_pages=n_pages, max_pages=most, dtype=dtype, lowprec=lowprec)
        self.k, self.v = (randn(g, B, P, Hkv, dh, dtype=dt(dtype)) for _ in range(2))
        if lowprec:   # NaN codes
            self.pools = [torch.full((h.hcsa_page_bytes(self.p),), 0x7F, dtype=torch.uint8, device="cuda") for _ in "kv"]
        else:
            self.pools = [torch.full((n_pages, Hkv, page, dh), math.nan, dtype=dt(dtype), device="cuda") for _ in "kv"]
        self.pages = h.make_pages(*self.pools, self.table)
        seq = torch.cat([torch.full((x + 1,), b, dtype=torch.int32) for b, x in enumerate(pos)]).cuda()
        at = torch.cat([torch.arange(x + 1, dtype=torch.int32) for x in pos]).cuda()
        n = Hkv * dh
        if len(seq):
            kv = torch.cat([self.k[seq.long(), at.long()].reshape(-1, n), self.v[seq.long(), at.long()].reshape(-1, n)], 1)
            h.swa_page_append(self.p, self.pages, at, kv[:, :n], kv[:, n:], seq)
        self.pos = torch.tensor(pos, dtype=torch.int32, device="cuda")
        self.q = randn(g, B, H * dh, dtype=dt(dtype))
        self.ws = torch.full((h.hcsa_workspace_bytes(self.p, h.OP_SWA_DECODE_ATTEND),), 0xFF, dtype=torch.uint8,
                             device="cuda")

    def decode(self, out=None, q=None):
        q = self.q if q is None else q
        out = torch.full_like(q, 9.0) if out is None else out
        self.h.swa_decode_attend(self.p, self.pages, self.pos, q, out, self.ws)
        return out

    def check(self, out):
        p = self.p
        lowprec = bool(p.lowprec)
        k, v = (rows_of(x, self.n_pages, p.Hkv, p.page, p.dh, lowprec) for x in self.pools)
        for b, x in enumerate(self.pos_h):
            if x < 0:
                assert (out[b] == 0).all()
                continue
            j = torch.arange(x + 1, device="cuda")
            ids = self.table[b, j // p.page].long()
            kk, vv = (t[ids, :, j % p.page] for t in (k, v))
            mask = seen_mask(torch.tensor([x], device="cuda"), x + 1, p.window, p.sinks)
            check(out[b:b + 1], self.q[b:b + 1].view(1, p.H, p.dh), kk, vv, mask, p.scale,
                  "bf16" if p.dtype == 1 else "f32", f"sequence {b}")


CACHES = [  # positions, H, Hkv, dh, window, sinks, page
    ([0], 1, 1, 64, 1, 0, 16), ([5, -1, 0], 8, 2, 128, 3, 1, 16), ([-1, -1], 4, 1, 64, 100, 0, 32),
    ([127, 128, 129], 16, 2, 128, 128, 4, 48), ([4098, 17, 700], 64, 8, 128, 128, 4, 16),
    ([1000, 3, -1, 2047, 512], 14, 2, 64, NO_WINDOW, 0, 64), ([5000, 40], 16, 1, 128, NO_WINDOW, 0, 128),
    ([3000, 2999], 6, 3, 128, 1000, 200, 256), ([900], 128, 1, 64, NO_WINDOW, 0, 16), ([700, 33], 7, 1, 128, 257, 300, 32),
    ([20000], 2, 1, 128, NO_WINDOW, 0, 64), ([300] * 40, 8, 8, 64, NO_WINDOW, 0, 16), ([2500, 10], 5, 1, 64, 2000, 7, 80),
    ([1200, 77], 40, 2, 128, NO_WINDOW, 0, 16), ([600, 601], 4, 2, 96, 128, 4, 16), ([300, 299], 4, 1, 256, 200, 20, 32),
    ([200, 3], 4, 1, 512, NO_WINDOW, 0, 16)]


@pytest.mark.parametrize("kind", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("pos,H,Hkv,dh,window,sinks,page", CACHES)
def test_decode(h, pos, H, Hkv, dh, window, sinks, page, kind):
    c = Paged(h, pos, H, Hkv, dh, window, sinks, page, "f32" if kind == "f32" else "bf16", kind == "fp8", seed=len(pos) + H)
    c.check(c.decode())


def test_decode_more_sequences_than_a_block_has_threads(h):
    pos = [(7 * b) % 90 - 1 for b in range(700)]
    c = Paged(h, pos, 4, 1, 64, NO_WINDOW, 0, 16, "bf16", seed=3)
    c.check(c.decode())
    c = Paged(h, pos, 4, 1, 64, 30, 1, 16, "bf16", seed=4)
    c.check(c.decode())


@pytest.mark.parametrize("kind", ["bf16", "f32", "fp8"])
@pytest.mark.parametrize("dh", [64, 128, 160])
def test_append(h, kind, dh):
    """Stored values: the rows as they are, or one rounding to 8 bits; skipped rows and all other tokens untouched."""
    B, Hkv, page, n_pages = 3, 2, 16, 9
    dtype, low = ("f32" if kind == "f32" else "bf16"), kind == "fp8"
    g = gen(21)
    table = torch.tensor([[4, 0, -1], [8, -1, -1], [2, 7, 1]], dtype=torch.int32, device="cuda")
    p = h.make_params(B=B, H=Hkv, Hkv=Hkv, dh=dh, C=2 * dh, m=1, width=1, page=page, n_pages=n_pages, max_pages=3,
                      dtype=dtype, lowprec=low)
    if low:
        pools = [torch.full((h.hcsa_page_bytes(p) + 16,), 0x7F, dtype=torch.uint8, device="cuda") for _ in "kv"]
    else:
        pools = [torch.full((n_pages, Hkv, page, dh), math.nan, dtype=dt(dtype), device="cuda") for _ in "kv"]
    pages = h.make_pages(*pools, table)
    rows = [(0, 0), (0, 31), (1, 15), (2, 16), (2, 47), (0, -1), (-1, 3), (2, 40)]
    seq, pos = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in zip(*rows))
    kv = randn(g, len(rows), 2 * Hkv * dh + 8, dtype=dt(dtype)) * torch.logspace(-3, 3, len(rows), device="cuda").to(dt(dtype))[:, None]
    k, v = kv[:, :Hkv * dh], kv[:, Hkv * dh:2 * Hkv * dh]
    k[3, 32:64] = 0
    h.swa_page_append(p, pages, pos, k, v, seq)
    if low:
        assert all((x[-16:] == 0x7F).all() for x in pools)
    for pool, x in zip(pools, (k, v)):
        got = rows_of(pool, n_pages, Hkv, page, dh, low)
        touched = torch.zeros(n_pages, page, dtype=torch.bool)
        for r, (b, t) in enumerate(rows):
            if b < 0 or t < 0:
                continue
            i = int(table[b, t // page])
            touched[i, t % page] = True
            w = x[r].double().view(Hkv, dh)
            if not low:
                assert torch.equal(got[i, :, t % page], w)
                continue
            blk = w.view(Hkv, dh // 32, 32)
            amax = blk.abs().amax(-1, keepdim=True)
            e = torch.ceil(torch.log2(amax / 448)).nan_to_num(neginf=0.0)
            tol = torch.maximum(blk.abs() * 2.0 ** -4, torch.exp2(e - 10))
            assert ((got[i, :, t % page].view_as(blk) - blk).abs() <= tol).all()
        assert torch.isnan(got[~touched.cuda()[:, None].expand(-1, Hkv, -1)]).all()


def test_append_fp8_extremes(h):
    """Infinite values stay infinite, NaN stays NaN, blocks of tiny values keep what the exponent range holds."""
    p = h.make_params(B=1, H=1, Hkv=1, dh=32, C=64, m=1, width=1, page=16, n_pages=1, max_pages=1, lowprec=True)
    pools = [torch.zeros(h.hcsa_page_bytes(p), dtype=torch.uint8, device="cuda") for _ in "kv"]
    pages = h.make_pages(*pools, torch.zeros(1, 1, dtype=torch.int32, device="cuda"))
    x = torch.ones(4, 32, dtype=torch.bfloat16, device="cuda")
    x[0, 0], x[0, 1] = math.inf, -math.inf
    x[1, 5] = math.nan
    x[2] = 1e-38
    x[3] = torch.finfo(torch.bfloat16).max
    seq = torch.zeros(4, dtype=torch.int32, device="cuda")
    h.swa_page_append(p, pages, torch.arange(4, dtype=torch.int32, device="cuda"), x, x, seq)
    got = rows_of(pools[0], 1, 1, 16, 32, True)[0, 0].float()
    assert got[0, 0] == math.inf and got[0, 1] == -math.inf
    assert torch.isnan(got[1, 5]) and (got[1, :5] == 1).all()
    assert ((got[2] / 1e-38 - 1).abs() <= 2.0 ** -4 + 2.0 ** -8).all()
    assert torch.isfinite(got[3]).all() and ((got[3] / x[3].float() - 1).abs() <= 2.0 ** -4).all()


def test_append_and_decode_report_what_lies_outside(h):
    """A position past the table or a page outside the pool: nothing of it is read or written, the status word says so,
    the other sequences are right."""
    c = Paged(h, [40, 60, 90], 8, 2, 64, NO_WINDOW, 0, 16, "bf16", seed=6)
    before = [x.clone() for x in c.pools]
    n = 2 * 64
    k = randn(gen(1), 3, n)
    bad = torch.tensor([16 * c.table.shape[1], 2 ** 31 - 1, -5], dtype=torch.int32, device="cuda")
    h.swa_page_append(c.p, c.pages, bad, k, k)
    torch.cuda.synchronize()
    assert h.hcsa_get_device_status() == HCSA_ERR_DEVICE
    far = torch.tensor([3, 2 ** 31 - 1, -1], dtype=torch.int32, device="cuda")
    h.swa_page_append(c.p, c.pages, torch.zeros(3, dtype=torch.int32, device="cuda"), k, k, far)
    torch.cuda.synchronize()
    assert h.hcsa_get_device_status() == HCSA_ERR_DEVICE
    assert all(torch.equal(a.view(torch.int16), b.view(torch.int16)) for a, b in zip(before, c.pools))
    want = c.decode()
    for bad_id in (c.n_pages, -1, 2 ** 31 - 1):
        keep = c.table.clone()
        c.table[1, 1] = bad_id
        out = c.decode()
        torch.cuda.synchronize()
        assert h.hcsa_get_device_status() == HCSA_ERR_DEVICE
        assert torch.equal(out[0], want[0]) and torch.equal(out[2], want[2])
        c.table.copy_(keep)
    c.pos[1] = 16 * c.table.shape[1]
    out = c.decode()
    torch.cuda.synchronize()
    assert h.hcsa_get_device_status() == HCSA_ERR_DEVICE
    # the split over CTAs follows the lengths: equal up to the order of the sums
    for b in (0, 2):
        assert ((out[b].float() - want[b].float()).abs() <= 2.0 ** -6 * (want[b].float().abs() + 1)).all()


@pytest.mark.parametrize("dh,kind", [(128, "bf16"), (64, "f32"), (128, "fp8")])
def test_decode_unseen_rows_hold_anything(h, dh, kind):
    """Tokens between the first ones and the window hold NaN: no trace of them."""
    c = Paged(h, [900, 333], 8, 2, dh, 100, 5, 32, "f32" if kind == "f32" else "bf16", kind == "fp8", seed=8)
    seq, at = [], []
    for b, x in enumerate(c.pos_h):
        t = list(range(5, x - 100 + 1))
        at += t
        seq += [b] * len(t)
    seq, at = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (seq, at))
    nan = torch.full((len(seq), 2 * dh), math.nan, dtype=c.q.dtype, device="cuda")
    h.swa_page_append(c.p, c.pages, at, nan, nan, seq)
    c.check(c.decode())


def test_decode_graph_streams_and_two_calls_at_once(h):
    a = Paged(h, [3000, 20, 999], 16, 2, 128, NO_WINDOW, 0, 16, "bf16", seed=9)
    b = Paged(h, [2500, 700, -1], 16, 2, 128, NO_WINDOW, 0, 16, "bf16", seed=10)
    want_a, want_b = a.decode(), b.decode()
    torch.cuda.synchronize()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    outs = [torch.zeros_like(a.q), torch.zeros_like(b.q)]
    for _ in range(5):
        with torch.cuda.stream(s1):
            a.decode(outs[0])
        with torch.cuda.stream(s2):
            b.decode(outs[1])
    torch.cuda.synchronize()
    assert torch.equal(outs[0], want_a) and torch.equal(outs[1], want_b)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a.decode(outs[0])
    # one call captured, replayed after the lengths moved
    a.pos.copy_(torch.tensor([500, -1, 998], dtype=torch.int32))
    a.pos_h = [500, -1, 998]
    graph.replay()
    torch.cuda.synchronize()
    a.check(outs[0])


def test_offsets_past_32_bits(h):
    """Pages whose offset in the array passes 2^31 elements."""
    Hkv, page, dh = 8, 256, 128
    n_pages = 2 ** 31 // (Hkv * page * dh) + 9
    pool = torch.zeros(n_pages, Hkv, page, dh, dtype=torch.bfloat16, device="cuda")
    table = torch.arange(n_pages - 4, n_pages, dtype=torch.int32, device="cuda").flip(0).view(1, 4).contiguous()
    p = h.make_params(B=1, H=16, Hkv=Hkv, dh=dh, C=2 * dh, m=1, width=1, window=NO_WINDOW, scale=dh ** -0.5, page=page,
                      n_pages=n_pages, max_pages=4)
    pages = h.make_pages(pool, pool, table)          # keys and values in one array
    g = gen(31)
    n = 1000
    x = randn(g, n, Hkv * dh)
    h.swa_page_append(p, pages, torch.arange(n, dtype=torch.int32, device="cuda"), x, x,
                      torch.zeros(n, dtype=torch.int32, device="cuda"))
    q = randn(g, 1, 16 * dh)
    out = torch.empty_like(q)
    ws = torch.empty(h.hcsa_workspace_bytes(p, h.OP_SWA_DECODE_ATTEND), dtype=torch.uint8, device="cuda")
    h.swa_decode_attend(p, pages, torch.tensor([n - 1], dtype=torch.int32, device="cuda"), q, out, ws)
    kv = x.view(n, Hkv, dh)
    check(out, q.view(1, 16, dh), kv, kv, torch.ones(1, n, dtype=torch.bool, device="cuda"), p.scale, "bf16")
    del pool, pages


# ---------------------------------------------------------------- together

@pytest.mark.parametrize("lowprec", [False, True])
def test_prefill_then_decode_through_the_layers(h, lowprec):
    """A chained stack of two sliding-window layers (norm, projection, attention, output projection): a prompt through
    the prefill layers, its keys and values into pages, then tokens one by one; the decode's attention equals the
    plain one over what the pages hold, and without FP8 the whole run equals a prefill of the longer sequence."""
    D, H, Hkv, dh, window, sinks, T, steps, page, L = 256, 8, 2, 64, 48, 3, 150, 6, 16, 2
    g = gen(41)
    W = [(randn(g, D, (H + 2 * Hkv) * dh) * D ** -0.5).contiguous() for _ in range(L)]
    Wo = [(randn(g, H * dh, D) * (H * dh) ** -0.5).contiguous() for _ in range(L)]
    nw = [(1 + 0.1 * randn(g, D)).contiguous() for _ in range(L)]
    tokens = randn(g, T + steps, D)
    spec = h.SlidingSpec(D=D, H=H, Hkv=Hkv, dh=dh, window=window, sinks=sinks, scale=dh ** -0.5, T=T)

    def prefill(n):
        import dataclasses
        layers = [h.SlidingPrefillLayer(dataclasses.replace(spec, T=n)) for _ in range(L)]
        x = tokens[:n].clone()
        for i, l in enumerate(layers):
            l.norm(x, nw[i])
            l.forward(l.h, W[i])
            l.out_project(x, Wo[i])
        return layers, x

    layers, _ = prefill(T)
    _, full = prefill(T + steps)
    n_pages = -(-(T + steps) // page)
    order = torch.randperm(n_pages + 2, generator=g, device="cuda").to(torch.int32)
    table = torch.full((2, n_pages), -1, dtype=torch.int32, device="cuda")
    table[1] = order[:n_pages]                       # slot 0 stays empty
    dec = [h.SlidingDecodeLayer(spec, 2, page, n_pages + 2, table, lowprec=lowprec) for _ in range(L)]
    for a, b in zip(layers, dec):
        a.to_pages(b.p, b.pages, 1)
    for t in range(T, T + steps):
        x = torch.zeros(2, D, dtype=torch.bfloat16, device="cuda")
        x[1] = tokens[t]
        pos = torch.tensor([-1, t], dtype=torch.int32, device="cuda")
        for i, l in enumerate(dec):
            l.norm(x, nw[i])
            l.step(l.h, W[i], pos)
            k, v = (rows_of(pool, n_pages + 2, Hkv, page, dh, lowprec) for pool in l.pages.tensors[:2])
            j = torch.arange(t + 1, device="cuda")
            ids = table[1, j // page].long()
            q = spec.views(l.y)[2][1].reshape(1, H, dh)
            check(l.out[1:], q, k[ids, :, j % page], v[ids, :, j % page],
                  seen_mask(torch.tensor([t], device="cuda"), t + 1, window, sinks), spec.scale, "bf16")
            assert (l.out[0] == 0).all()
            l.out_project(x, Wo[i])
        if not lowprec:
            # two ways through the same layers: the stored roundings differ in places, each at most a step of
            # bf16 (2^-7) of values near 1, averaged by the projections
            assert ((x[1].float() - full[t].float()).abs().max() <= 2.0 ** -4)
    torch.cuda.synchronize()


@pytest.mark.parametrize("dh", [64, 128])
@pytest.mark.parametrize("what", ["spread", "rising", "falling", "wide query", "huge", "tiny"])
def test_decode_fp8_exponents(h, dh, what):
    """FP8 pages whose blocks' exponents differ by far more than fp16 spans, rise or fall along the sequence, or lie at the
    ends of the range; a query whose channels span more than fp16 does."""
    n, H, Hkv = 700, 16, 2
    c = Paged(h, [n - 1, 130], H, Hkv, dh, NO_WINDOW, 0, 32, "bf16", True, seed=17)
    g = gen(18)
    k, v = randn(g, n, Hkv * dh), randn(g, n, Hkv * dh)
    step = torch.arange(n, device="cuda")[:, None]
    if what == "spread":         # value blocks 2^-40 .. 2^30 next to each other, keys 2^-20 .. 1
        v = v * torch.exp2(((step * 7 + torch.arange(Hkv * dh, device="cuda") // 32 * 13) % 71 - 40).float()).to(v.dtype)
        k = k * torch.exp2(-((step * 5) % 21).float()).to(k.dtype)
    elif what == "rising":
        v = v * torch.exp2((step // 10 - 30).float()).to(v.dtype)
        k = k * torch.exp2((step // 100 - 6).float()).to(k.dtype)
    elif what == "falling":
        v = v * torch.exp2((30 - step // 10).float()).to(v.dtype)
        k = k * torch.exp2((-(step // 50)).float()).to(k.dtype)
    elif what == "wide query":
        c.q = c.q * torch.exp2((torch.arange(H * dh, device="cuda") % 50 - 49).float()).to(c.q.dtype)
    elif what == "huge":
        v = v * 2.0 ** 100
        k, c.q = k * 2.0 ** 90, c.q * 2.0 ** -90
    else:
        v = v * 2.0 ** -100
        k, c.q = k * 2.0 ** -90, c.q * 2.0 ** 90
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    for b, x in enumerate(c.pos_h):
        h.swa_page_append(c.p, c.pages, at[:x + 1], k[:x + 1], v[:x + 1], torch.full_like(at[:x + 1], b))
    c.check(c.decode())


def test_norm_fp8_in_place(h):
    """x_out = x with an 8-bit output: the same codes and stream as with a buffer of its own; enough rows that some
    have a block maximum next to a power-of-two border."""
    rows, D = 3000, 2048
    g = gen(51)
    x, d, w = randn(g, rows, D), randn(g, rows, D), randn(g, D)
    p = h.make_params(D=D)
    y8 = [torch.empty(rows * (D + D // 32), dtype=torch.uint8, device="cuda") for _ in range(2)]
    xo = torch.empty_like(x)
    h.hcsa_add_rmsnorm(p, x, d, w, 1e-6, xo, None, y8[0])
    h.hcsa_add_rmsnorm(p, x, d, w, 1e-6, x, None, y8[1])
    assert torch.equal(x, xo) and torch.equal(y8[0], y8[1])


@pytest.mark.parametrize("dtype,dh,window", [("bf16", 128, NO_WINDOW), ("bf16", 64, 200), ("f32", 64, 300), ("bf16", 72, 90)])
def test_attend_a_bad_channel_leaves_the_others(h, dtype, dh, window):
    """One channel infinite in every value: that channel is not finite, the others are as without it, and it takes no
    key-by-key pass over the rows."""
    T, H, Hkv = 2500, 4, 2
    g = gen(61)
    q, k, v = (randn(g, T, n * dh, dtype=dt(dtype)) for n in (H, Hkv, Hkv))
    v2 = v.clone()
    v2.view(T, Hkv, dh)[:, :, 5] = math.inf
    p = attend_params(h, T, H, Hkv, dh, window, 3, dtype)
    out = torch.empty_like(q)
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    h.swa_attend(p, q, k, v2, out)
    end.record()
    torch.cuda.synchronize()
    assert start.elapsed_time(end) < 500
    got = out.view(T, H, dh)
    assert not torch.isfinite(got[:, :, 5].float()).any()
    mask = seen_mask(torch.arange(T, device="cuda"), T, window, 3)
    got[:, :, 5] = 0
    v.view(T, Hkv, dh)[:, :, 5] = 0
    check(out, q.view(T, H, dh), k.view(T, Hkv, dh), v.view(T, Hkv, dh), mask, p.scale, dtype)


@pytest.mark.parametrize("kind,dh", [("bf16", 128), ("fp8", 64), ("f32", 64)])
def test_decode_pages_behind_the_window_may_be_given_back(h, kind, dh):
    c = Paged(h, [900, 333], 8, 2, dh, 100, 5, 32, "f32" if kind == "f32" else "bf16", kind == "fp8", seed=71)
    want = c.decode()
    for b, x in enumerate(c.pos_h):
        for i in range(c.table.shape[1]):
            if 32 * i >= 5 and 32 * i + 31 <= x - 100:       # no token of the page is seen
                c.table[b, i] = -1
    assert torch.equal(c.decode(), want)                     # (the status word is checked at the end)


def test_calls_on_another_stream_than_the_inputs_and_given_streams(h):
    """stream=: the call runs there; inputs made on one stream, used on another after a wait."""
    side = torch.cuda.Stream()
    g = gen(81)
    x, d, w = randn(g, 500, 512), randn(g, 500, 512), randn(g, 512)
    xo, y = torch.empty_like(x), torch.empty_like(x)
    p = h.make_params(D=512)
    side.wait_stream(torch.cuda.current_stream())
    h.hcsa_add_rmsnorm(p, x, d, w, 1e-6, xo, y, stream=side)
    side.synchronize()
    xo2, y2 = torch.empty_like(x), torch.empty_like(x)
    h.hcsa_add_rmsnorm(p, x, d, w, 1e-6, xo2, y2)
    assert torch.equal(xo, xo2) and torch.equal(y, y2)


def test_cpu_tensors_are_refused(h):
    x, w = torch.zeros(3, 64, dtype=torch.bfloat16), torch.ones(64, dtype=torch.bfloat16)
    p = h.make_params(D=64)
    for args in ((x, None, w, 1e-6, None, x.clone()), (x.cuda(), None, w, 1e-6, None, x.cuda())):
        with pytest.raises(h.HcsaError) as e:
            h.hcsa_add_rmsnorm(p, *args)
        assert e.value.code == 2


@pytest.mark.parametrize("dtype,H,Hkv,dh", [("bf16", 64, 8, 128), ("f32", 64, 2, 64)])
def test_attend_offsets_past_32_bits(h, dtype, H, Hkv, dh):
    """Queries and outputs of more than 2^31 elements: the last rows, and some in the middle."""
    T, window, sinks = 2 ** 31 // (H * dh) + 3000, 60, 3
    g = gen(91)
    q = torch.empty(T, H * dh, dtype=dt(dtype), device="cuda").normal_(generator=g)
    k, v = (torch.empty(T, Hkv * dh, dtype=dt(dtype), device="cuda").normal_(generator=g) for _ in range(2))
    out = torch.empty_like(q)
    h.swa_attend(attend_params(h, T, H, Hkv, dh, window, sinks, dtype), q, k, v, out)
    for a in (0, T // 2, T - 40):
        lo = max(0, a - window)
        rows = torch.arange(a, a + 40, device="cuda")
        cols = torch.cat([torch.arange(min(sinks, lo), device="cuda"), torch.arange(lo, a + 40, device="cuda")])
        t, j = rows[:, None], cols[None]
        mask = (j <= t) & ((j > t - window) | (j < sinks))
        check(out[a:a + 40], q[a:a + 40].view(40, H, dh), k[cols].view(-1, Hkv, dh), v[cols].view(-1, Hkv, dh), mask,
              dh ** -0.5, dtype)
    del q, k, v, out
    torch.cuda.empty_cache()


def test_empty_batches(h):
    """Tensors of no rows: nothing happens, no error."""
    x = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, dtype=torch.bfloat16, device="cuda")
    h.hcsa_add_rmsnorm(h.make_params(D=256), x, x.clone(), w, 1e-6, x.clone(), x.clone())
    p = attend_params(h, 0, 4, 1, 64, 10, 0, "bf16")
    kv = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    h.swa_attend(p, x, kv, kv, x.clone())
    c = Paged(h, [5], 4, 1, 64, 10, 0, 16, "bf16")
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    h.swa_page_append(c.p, c.pages, none, kv, kv, none)
    c.check(c.decode())


def class_of(x):
    """0 finite, 1 / -1 infinite, 2 NaN."""
    return torch.where(torch.isnan(x), 2.0, torch.where(torch.isinf(x), x.sign().double(), 0.0))


@pytest.mark.parametrize("size", [1.0, 2.0 ** -14])
@pytest.mark.parametrize("dh", [64, 96, 128])
@pytest.mark.parametrize("pos,window,page", [([700, 130], NO_WINDOW, 32), ([700, 130], 200, 16), ([9000], NO_WINDOW, 32)])
def test_decode_fp8_infinite_values(h, pos, window, page, dh, size):
    """Infinite and NaN values in FP8 pages: their channels are infinite or NaN whatever the weights (all below a half),
    the others are as without them; the same on the tensor cores (dh 64, 128) and the CUDA cores (96)."""
    H, Hkv = 16, 2
    c = Paged(h, pos, H, Hkv, dh, window, 2, page, "bf16", True, seed=23)
    last = [x - 9 for x in pos]
    for b, x in enumerate(last):
        n = 3
        at = torch.arange(x, x + n, dtype=torch.int32, device="cuda")
        g = gen(24 + b)
        k, v = randn(g, n, Hkv, dh) * 0.25, randn(g, n, Hkv, dh) * size
        v[0, :, 3], v[1, :, 40], v[0, :, 41] = math.inf, -math.inf, math.inf
        v[0, :, 50], v[2, :, 50] = math.inf, -math.inf          # both signs: NaN
        v[0, 0, 60], v[0, 0, 61] = math.nan, math.inf
        v[2, 1, 7] = math.nan                                    # in a block without infinities
        h.swa_page_append(c.p, c.pages, at, k.view(n, -1), v.view(n, -1), torch.full_like(at, b))
    if size < 1:                                                 # every other value as small
        for b, x in enumerate(pos):
            at = torch.tensor([t for t in range(x + 1) if not last[b] <= t < last[b] + 3], dtype=torch.int32, device="cuda")
            h.swa_page_append(c.p, c.pages, at, c.k[b, at.long()].reshape(len(at), -1),
                              (c.v[b, at.long()] * size).reshape(len(at), -1), torch.full_like(at, b))
    out = c.decode().view(len(pos), H, dh)
    k, v = (rows_of(x, c.n_pages, Hkv, page, dh, True) for x in c.pools)
    v = v.float().double()                                       # 448 x 2^120 is infinite in 32 bits
    for b, x in enumerate(pos):
        j = torch.arange(x + 1, device="cuda")
        ids = c.table[b, j // page].long()
        kk, vv = (t[ids, :, j % page] for t in (k, v))
        mask = seen_mask(torch.tensor([x], device="cuda"), x + 1, window, 2)
        seen = vv[mask[0]].repeat_interleave(H // Hkv, 1)        # [n, H, dh]
        up, down, nan = (seen == math.inf).any(0), (seen == -math.inf).any(0), torch.isnan(seen).any(0)
        want = torch.where(nan | (up & down), 2.0, up.double() - down.double())
        assert torch.equal(class_of(out[b]), want)
        assert want[0, 3] == 1 and want[0, 40] == -1 and want[0, 41] == 1 and want[0, 50] == 2 and want[0, 60] == 2
        fine = torch.where(want == 0, out[b].double(), 0.0)
        vv = torch.where((want == 0).view(Hkv, H // Hkv, dh)[:, 0], vv.nan_to_num(0, 0, 0), 0.0)
        check(fine.view(1, -1), c.q[b:b + 1].view(1, H, dh), kk, vv, mask, c.p.scale, "bf16", f"sequence {b}")


@pytest.mark.parametrize("D", [160, 512, 2048, 8192])
def test_norm_fp8_exponents_beside_a_border(h, D):
    """Blocks of zeros, of NaN, infinite ones and ones past the exponent range have the exponent of their own values,
    whether or not another block of the row, or a row next to it, lies at a power-of-two border."""
    x = torch.ones(6, D, dtype=torch.bfloat16, device="cuda")
    x[1, 3], x[2, 5] = math.nan, math.inf          # all of the row NaN; one channel NaN, the others zero
    x[3] = 0
    x[4, D // 2:] = 0
    w = torch.ones(D, dtype=torch.bfloat16, device="cuda")
    w[32:64] = 0
    w[64:96] = math.inf
    w[96:128] = torch.finfo(torch.bfloat16).max    # y up to 1.5 times it: past fp32 in row 4
    w[128:160] = 2.0 ** -133
    p = h.make_params(D=D)
    for border in (1.0, 1.75):                     # 1.75: y just below 448 / 2^8 in each row of ones
        w[:32] = border
        y8 = torch.zeros(6 * (D + D // 32), dtype=torch.uint8, device="cuda")
        h.hcsa_add_rmsnorm(p, x, None, w, 1e-12, None, None, y8)
        got = y8[6 * D:].view(torch.int8).view(6, D // 32).double()
        s = x.double()
        y = (s / (s.square().mean(-1, keepdim=True) + 1e-12).sqrt() * w.double()).view(6, D // 32, 32).abs()
        amax = y.nan_to_num(0, math.inf, -math.inf).amax(-1)
        e = torch.ceil(torch.log2(amax / 448))
        e = torch.where(amax > 448 * torch.exp2(e), e + 1, torch.where(amax <= 224 * torch.exp2(e), e - 1, e))
        e = torch.where(torch.isnan(y).all(-1) | torch.isinf(amax), 120.0, torch.where(amax == 0, 0.0, e.clamp(-126, 120)))
        assert torch.equal(got, e), (border, (got != e).nonzero().tolist())


@pytest.mark.parametrize("dh,Hkv", [(128, 1), (64, 2)])
def test_attend_a_late_bad_value_of_a_long_sequence(h, dh, Hkv):
    """One NaN near the end of a long causal sequence: the rows in front of it that share its block, each with more than
    131000 keys, are as without it, and so is every block that its CTA takes later."""
    T, H, bad = 131072, 2 * Hkv, 131069
    g = gen(101)
    q, k, v = (randn(g, T, n * dh) for n in (H, Hkv, Hkv))
    v[bad, dh // 2] = math.nan                       # head 0
    out = torch.full_like(q, math.nan)
    h.swa_attend(attend_params(h, T, H, Hkv, dh, NO_WINDOW, 0, "bf16"), q, k, v, out)
    torch.cuda.synchronize()
    assert h.hcsa_get_device_status() == 0
    got = out.view(T, Hkv, 2, dh)
    assert torch.isnan(got[bad:, 0, :, dh // 2]).all()
    got[bad:, 0, :, dh // 2] = 0
    v[bad, dh // 2] = 0
    assert torch.isfinite(out.float()).all()
    for rows in (torch.arange(T - 140, bad, 7, device="cuda"), torch.arange(70000, 70016, device="cuda")):
        mask = seen_mask(rows, T, NO_WINDOW, 0)
        check(out[rows], q[rows].view(-1, H, dh), k.view(T, Hkv, dh), v.view(T, Hkv, dh), mask, dh ** -0.5, "bf16")


@pytest.mark.parametrize("dtype,H,Hkv,dh,window,sinks", [
    ("bf16", 4, 2, 128, NO_WINDOW, 0), ("bf16", 8, 1, 64, 60, 5), ("bf16", 3, 1, 128, 128, 20), ("bf16", 1, 1, 64, 300, 0),
    ("bf16", 128, 1, 64, 90, 3), ("f32", 4, 2, 64, NO_WINDOW, 0), ("f32", 2, 1, 128, 50, 7), ("f32", 3, 1, 200, 100, 2),
    ("f32", 1, 1, 512, 40, 0), ("bf16", 5, 1, 72, 64, 3), ("bf16", 2, 1, 256, 33, 1)])
def test_attend_infinite_values_by_what_a_row_sees(h, dtype, H, Hkv, dh, window, sinks):
    """Each output is infinite with the sign, NaN or finite as the values that its row sees make it, whatever lies next to
    them: infinities and NaN of the same channels at neighbouring tokens, of which a row sees some."""
    T = 450
    g = gen(111)
    q, k, v = (randn(g, T, n * dh, dtype=dt(dtype)) for n in (H, Hkv, Hkv))
    vv = v.view(T, Hkv, dh)
    vv[100, :, 3], vv[103, :, 3] = math.inf, math.nan            # rows 100 .. 102: infinite
    vv[200, :, 9], vv[207, :, 9] = -math.inf, math.inf           # rows 200 .. 206: infinite, then NaN, later infinite
    vv[290, :, 17] = math.inf
    vv[300:310, 0, 20:40] = math.nan
    vv[8, :, 50], vv[12, :, 51], vv[2, :, 60], vv[6, :, 60] = math.inf, math.nan, math.inf, -math.inf
    vv[T - 2, Hkv - 1, dh - 1] = -math.inf
    k.view(T, Hkv, dh)[350, 0, 4] = math.nan                     # weights of the rows that see it
    out = torch.empty_like(q)
    p = attend_params(h, T, H, Hkv, dh, window, sinks, dtype)
    h.swa_attend(p, q, k, v, out)
    got = out.view(T, H, dh)
    mask = seen_mask(torch.arange(T, device="cuda"), T, window, sinks)
    see = mask.double()

    def any_seen(x):                                             # [T, Hkv, dh] truth -> [T, H, dh]
        return (torch.einsum("tj,jgd->tgd", see, x.double()) > 0).repeat_interleave(H // Hkv, 1)

    up, down, nan = any_seen(vv == math.inf), any_seen(vv == -math.inf), any_seen(torch.isnan(vv))
    lost = (mask[:, 350, None, None] & (torch.arange(H, device="cuda") < H // Hkv)[:, None]).expand(T, H, dh)
    want = torch.where(nan | (up & down) | lost, 2.0, up.double() - down.double())
    wrong = class_of(got) != want
    assert not wrong.any(), (int(wrong.sum()), wrong.nonzero()[:5].tolist())
    assert want[101, 0, 3] == 1 and want[204, 0, 9] == -1 and (want[1] == 0).all()
    clean_k, clean_v = k.nan_to_num(0).view(T, Hkv, dh), torch.where(torch.isfinite(vv), vv, 0.0)
    plain, _, _ = attend64(q.view(T, H, dh), clean_k, clean_v, mask, p.scale)
    check(torch.where(want == 0, got.double(), plain), q.view(T, H, dh), clean_k, clean_v, mask, p.scale, dtype)


def test_a_single_row_of_any_stride(h):
    """One token's row out of a tensor whose rows are not multiples of 16 bytes apart: its stride is never used."""
    g = gen(121)

    def row(n):
        return randn(g, 3, n + 5)[:1, :n]

    x, y, w = row(256), row(256), randn(g, 256)
    h.hcsa_add_rmsnorm(h.make_params(D=256), x, None, w, 1e-6, None, y)
    want = x.double() / (x.double().square().mean(-1, keepdim=True) + 1e-6).sqrt() * w.double()
    assert ((y.double() - want).abs() <= (2.0 ** -8 + 2.0 ** -17) * want.abs()).all()
    q, k, v, out = row(8 * 64), row(2 * 64), row(2 * 64), row(8 * 64)
    h.swa_attend(attend_params(h, 1, 8, 2, 64, 5, 1, "bf16"), q, k, v, out)
    assert torch.equal(out.view(2, 4, 64), v.view(2, 1, 64).expand(2, 4, 64))
    c = Paged(h, [40], 8, 2, 64, NO_WINDOW, 0, 16, "bf16", seed=5)
    h.swa_page_append(c.p, c.pages, c.pos, k, v)
    c.q = row(8 * 64)
    c.check(c.decode(out))


@pytest.mark.parametrize("dtype,rows,D", [("bf16", 3000, 416), ("f32", 70, 2048)])
def test_norm_over_its_inputs(h, dtype, rows, D):
    """y over x or over delta, x_out over the other one."""
    g = gen(131)
    x, d, w = (randn(g, *s, dtype=dt(dtype)) for s in ((rows, D), (rows, D), (D,)))
    p = h.make_params(D=D, dtype=dtype)
    xo, y = torch.empty_like(x), torch.empty_like(x)
    h.hcsa_add_rmsnorm(p, x, d, w, 1e-6, xo, y)
    for swap in (False, True):
        a, b = x.clone(), d.clone()
        h.hcsa_add_rmsnorm(p, a, b, w, 1e-6, *((b, a) if swap else (a, b)))
        got = (b, a) if swap else (a, b)
        assert torch.equal(got[0], xo) and torch.equal(got[1], y)


@pytest.mark.parametrize("dh", [64, 96, 128])
def test_decode_fp8_nan_and_infinity_in_one_channel(h, dh):
    """A NaN in a block of ordinary values and an infinite value of the same channel in another token: NaN."""
    n = 60
    c = Paged(h, [n - 1], 4, 1, dh, NO_WINDOW, 0, 32, "bf16", True, seed=29)
    v = c.v[0].clone()
    v[50, 0, 5], v[20, 0, 5] = math.nan, -math.inf
    v[50, 0, 40], v[51, 0, 40] = math.inf, math.nan
    at = torch.arange(n, dtype=torch.int32, device="cuda")
    h.swa_page_append(c.p, c.pages, at, c.k[0].view(n, -1), v.view(n, -1), torch.zeros_like(at))
    got = c.decode().view(4, dh)
    assert torch.isnan(got[:, 5]).all() and torch.isnan(got[:, 40]).all()
    assert torch.isfinite(got[:, :5]).all() and torch.isfinite(got[:, 6:40]).all() and torch.isfinite(got[:, 41:]).all()


@pytest.mark.parametrize("dtype,H,Hkv,dh,window,sinks", [("bf16", 8, 2, 128, NO_WINDOW, 0), ("bf16", 4, 4, 64, 700, 300), ("bf16", 7, 1, 64, 20, 9),
                                                         ("bf16", 1, 1, 128, 3, 0), ("f32", 4, 2, 64, NO_WINDOW, 0), ("bf16", 2, 1, 72, 90, 3)])
def test_attend_a_channel_of_infinities(h, dtype, H, Hkv, dh, window, sinks):
    """A channel infinite in every value is infinite in every output, another one of both signs NaN from where a row sees both; the other
    channels are as without them."""
    T = 3001
    g = gen(141)
    q, k, v = (randn(g, T, n * dh, dtype=dt(dtype)) for n in (H, Hkv, Hkv))
    vv = v.view(T, Hkv, dh)
    clean = vv.clone()
    vv[:, :, 5], vv[:, :, 30], vv[1500, :, 30] = math.inf, -math.inf, math.inf
    vv[2000, 0, 11] = math.nan
    out = torch.empty_like(q)
    h.swa_attend(attend_params(h, T, H, Hkv, dh, window, sinks, dtype), q, k, v, out)
    got = out.view(T, H, dh)
    mask = seen_mask(torch.arange(T, device="cuda"), T, window, sinks)
    assert (got[:, :, 5] == math.inf).all()
    both = mask[:, 1500] & (mask.sum(1) > 1)
    assert torch.isnan(got[both][:, :, 30]).all() and (got[~mask[:, 1500]][:, :, 30] == -math.inf).all()
    head = torch.arange(H, device="cuda") < H // Hkv
    assert torch.equal(torch.isnan(got[:, :, 11]), mask[:, 2000, None] & head)
    clean[:, :, [5, 30]] = 0
    got[:, :, [5, 30]] = 0
    clean[2000, 0, 11] = 0
    plain, _, _ = attend64(q.view(T, H, dh), k.view(T, Hkv, dh), clean, mask, dh ** -0.5)
    check(torch.where(torch.isnan(got), plain, got.double()), q.view(T, H, dh), k.view(T, Hkv, dh), clean, mask, dh ** -0.5, dtype)
