"""What is measured of the sliding-window layer's operators: inputs, plain forms, calls and 64-bit values.

Four operators that stand beside the compressed attention of this package and make, together, the
uncompressed layers of a hybrid stack:

  norm    x' = x + delta, y = x' / sqrt(mean(x'^2) + eps) * w: the residual addition and the
          root-mean-square norm between two layers; y in the storage type, or in 8 bits (E4M3 codes with
          one power-of-two scale per 32 channels)
  swa     causal attention of a whole sequence over its last `window` tokens and its first `sinks` tokens,
          query heads in groups that share a key / value head
  append  new tokens' keys and values into a paged cache (storage type or 8 bits)
  decode  attention of one new token per sequence over that paged cache, window and sinks as above

`own` false: plain torch in 32 bits (64 where a value next to a rounding border matters); `own` true: the
package's calls.
"""
import math

import torch

own = False

NO_WINDOW = 2 ** 31 - 1      # the window of a layer that sees every earlier token


def listed():
    return [
        # the norm between two layers of a decode stack: 4 sequences, one token each; latency alone counts
        dict(name="norm_decode_b4", op="norm", rows=4, D=2048, dtype="bf16", fp8=False),
        # the same norm over a whole 131072-token prefill, 8-bit output for the next product: bandwidth
        dict(name="norm_prefill_fp8", op="norm", rows=131072, D=2048, dtype="bf16", fp8=True),
        # 32-bit storage, a ragged number of rows
        dict(name="norm_f32_ragged", op="norm", rows=5003, D=512, dtype="f32", fp8=False),
        # a short prompt of odd length through a window layer with 64-wide heads: latency
        dict(name="swa_prompt_517", op="swa", T=517, H=8, Hkv=2, dh=64, window=128, sinks=4, dtype="bf16"),
        # a long document through a 128-token window layer: little work per token, 64 heads
        dict(name="swa_window_64k", op="swa", T=65536, H=64, Hkv=8, dh=128, window=128, sinks=4, dtype="bf16"),
        # full causal attention of an 8k prompt (no window): the matrix-product-bound end
        dict(name="swa_full_8k", op="swa", T=8192, H=32, Hkv=8, dh=128, window=NO_WINDOW, sinks=0, dtype="bf16"),
        # 32-bit storage at the small correctness layer's sizes, a key head per query head
        dict(name="swa_f32_2048", op="swa", T=2048, H=8, Hkv=8, dh=64, window=128, sinks=4, dtype="f32"),
        # a prompt's keys and values into pages, stored in 8 bits
        dict(name="append_prompt_fp8", op="append", rows=8191, B=1, Hkv=8, dh=128, page=64, P=8192, dtype="bf16",
             fp8=True),
        # one new token for each of 32 sequences: latency
        dict(name="append_token_b32", op="append", rows=32, B=32, Hkv=8, dh=128, page=16, P=1024, dtype="bf16",
             fp8=False),
        # one decode step of a window layer for a few sequences of odd lengths: latency
        dict(name="decode_window_b4", op="decode", B=4, P=4099, H=64, Hkv=8, dh=128, window=128, sinks=4, page=16,
             dtype="bf16", fp8=False),
        # one decode step over long uncompressed caches of very different lengths: cache bandwidth
        dict(name="decode_ragged_b32", op="decode", B=32, P=32768, H=64, Hkv=8, dh=128, window=NO_WINDOW, sinks=0,
             page=64, dtype="bf16", fp8=False),
        # one key head for 16 query heads over 8-bit caches of up to 262144 tokens
        dict(name="decode_long_fp8", op="decode", B=8, P=262144, H=16, Hkv=1, dh=128, window=NO_WINDOW, sinks=0,
             page=128, dtype="bf16", fp8=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "swa", "swa", "append", "decode", "decode"])
    dtype = "f32" if rng.random() < 0.2 else "bf16"
    dh = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 3, 4, 8])
    H = Hkv * rng.choice([1, 2, 3, 4, 5, 7, 8, 16])
    window = rng.choice([NO_WINDOW, _log(rng, 16, 4096)])
    sinks = rng.choice([0, 1, 4, _log(rng, 1, 200)])
    if op == "norm":
        D = 32 * _log(rng, 2, 256)
        return dict(op=op, rows=_log(rng, 1, max(1, 2 ** 27 // D)), D=D, dtype=dtype,
                    fp8=dtype == "bf16" and rng.random() < 0.5)
    if op == "swa":
        T = _log(rng, 1, 65536 if dtype == "bf16" else 4096)
        while H * T * min(T, window) > 2 ** 30 or H * T > 2 ** 22:   # no more than the listed cases' scores
            T = (T + 1) // 2
        return dict(op=op, T=T, H=H, Hkv=Hkv, dh=dh, window=window, sinks=sinks, dtype=dtype)
    page = rng.choice([16, 32, 48, 64, 128, 256])
    fp8 = dtype == "bf16" and rng.random() < 0.4
    if op == "append":
        B = _log(rng, 1, 64)
        P = _log(rng, 1, 32768 // B)
        rows = rng.choice([B, B * P])            # one token of each sequence, or whole prompts
        return dict(op=op, rows=rows, B=B, Hkv=Hkv, dh=dh, page=page, P=P, dtype=dtype, fp8=fp8)
    B = _log(rng, 1, 128)
    P = _log(rng, 1, 2 ** 22 // (B * Hkv))
    return dict(op=op, B=B, P=P, H=H, Hkv=Hkv, dh=dh, window=window, sinks=sinks, page=page, dtype=dtype, fp8=fp8)


# ---------------------------------------------------------------- inputs

def _torch(dtype):
    return torch.bfloat16 if dtype == "bf16" else torch.float32


def _positions(c):
    """The new token's position in each sequence: spread over [P / 8, P), the first one the longest; every
    seventh slot of a larger batch is empty (-1), as in a batch that sequences leave and join."""
    P, B = c["P"], c["B"]
    pos = [P - 1] + [min(P - 1, int(P * (0.125 + 0.875 * ((b * 0.6180339887) % 1.0)))) for b in range(1, B)]
    return [-1 if B >= 8 and b % 7 == 6 else x for b, x in enumerate(pos)]


def _tokens(c):
    """(sequence, position) of each appended row."""
    if c["rows"] == c["B"]:
        return list(range(c["B"])), _positions(c)
    per = c["rows"] // c["B"]
    return [r // per for r in range(per * c["B"])], [r % per for r in range(per * c["B"])]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = _torch(c["dtype"])

    def normal(*shape, std=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device="cuda") * std).to(dtype)

    if c["op"] == "norm":
        rows, D = c["rows"], c["D"]
        s = dict(x=normal(rows, D), delta=normal(rows, D, std=0.5),
                 w=(1 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dt), eps=1e-6)
        s["x_out"] = torch.empty_like(s["x"])
        s["y"] = None if c["fp8"] else torch.empty_like(s["x"])
        s["y8"] = torch.zeros(rows * (D + D // 32), dtype=torch.uint8, device="cuda") if c["fp8"] else None
    elif c["op"] == "swa":
        T, H, Hkv, dh = c["T"], c["H"], c["Hkv"], c["dh"]
        y = normal(T, (2 * Hkv + H) * dh)        # the projection's columns [k | v | q], read in place
        a, b = Hkv * dh, 2 * Hkv * dh
        s = dict(k=y[:, :a], v=y[:, a:b], q=y[:, b:], scale=1.0 / math.sqrt(dh),
                 out=torch.empty(T, H * dh, dtype=dt, device="cuda"))
    else:
        B, Hkv, dh, page, P = c["B"], c["Hkv"], c["dh"], c["page"], c["P"]
        most = -(-P // page)
        need = [-(-(x + 1) // page) for x in _positions(c)] if c["op"] == "decode" else [most] * B
        n_pages = sum(need) + 3
        order = torch.randperm(n_pages, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, most), -1, dtype=torch.int32)
        at = 0
        order_h = order.cpu()
        for b, n in enumerate(need):
            table[b, :n] = order_h[at:at + n]
            at += n
        rows = n_pages * Hkv * page
        s = dict(table=table.cuda(), n_pages=n_pages)
        for name in ("k_pages", "v_pages"):
            if c["fp8"]:
                buf = torch.empty(rows * (dh + dh // 32), dtype=torch.uint8, device="cuda")
                if c["op"] == "append":
                    buf.zero_()
                else:
                    for r in range(0, rows, 1 << 20):     # in pieces: the scratch stays small
                        e = min(rows, r + (1 << 20))
                        x = torch.randn(e - r, dh, generator=g, device="cuda").to(torch.bfloat16)
                        codes, exps = _quantize(x)
                        buf[r * dh:e * dh] = codes.view(torch.uint8).reshape(-1)
                        buf[rows * dh + r * dh // 32:rows * dh + e * dh // 32] = exps.view(torch.uint8).reshape(-1)
                s[name] = buf
            elif c["op"] == "append":
                s[name] = torch.zeros(n_pages, Hkv, page, dh, dtype=dt, device="cuda")
            else:
                x = torch.empty(n_pages, Hkv, page, dh, dtype=dt, device="cuda")
                s[name] = x.normal_(generator=g)
        if c["op"] == "append":
            seq, pos = _tokens(c)
            y = normal(len(seq), 2 * Hkv * dh)
            s.update(seq=torch.tensor(seq, dtype=torch.int32, device="cuda"),
                     pos=torch.tensor(pos, dtype=torch.int32, device="cuda"),
                     k=y[:, :Hkv * dh], v=y[:, Hkv * dh:])
        else:
            H = c["H"]
            s.update(pos=torch.tensor(_positions(c), dtype=torch.int32, device="cuda"), q=normal(B, H * dh),
                     scale=1.0 / math.sqrt(dh), out=torch.empty(B, H * dh, dtype=dt, device="cuda"))
    s["case"] = c
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a user's program sets up once: the call parameters, the page handle and the workspace."""
    import long_context_compressed_05_b200 as h
    c = s["case"]
    if c["op"] == "norm":
        s["p"] = h.make_params(D=c["D"], dtype=c["dtype"])
        return
    # C = 2 dh: the key and the value of one head, as in the package's other layers
    p = dict(Hkv=c["Hkv"], dh=c["dh"], C=2 * c["dh"], m=1, width=1, dtype=c["dtype"])
    if c["op"] != "append":
        p.update(H=c["H"], window=c["window"], sinks=c["sinks"], scale=s["scale"])
    else:
        p.update(H=c["Hkv"])
    if c["op"] == "swa":
        s["p"] = h.make_params(T=c["T"], **p)
        return
    s["p"] = h.make_params(B=c["B"], page=c["page"], n_pages=s["n_pages"], max_pages=s["table"].shape[1],
                           lowprec=c["fp8"], **p)
    s["pages"] = h.make_pages(s["k_pages"], s["v_pages"], s["table"])
    if c["op"] == "decode":
        n = h.hcsa_workspace_bytes(s["p"], h.OP_SWA_DECODE_ATTEND)
        s["ws"] = torch.empty(n, dtype=torch.uint8, device="cuda")


# ---------------------------------------------------------------- one pass

def run(state):
    s = state
    return {"norm": _norm, "swa": _swa, "append": _append, "decode": _decode}[s["case"]["op"]](s)


def _quantize(x):
    """Rows [n, ch] -> (E4M3 codes [n, ch], int8 exponents [n, ch / 32]): every 32 channels share 2^e, e the
    smallest integer with amax / 2^e <= 448."""
    b = x.unflatten(-1, (-1, 32))
    f, k = torch.frexp(b.abs().amax(-1))                      # amax = f 2^k, f in [0.5, 1); 448 = 0.875 2^9
    e = torch.where(f == 0, torch.zeros_like(k), torch.where(f <= 0.875, k - 9, k - 8))
    codes = torch.ldexp(b, -e.unsqueeze(-1).to(b.dtype)).flatten(-2).float().to(torch.float8_e4m3fn)
    return codes, e.to(torch.int8)


def _split8(buf, n, ch):
    """The codes as E4M3 numbers and the exponents of an 8-bit array of n rows."""
    return buf[:n * ch].view(torch.float8_e4m3fn).view(n, ch), buf[n * ch:].view(torch.int8).view(n, ch // 32)


def _norm(s):
    c = s["case"]
    if own:
        import long_context_compressed_05_b200 as h
        h.hcsa_add_rmsnorm(s["p"], s["x"], s["delta"], s["w"], s["eps"], s["x_out"], s["y"], s["y8"])
        if not c["fp8"]:
            return s["x_out"], s["y"]
        return s["x_out"], *_split8(s["y8"], c["rows"], c["D"])
    wide = torch.float64 if c["fp8"] else torch.float32       # block maxima next to a power-of-two border
    x = s["x"].to(wide) + s["delta"].to(wide)
    y = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * s["w"].to(wide)
    if not c["fp8"]:
        return x.to(s["x"].dtype), y.to(s["x"].dtype)
    return x.to(s["x"].dtype), *_quantize(y)


def _swa(s):
    c = s["case"]
    if own:
        import long_context_compressed_05_b200 as h
        h.swa_attend(s["p"], s["q"], s["k"], s["v"], s["out"])
        return s["out"]
    T, H, Hkv, dh, S = c["T"], c["H"], c["Hkv"], c["dh"], min(c["sinks"], c["T"])
    W, G = min(c["window"], T), H // Hkv
    n = min(T, max(W, 128))                                   # query blocks of n tokens see n + W - 1 keys
    nb = -(-T // n)
    pad = torch.nn.functional.pad
    q = pad(s["q"].float() * s["scale"], (0, 0, 0, nb * n - T)).view(nb, n, Hkv, G, dh).permute(0, 2, 3, 1, 4)
    q = q.reshape(nb, Hkv, G * n, dh)
    k, v = s["k"].float().view(T, Hkv, dh), s["v"].float().view(T, Hkv, dh)
    kb, vb = (pad(x, (0, 0, 0, 0, W - 1, nb * n - T)).unfold(0, n + W - 1, n) for x in (k, v))
    blk = torch.arange(nb, device=q.device).view(nb, 1, 1, 1, 1)
    i = torch.arange(n, device=q.device).view(n, 1)
    at = torch.arange(n + W - 1, device=q.device)             # key blk n - (W - 1) + at
    p = (q @ kb).view(nb, Hkv, G, n, n + W - 1)
    p.masked_fill_((at < i) | (at > i + W - 1) | (blk * n - (W - 1) + at < 0), -math.inf)
    top = p.amax(-1, keepdim=True)
    if S:
        ps = (q @ k[:S].permute(1, 2, 0)).view(nb, Hkv, G, n, S)
        ps.masked_fill_(torch.arange(S, device=q.device) > blk * n + i - W, -math.inf)
        top = torch.maximum(top, ps.amax(-1, keepdim=True))
    p.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(nb, Hkv, G * n, -1) @ vb.transpose(-1, -2)).view(nb, Hkv, G, n, dh)
    if S:
        ps.sub_(top).exp_()
        total = total + ps.sum(-1, keepdim=True)
        o = o + (ps.view(nb, Hkv, G * n, S) @ v[:S].transpose(0, 1)).view(nb, Hkv, G, n, dh)
    o = (o / total).permute(0, 3, 1, 2, 4).reshape(nb * n, H * dh)[:T]
    return o.to(s["out"].dtype)


def _append(s):
    c = s["case"]
    Hkv, dh, page = c["Hkv"], c["dh"], c["page"]
    rows = s["n_pages"] * Hkv * page
    if own:
        import long_context_compressed_05_b200 as h
        h.swa_page_append(s["p"], s["pages"], s["pos"], s["k"], s["v"], s["seq"])
    else:
        live = s["pos"] >= 0
        seq, pos = s["seq"][live].long(), s["pos"][live].long()
        slot = s["table"][seq, pos // page].long(), pos % page
        # row of head h: (page_id Hkv + h) page + offset
        at = (slot[0][:, None] * Hkv + torch.arange(Hkv, device=pos.device)) * page + slot[1][:, None]
        for pool, x in ((s["k_pages"], s["k"]), (s["v_pages"], s["v"])):
            x = x[live].reshape(-1, dh)
            if c["fp8"]:
                codes, exps = _quantize(x.float())
                pool[:rows * dh].view(rows, dh)[at.view(-1)] = codes.view(torch.uint8)
                pool[rows * dh:].view(rows, dh // 32)[at.view(-1)] = exps.view(torch.uint8)
            else:
                pool.view(rows, dh)[at.view(-1)] = x
    if c["fp8"]:
        return *_split8(s["k_pages"], rows, dh), *_split8(s["v_pages"], rows, dh)
    return s["k_pages"], s["v_pages"]


def _decode(s):
    c = s["case"]
    if own:
        import long_context_compressed_05_b200 as h
        h.swa_decode_attend(s["p"], s["pages"], s["pos"], s["q"], s["out"], s["ws"])
        return s["out"]
    B, H, Hkv, dh, page, P = c["B"], c["H"], c["Hkv"], c["dh"], c["page"], c["P"]
    S, W = min(c["sinks"], P), min(c["window"], P)
    pos = s["pos"].long().view(B, 1)
    dev = pos.device
    first = (pos - W + 1).clamp(min=0)
    near = first + torch.arange(W, device=dev)
    far = torch.arange(S, device=dev).expand(B, S)
    key = torch.cat([far, near], 1)                                        # [B, S + W] key positions
    seen = torch.cat([far < first, near <= pos], 1) & (pos >= 0)
    key = torch.where(seen, key, torch.zeros_like(key))
    ids = s["table"].gather(1, key // page).long().clamp(min=0)
    at = (ids[:, None] * Hkv + torch.arange(Hkv, device=dev)[:, None]) * page + (key % page)[:, None]
    rows = s["n_pages"] * Hkv * page

    def fetch(pool):                                                       # [B, Hkv, S + W, dh] in 32 bits
        if not c["fp8"]:
            return pool.view(rows, dh)[at].float()
        codes = pool[:rows * dh].view(rows, dh)[at].view(torch.float8_e4m3fn).float()
        exps = pool[rows * dh:].view(torch.int8).view(rows, dh // 32)[at].float()
        return (codes.unflatten(-1, (-1, 32)) * torch.exp2(exps).unsqueeze(-1)).flatten(-2)

    q = s["q"].float().view(B, Hkv, H // Hkv, dh) * s["scale"]
    p = q @ fetch(s["k_pages"]).transpose(-1, -2)
    seen = seen[:, None, None]
    p = p.masked_fill_(~seen, -math.inf)
    p = p.sub_(p.amax(-1, keepdim=True).clamp(min=-3e38)).exp_()
    o = p @ fetch(s["v_pages"])
    o = o / p.sum(-1, keepdim=True).clamp(min=1e-30)                        # an empty slot gives zeros
    return o.view(B, H * dh).to(s["out"].dtype)


# ---------------------------------------------------------------- what a pass cannot do without

def _pairs(pos, W, S):
    """Keys that the query at position pos sees."""
    near = min(pos + 1, W)
    return near + min(S, pos + 1 - near)


def work(case):
    c = case
    e = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "norm":
        n = c["rows"] * c["D"]
        return {"bytes": n * (3 * e + (1 + 1 / 32 if c["fp8"] else e)) + c["D"] * e, "flops": 5 * n}
    dh, Hkv = c["dh"], c["Hkv"]
    if c["op"] == "append":
        live = sum(x >= 0 for x in _tokens(c)[1])
        to = dh + dh // 32 if c["fp8"] else dh * e
        return {"bytes": live * 2 * Hkv * (dh * e + to), "flops": 0}
    H, W, S = c["H"], c["window"], c["sinks"]
    if c["op"] == "swa":
        T = c["T"]
        n = min(T, W)
        seen = n * (n + 1) // 2 + (T - n) * n + sum(min(S, t + 1 - n) for t in range(n, min(T, n + S)))
        seen += max(0, T - n - S) * S
        return {"bytes": T * 2 * (H + Hkv) * dh * e, "flops": 4 * seen * H * dh}
    seen = sum(_pairs(x, W, S) for x in _positions(c) if x >= 0)
    row = dh + dh // 32 if c["fp8"] else dh * e
    return {"bytes": seen * 2 * Hkv * row + 2 * c["B"] * H * dh * e, "flops": 4 * seen * H * dh}


# ---------------------------------------------------------------- the definitions in 64 bits

def _to_e4m3(y):
    """64-bit rows -> (codes as E4M3 numbers in 64 bits, exponents): nearest, ties to even, from the grid of
    E4M3 (steps of 2^(max(floor(log2 |v|), -6) - 3))."""
    n = y.shape[-1] // 32
    blocks = y.reshape(*y.shape[:-1], n, 32)
    most = blocks.abs().max(dim=-1).values
    e = torch.ceil(torch.log2(most / 448)).nan_to_num(neginf=0.0)
    e = e + (most > 448 * torch.exp2(e)).to(e.dtype)
    e = e - ((most > 0) & (most <= 448 * torch.exp2(e - 1))).to(e.dtype)
    v = blocks / torch.exp2(e)[..., None]
    fine = torch.exp2(torch.floor(torch.log2(v.abs().clamp(min=2.0 ** -6))) - 3)
    return (torch.round(v / fine) * fine).reshape(y.shape), e


def exact(case, seed):
    c = case
    s = prepare(c, seed)
    f8 = bool(c.get("fp8"))
    if c["op"] == "norm":
        total = s["x"].double() + s["delta"].double()
        rms = (total.pow(2).sum(-1) / c["D"] + s["eps"]).sqrt()
        y = total / rms[:, None] * s["w"].double()
        if not f8:
            return total, y
        codes, e = _to_e4m3(y)
        return total, codes, None
    Hkv, dh = c["Hkv"], c["dh"]
    if c["op"] == "append":
        pools = []
        for name in ("k", "v"):
            rows = [torch.zeros(s["n_pages"], Hkv, c["page"], dh, dtype=torch.float64, device="cuda")]
            x = s[name].double().reshape(-1, Hkv, dh)
            if f8:
                x, _ = _to_e4m3(x)
            keep = (s["pos"] >= 0).nonzero().view(-1)
            pos, seq = s["pos"][keep].long(), s["seq"][keep].long()
            page = s["table"][seq, torch.div(pos, c["page"], rounding_mode="floor")].long()
            rows[0][page, :, pos.remainder(c["page"])] = x[keep]
            pools.append(rows[0])
        if not f8:
            return tuple(pools)
        return pools[0].view(-1, dh), None, pools[1].view(-1, dh), None
    H, W, S = c["H"], c["window"], c["sinks"]
    G = H // Hkv
    if c["op"] == "swa":
        T = c["T"]
        q = s["q"].double().reshape(T, Hkv, G, dh)
        k, v = s["k"].double().reshape(T, Hkv, dh), s["v"].double().reshape(T, Hkv, dh)
        out = torch.empty(T, Hkv, G, dh, dtype=torch.float64, device="cuda")
        step = 256
        for a in range(0, T, step):
            b = min(T, a + step)
            lo = max(0, a - W + 1)
            cols = torch.cat([torch.arange(min(S, lo)), torch.arange(lo, b)]).cuda()
            t = torch.arange(a, b, device="cuda")[:, None]
            see = (cols <= t) & ((cols > t - W) | (cols < S))
            z = torch.einsum("thgd,jhd->hgtj", q[a:b], k[cols]) * s["scale"]
            w = torch.softmax(torch.where(see, z, torch.full_like(z, -math.inf)), dim=-1)
            out[a:b] = torch.einsum("hgtj,jhd->thgd", w, v[cols])
        return out.reshape(T, H * dh)
    out = torch.zeros(c["B"], H * dh, dtype=torch.float64, device="cuda")
    rows = s["n_pages"] * Hkv * c["page"]
    for b, pos in enumerate(_positions(c)):
        if pos < 0:
            continue
        j = torch.arange(pos + 1, device="cuda")
        j = j[(j > pos - W) | (j < S)]
        page = s["table"][b, torch.div(j, c["page"], rounding_mode="floor")].long()
        kv = []
        for name in ("k_pages", "v_pages"):
            if f8:
                line = (page[:, None] * Hkv + torch.arange(Hkv, device="cuda")) * c["page"] + \
                    j.remainder(c["page"])[:, None]
                codes, exps = _split8(s[name], rows, dh)
                scale = torch.pow(torch.tensor(2.0, dtype=torch.float64, device="cuda"), exps[line].double())
                kv.append(codes.view(torch.uint8)[line].view(torch.float8_e4m3fn).double() *
                          scale.repeat_interleave(32, dim=-1))
            else:
                kv.append(s[name][page, :, j.remainder(c["page"])].double())
        z = torch.einsum("hgd,jhd->hgj", s["q"][b].double().reshape(Hkv, G, dh), kv[0]) * s["scale"]
        out[b] = torch.einsum("hgj,jhd->hgd", torch.softmax(z, -1), kv[1]).reshape(-1)
    return out
