"""Cases for timing the low-precision serving operators, with their plain forms.

Four operators that a serving step runs one after the other:

* ``quantize`` — a matrix to microscaled 4-bit floating point and back to the
  values its codes stand for (``quantize_fp4``, ``dequantize_fp4``);
* ``gemm`` — the product of two such matrices, C = A·Bᵀ in bf16 (``gemm_fp4``);
* ``append`` — new keys and values into a paged 8-bit cache with one scale per
  page and head (``kv8_append``);
* ``attention`` — queries over that cache (``attention_kv8``).

``run`` computes them in elementary torch operations, or through the package's
entry points where ``own`` is true. ``exact`` computes them in 64 bits.
"""
import math

import torch

own = False

_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)      # magnitudes of E2M1
_BLOCK = {"mxfp4": 32, "nvfp4": 16}
_DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one token's hidden state, quantised ahead of a projection
        {"name": "quantize mxfp4 1x8192", "op": "quantize", "format": "mxfp4", "rows": 1, "cols": 8192, "dtype": "bf16"},
        # an odd matrix: fp32 master weights with a last block that is not whole
        {"name": "quantize nvfp4 1000x5003 fp32", "op": "quantize", "format": "nvfp4", "rows": 1000, "cols": 5003,
         "dtype": "fp32"},
        # a prompt's activations (or a weight matrix)
        {"name": "quantize mxfp4 16384x8192", "op": "quantize", "format": "mxfp4", "rows": 16384, "cols": 8192,
         "dtype": "bf16"},
        # single-token decode through the up-projection: weights streamed once
        {"name": "gemm mxfp4 1x28672x8192", "op": "gemm", "format": "mxfp4", "M": 1, "N": 28672, "K": 8192},
        # a batch of decoding sequences, ragged sizes
        {"name": "gemm nvfp4 100x8200x5000", "op": "gemm", "format": "nvfp4", "M": 100, "N": 8200, "K": 5000},
        # a prompt chunk through the same projection as the bf16 benchmark's square shapes
        {"name": "gemm nvfp4 4096x4096x4096", "op": "gemm", "format": "nvfp4", "M": 4096, "N": 4096, "K": 4096},
        {"name": "gemm mxfp4 8192x8192x8192", "op": "gemm", "format": "mxfp4", "M": 8192, "N": 8192, "K": 8192},
        # one new token for each sequence of a decoding batch
        {"name": "append decode b64", "op": "append", "B": 64, "T": 1, "Hkv": 8, "D": 128, "page": 64, "past": 1000},
        # a batch of prompts, each of another length
        {"name": "append prompts b8 t2048", "op": "append", "B": 8, "T": 2048, "Hkv": 8, "D": 128, "page": 64,
         "past": 37},
        # one short sequence decoding: latency
        {"name": "attention decode b1 l500", "op": "attention", "B": 1, "T": 1, "Hq": 64, "Hkv": 8, "D": 128,
         "page": 64, "len": 500},
        # a decoding batch, sequences of every length up to 32768
        {"name": "attention decode b64 l32768", "op": "attention", "B": 64, "T": 1, "Hq": 64, "Hkv": 8, "D": 128,
         "page": 64, "len": 32768},
        # a chunk of a long prompt against what the cache holds already
        {"name": "attention chunk b2 t2048 l16384", "op": "attention", "B": 2, "T": 2048, "Hq": 64, "Hkv": 8, "D": 128,
         "page": 64, "len": 16384},
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    n = min(max(n, lo), hi)
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(("quantize", "gemm", "append", "attention"))
    if op == "quantize":
        cols = _log_int(rng, 64, 28672)
        return {"op": op, "format": rng.choice(("mxfp4", "nvfp4")), "rows": _log_int(rng, 1, min(32768, (1 << 27) // cols)),
                "cols": cols, "dtype": rng.choice(("bf16", "bf16", "fp16", "fp32"))}
    if op == "gemm":
        while True:
            M, N, K = _log_int(rng, 1, 8192), _log_int(rng, 256, 28672), _log_int(rng, 256, 16384)
            if rng.random() < 0.7:      # widths of models are round, those of vocabularies and batches are not
                N, K = -(-N // 128) * 128, -(-K // 128) * 128
            if M * N * K <= 1 << 38 and 3072 not in (N, K):
                return {"op": op, "format": rng.choice(("mxfp4", "nvfp4")), "M": M, "N": N, "K": K}
    D, page, Hkv = rng.choice((64, 128)), rng.choice((16, 32, 64, 128)), rng.choice((1, 2, 4, 8))
    if op == "append":
        B = _log_int(rng, 1, 128)
        return {"op": op, "B": B, "T": _log_int(rng, 1, max(1, 16384 // B)), "Hkv": Hkv, "D": D, "page": page,
                "past": rng.choice((0, _log_int(rng, 1, 2000)))}
    group = rng.choice((1, 2, 4, 7, 8))
    if rng.random() < 0.6:              # decoding, one or a few tokens a step
        B = _log_int(rng, 1, 128)
        T = rng.choice((1, 1, 2, 5))
        length = _log_int(rng, 16, min(131072, (1 << 21) // B))
    else:                               # a prompt's chunk
        B, T = rng.choice((1, 1, 2, 4)), _log_int(rng, 16, 2048)
        length = _log_int(rng, T, 16384)
        while B * T * length * Hkv * group * D > 2 * 2048 * 16384 * 64 * 128:
            B, T = 1, -(-T // 2)
    return {"op": op, "B": B, "T": T, "Hq": Hkv * group, "Hkv": Hkv, "D": D, "page": page, "len": max(length, T)}


# ------------------------------------------------------------------ inputs --

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _activations(g, rows, cols, dtype):
    """Normal values with a few columns that are much larger, as hidden states have them."""
    x = torch.randn(rows, cols, generator=g, device="cuda", dtype=torch.float32)
    x *= 1.0 + 15.0 * (torch.rand(cols, generator=g, device="cuda") < 0.01)
    return x.to(dtype)


def _pack_fp4(x, fmt, g):
    """Codes [rows, K/2 padded], scales in 128×4 tiles, as a quantised matrix is kept."""
    rows, K = x.shape
    blk = _BLOCK[fmt]
    Kp = -(-K // 256) * 256
    values, scales = _fp4_parts(torch.nn.functional.pad(x.float(), (0, Kp - K)), fmt, g)
    grid = torch.tensor(_GRID, device=x.device)
    code = torch.searchsorted(grid, values.abs()).to(torch.uint8) + 8 * torch.signbit(values).to(torch.uint8)
    code = code.view(rows, Kp)
    codes = code[:, 0::2] | (code[:, 1::2] << 4)
    if fmt == "mxfp4":
        byte = torch.where(scales == 0, 0, torch.frexp(scales)[1] + 126).to(torch.uint8)
    else:
        byte = scales.to(torch.float8_e4m3fn).view(torch.uint8)
    nb = Kp // blk
    rp = -(-rows // 128) * 128
    full = torch.zeros(rp, nb, dtype=torch.uint8, device=x.device)
    full[:rows] = byte
    tiles = full.view(rp // 128, 4, 32, nb // 4, 4).permute(0, 3, 2, 1, 4).contiguous().view(-1)
    return codes[:, : -(-K // 32) * 16].contiguous(), tiles


def _weights_fp4(g, rows, cols, fmt, gscale):
    codes, tiles = [], []
    for r in range(0, rows, 4096):      # (a multiple of 128 rows at a time keeps the tiles whole)
        x = torch.randn(min(4096, rows - r), cols, generator=g, device="cuda")
        c, t = _pack_fp4(x, fmt, gscale)
        codes.append(c)
        tiles.append(t)
    return torch.cat(codes), torch.cat(tiles)


def _pool(g, pages, Hkv, page, D, used):
    """Pages of an 8-bit cache as earlier appends left them: codes and a power of two for each page and head."""
    codes = torch.empty(pages, Hkv, page, D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, Hkv, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (Hkv * page * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn(n, Hkv, page, D, generator=g, device="cuda", dtype=torch.bfloat16).float()
        x *= 0.5 + torch.rand(n, Hkv, 1, 1, generator=g, device="cuda")
        s = _page_scale(x.abs().amax((2, 3)))
        codes[p:p + n] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[p:p + n] = s
    return codes, scales


def prepare(case, seed):
    g = _generator(seed)
    op = case["op"]
    if op == "quantize":
        x = _activations(g, case["rows"], case["cols"], _DTYPE[case["dtype"]])
        gs = x.float().abs().amax().reshape(1) / 2688.0 if case["format"] == "nvfp4" else None
        return {"case": case, "x": x, "gscale": gs}
    if op == "gemm":
        fmt = case["format"]
        ga = torch.full((1,), 0.02, device="cuda") if fmt == "nvfp4" else None
        gb = torch.full((1,), 0.002, device="cuda") if fmt == "nvfp4" else None
        a = _weights_fp4(g, case["M"], case["K"], fmt, ga)
        b = _weights_fp4(g, case["N"], case["K"], fmt, gb)
        return {"case": case, "a": a, "b": b, "ga": ga, "gb": gb}
    B, T, Hkv, D, page = (case[k] for k in ("B", "T", "Hkv", "D", "page"))
    if op == "append":
        spread = torch.rand(B, generator=g, device="cuda")
        starts = (case["past"] * (0.5 + 0.5 * spread)).to(torch.int32)
        counts = (T - (T // 2) * torch.rand(B, generator=g, device="cuda")).to(torch.int32).clamp(1, T)
        width = -(-(case["past"] + T) // page)
    else:
        spread = torch.rand(B, generator=g, device="cuda")
        spread[0] = 1.0                  # the longest is there, the others are spread below it
        lengths = (case["len"] * (0.25 + 0.75 * spread)).to(torch.int32).clamp(min=min(T, case["len"]))
        width = -(-case["len"] // page)
    pages = B * width + 3
    table = torch.randperm(pages, generator=g, device="cuda")[: B * width].view(B, width).to(torch.int32)
    kc, ks = _pool(g, pages, Hkv, page, D, width)
    vc, vs = _pool(g, pages, Hkv, page, D, width)
    state = {"case": case, "k_codes": kc, "k_scale": ks, "v_codes": vc, "v_scale": vs, "table": table}
    if op == "append":
        shape = (B, T, Hkv, D)
        state["k"] = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        state["v"] = torch.randn(shape, generator=g, device="cuda").to(torch.bfloat16)
        state["starts"], state["counts"] = starts, counts
    else:
        state["q"] = torch.randn(B, T, case["Hq"], D, generator=g, device="cuda").to(torch.bfloat16)
        state["lengths"] = lengths
    return state


# -------------------------------------------------------------- plain forms --

def _fp4_parts(x, fmt, gscale):
    """(E2M1 values [R, blocks, blk], scales [R, blocks]) of x in 32 bits; x's width is a multiple of the block."""
    R, K = x.shape
    b = x.float().view(R, -1, _BLOCK[fmt])
    amax = b.abs().amax(-1)
    finite = torch.isfinite(amax)
    if fmt == "mxfp4":
        e = (torch.frexp(amax)[1] - 3).clamp(-127, 127)
        one = torch.ones_like(amax)
        scale = torch.where(amax > 0, torch.ldexp(one, e), torch.zeros_like(one))
        y = b * torch.ldexp(one, -e)[..., None]
    else:
        s = (amax / (6.0 * gscale)).clamp(max=448.0).to(torch.float8_e4m3fn).float()
        d = s * gscale
        scale = s
        y = b * torch.where(d > 0, 1.0 / d, torch.zeros_like(d))[..., None]
    m = y.abs()
    q = torch.zeros_like(m)
    # a step up at each border; a tie goes to the code that is even
    for border, step, tie_up in ((0.25, 0.5, False), (0.75, 0.5, True), (1.25, 0.5, False), (1.75, 0.5, True),
                                 (2.5, 1.0, False), (3.5, 1.0, True), (5.0, 2.0, False)):
        q += step * ((m >= border) if tie_up else (m > border))
    q = torch.copysign(q, b)
    q = torch.where(finite[..., None], q, torch.zeros_like(q))
    return q, torch.where(finite, scale, torch.full_like(scale, float("nan")))


def _plain_quantize(state):
    x, fmt = state["x"], state["case"]["format"]
    R, K = x.shape
    pad = -K % _BLOCK[fmt]
    values, scales = _fp4_parts(torch.nn.functional.pad(x, (0, pad)), fmt, state["gscale"])
    if fmt == "nvfp4":
        scales = scales * state["gscale"]
    return (values * scales[..., None]).view(R, -1)[:, :K].to(torch.bfloat16)


def _fp4_values(codes, tiles, fmt, rows, K, dtype):
    """The values of a quantised matrix [rows, K] without its global scale."""
    lut = torch.tensor(_GRID + tuple(-v for v in _GRID), device=codes.device, dtype=dtype)
    c = torch.stack((codes & 15, codes >> 4), -1).view(rows, -1)[:, :K].long()
    blk = _BLOCK[fmt]
    nb = -(-K // 256) * 256 // blk
    s = tiles.view(-1, nb // 4, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, nb)[:rows]
    if fmt == "mxfp4":
        s = torch.ldexp(torch.ones_like(s, dtype=dtype), s.int() - 127)
    else:
        s = s.view(torch.float8_e4m3fn).to(dtype)
    return lut[c] * s.repeat_interleave(blk, 1)[:, :K]


def _plain_gemm(state):
    c = state["case"]
    a = _fp4_values(*state["a"], c["format"], c["M"], c["K"], torch.float32)
    b = _fp4_values(*state["b"], c["format"], c["N"], c["K"], torch.float32)
    r = a @ b.t()
    if state["ga"] is not None:
        r = r * (state["ga"] * state["gb"])
    return r.to(torch.bfloat16)


def _page_scale(amax):
    """The smallest power of two s with amax <= 448 s."""
    m, e = torch.frexp(amax)
    e = torch.where(amax > 0, e - 9 + (m > 0.875), torch.full_like(e, -126)).clamp(-126, 127)
    return torch.ldexp(torch.ones_like(amax), e)


def _append_one(codes, scales, new, table, starts, counts):
    P, Hkv, page, D = codes.shape
    B, T = new.shape[:2]
    first = starts.long() // page                                   # first page of each sequence that is touched
    n = (T + page - 2) // page + 1                                  # pages a sequence can touch
    slot = first[:, None] + torch.arange(n, device=new.device)
    last = (starts.long() + counts - 1) // page
    live = (slot <= last[:, None]) & (slot < table.shape[1])
    ids = torch.where(live, table.long().gather(1, slot.clamp(max=table.shape[1] - 1)), 0)
    pos = slot[:, :, None] * page + torch.arange(page, device=new.device)          # [B, n, page]
    t = pos - starts.long()[:, None, None]
    is_new = (t >= 0) & (t < counts.long()[:, None, None])
    is_old = t < 0
    rows = new.float()[torch.arange(B, device=new.device)[:, None, None], t.clamp(0, T - 1)]   # [B, n, page, Hkv, D]
    rows = rows.permute(0, 1, 3, 2, 4)                              # [B, n, Hkv, page, D]
    mag = torch.where(is_new[:, :, None, :, None] & torch.isfinite(rows), rows.abs(), 0.0).amax((3, 4))
    need = _page_scale(mag)
    had = scales[ids]
    old_there = is_old.any(-1)[:, :, None]
    s = torch.where(old_there, torch.maximum(need, had), need)
    old = codes[ids]
    shrunk = (old.view(torch.float8_e4m3fn).float() * (had / s)[..., None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    put = (rows / s[..., None, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
    pick = torch.where(is_new[:, :, None, :, None], put, torch.where(is_old[:, :, None, :, None], shrunk, old))
    at = ids[live]
    codes[at] = pick[live]
    scales[at] = s[live]


def _plain_append(state):
    _append_one(state["k_codes"], state["k_scale"], state["k"], state["table"], state["starts"], state["counts"])
    _append_one(state["v_codes"], state["v_scale"], state["v"], state["table"], state["starts"], state["counts"])
    return _cache_outputs(state)


def _cache_outputs(state):
    return {"k": state["k_codes"].view(torch.float8_e4m3fn), "v": state["v_codes"].view(torch.float8_e4m3fn),
            "k_scale": state["k_scale"], "v_scale": state["v_scale"]}


def _gathered(codes, scales, table):
    """[B, Hkv, L, D] in 32 bits."""
    ids = table.long()
    x = codes[ids].view(torch.float8_e4m3fn).float() * scales[ids][..., None, None]
    B, n, Hkv, page, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(B, Hkv, n * page, D)


def _plain_attention(state):
    q, lengths = state["q"], state["lengths"].long()
    B, T, Hq, D = q.shape
    k = _gathered(state["k_codes"], state["k_scale"], state["table"])
    v = _gathered(state["v_codes"], state["v_scale"], state["table"])
    Hkv, L = k.shape[1:3]
    rows = q.float().view(B, T, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    s = rows @ k.transpose(2, 3)
    s *= D ** -0.5
    at = (lengths[:, None] - T + torch.arange(T, device=q.device)).repeat(1, Hq // Hkv)     # position of each row
    hidden = torch.arange(L, device=q.device) > at[:, :, None]
    s.masked_fill_(hidden[:, None], float("-inf"))
    m = s.amax(-1, keepdim=True)
    p = torch.exp_(s.sub_(torch.where(m > float("-inf"), m, 0.0)))
    l = p.sum(-1, keepdim=True)
    o = (p @ v) / torch.where(l > 0, l, 1.0)
    return o.view(B, Hkv, Hq // Hkv, T, D).permute(0, 3, 1, 2, 4).reshape(B, T, Hq, D).to(q.dtype)


# ---------------------------------------------------------------------- run --

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return {"quantize": _plain_quantize, "gemm": _plain_gemm, "append": _plain_append,
            "attention": _plain_attention}[op](state)


def _own_quantize(state):
    import dense_bf16_gemm_02_gb300 as hk
    q = hk.quantize_fp4(state["x"], format=state["case"]["format"], global_scale=state["gscale"])
    return hk.dequantize_fp4(q)


def _own_gemm(state):
    import dense_bf16_gemm_02_gb300 as hk
    c = state["case"]
    a = hk.Fp4Matrix(*state["a"], c["M"], c["K"], c["format"], state["ga"])
    b = hk.Fp4Matrix(*state["b"], c["N"], c["K"], c["format"], state["gb"])
    return hk.gemm_fp4(a, b)


def _own_cache(state):
    import dense_bf16_gemm_02_gb300 as hk
    return hk.Kv8Cache(state["k_codes"], state["v_codes"], state["k_scale"], state["v_scale"])


def _own_append(state):
    import dense_bf16_gemm_02_gb300 as hk
    hk.kv8_append(_own_cache(state), state["k"], state["v"], state["table"], state["starts"], counts=state["counts"])
    return _cache_outputs(state)


def _own_attention(state):
    import dense_bf16_gemm_02_gb300 as hk
    return hk.attention_kv8(state["q"], _own_cache(state), state["table"], state["lengths"], causal=True)


_OWN = {"quantize": _own_quantize, "gemm": _own_gemm, "append": _own_append, "attention": _own_attention}


# --------------------------------------------------------------------- work --

def work(case):
    op = case["op"]
    if op == "quantize":
        n = case["rows"] * case["cols"]
        packed = n / 2 + n / _BLOCK[case["format"]]
        size = 4 if case["dtype"] == "fp32" else 2
        return {"bytes": n * size + packed + 2 * n, "flops": 4 * n}
    if op == "gemm":
        M, N, K = case["M"], case["N"], case["K"]
        return {"bytes": (M + N) * K * (0.5 + 1 / _BLOCK[case["format"]]) + 2 * M * N, "flops": 2 * M * N * K}
    B, T, Hkv, D = (case[k] for k in ("B", "T", "Hkv", "D"))
    if op == "append":
        new = 2 * 0.75 * B * T * Hkv * D if T > 1 else 2 * B * T * Hkv * D
        return {"bytes": 3 * new, "flops": 4 * new}
    mean = (1.0 if B == 1 else 1 / B + (1 - 1 / B) * 0.625) * case["len"]
    seen = max(1.0, mean - T / 2)
    return {"bytes": 2 * B * mean * Hkv * D + 4 * B * T * case["Hq"] * D, "flops": 4 * B * T * seen * case["Hq"] * D}


# -------------------------------------------------------------------- exact --

def _exact_quantize(state):
    x, fmt = state["x"].double(), state["case"]["format"]
    R, K = x.shape
    blk = _BLOCK[fmt]
    b = torch.nn.functional.pad(x, (0, -K % blk)).view(R, -1, blk)
    top = b.abs().max(-1, keepdim=True).values
    if fmt == "mxfp4":
        d = torch.exp2(_floor_log2(top.clamp(min=2.0 ** -140)) - 2).clamp(min=2.0 ** -127)
    else:
        d = _half_even(top / (6 * state["gscale"].double()), 3, -6, 448.0) * state["gscale"].double()
    y = torch.where(d > 0, b / d, 0.0)
    return (_half_even(y, 1, 0, 6.0) * d).view(R, -1)[:, :K]


def _floor_log2(x):
    return torch.frexp(x)[1].double() - 1     # (a logarithm may round past a power of two)


def _half_even(y, bits, e_min, top):
    """y to the nearest number of `bits` fraction bits and least exponent e_min, halves to even, at most `top`."""
    step = torch.exp2(_floor_log2(y.abs().clamp(min=2.0 ** -300)).clamp(min=e_min) - bits)
    return (torch.round(y / step) * step).clamp(-top, top)


def _exact_gemm(state):
    c = state["case"]
    if c["M"] * c["N"] * c["K"] > 1 << 40:
        return None
    a = _fp4_values(*state["a"], c["format"], c["M"], c["K"], torch.float64)
    b = _fp4_values(*state["b"], c["format"], c["N"], c["K"], torch.float64)
    scale = float(state["ga"].double() * state["gb"].double()) if state["ga"] is not None else 1.0
    return torch.einsum("mk,nk->mn", a, b) * scale


def _exact_append(state):
    out = {}
    for name in ("k", "v"):
        codes, scale, new = state[name + "_codes"].clone(), state[name + "_scale"].double(), state[name].double()
        P, Hkv, page, D = codes.shape
        values = codes.view(torch.float8_e4m3fn).double()
        starts, counts, table = state["starts"].tolist(), state["counts"].tolist(), state["table"].tolist()
        for b, (s0, n) in enumerate(zip(starts, counts)):
            for slot in range(s0 // page, (s0 + n - 1) // page + 1):
                p = table[b][slot]
                lo, hi = max(s0, slot * page), min(s0 + n, (slot + 1) * page)
                x = new[b, lo - s0:hi - s0].transpose(0, 1)             # [Hkv, tokens, D]
                ratio = x.abs().amax((1, 2)).clamp(min=2.0 ** -130) / 448.0
                e = _floor_log2(ratio)
                s = torch.exp2((e + (torch.exp2(e) < ratio)).clamp(min=-126))
                if lo > slot * page:
                    s = torch.maximum(s, scale[p])
                    keep = slice(0, lo - slot * page)
                    values[p, :, keep] = _half_even(values[p, :, keep] * (scale[p] / s)[:, None, None], 3, -6, 448.0)
                values[p, :, lo - slot * page:hi - slot * page] = _half_even(x / s[:, None, None], 3, -6, 448.0)
                scale[p] = s
        out[name], out[name + "_scale"] = values, scale
    return {k: out[k] for k in ("k", "v", "k_scale", "v_scale")}


def _exact_attention(state):
    q, page = state["q"].double(), state["case"]["page"]
    B, T, Hq, D = q.shape
    Hkv = state["k_codes"].shape[1]
    out = torch.zeros_like(q)
    for b, n in enumerate(state["lengths"].tolist()):
        ids = state["table"][b, : -(-n // page)].long()
        kv = []
        for codes, scale in ((state["k_codes"], state["k_scale"]), (state["v_codes"], state["v_scale"])):
            x = codes[ids].view(torch.float8_e4m3fn).double() * scale[ids].double()[:, :, None, None]
            kv.append(x.transpose(1, 2).reshape(-1, Hkv, D)[:n])
        for h in range(Hkv):
            hs = slice(h * (Hq // Hkv), (h + 1) * (Hq // Hkv))
            s = torch.einsum("tgd,ld->gtl", q[b, :, hs], kv[0][:, h]) / math.sqrt(D)
            seen = torch.arange(n, device=q.device)[None, :] <= (n - T + torch.arange(T, device=q.device))[:, None]
            s = torch.softmax(s.masked_fill(~seen, float("-inf")), -1).nan_to_num(0.0)
            out[b, :, hs] = torch.einsum("gtl,ld->tgd", s, kv[1][:, h])
    return out


def exact(case, seed):
    state = prepare(case, seed)
    return {"quantize": _exact_quantize, "gemm": _exact_gemm, "append": _exact_append,
            "attention": _exact_attention}[case["op"]](state)
