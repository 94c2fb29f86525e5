"""Cases for timing the operators of serving a batch that shares its prompts, with their plain forms.

Four operators, in the order in which a decoding step of such a batch uses them:

* ``arrange`` — which pages of an 8-bit cache each sequence holds: growing, cutting back,
  ending, forking and reordering sequences, with the copies of pages that only one
  sequence may write (``kv8_arrange``);
* ``compact`` — moving a pool's pages together (``kv8_compact``);
* ``rope`` — the norm of each head's query and key and the rotation by its position,
  of one or several axes, in one pass (``qk_norm_rope``);
* ``shared`` — attention over the cache for sequences that begin with the same
  tokens in the same pages (``attention_kv8_shared``).

``run`` computes them in elementary torch operations, or through the package's
entry points where ``own`` is true. ``exact`` computes them in 64 bits.
"""
import math

import torch

own = False

_DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one new token of each sequence of a decoding batch
        {"name": "rope decode b64", "op": "rope", "B": 64, "T": 1, "Hq": 64, "Hk": 8, "D": 128, "rot": 128, "axes": 1,
         "interleaved": False, "dtype": "bf16", "far": 131072},
        # prompts
        {"name": "rope prompts b8 t2048", "op": "rope", "B": 8, "T": 2048, "Hq": 64, "Hk": 8, "D": 128, "rot": 128,
         "axes": 1, "interleaved": False, "dtype": "bf16", "far": 8192},
        # patches of a video: time, height and width, part of each head turned
        {"name": "rope video t5003 fp16", "op": "rope", "B": 1, "T": 5003, "Hq": 24, "Hk": 24, "D": 128, "rot": 96,
         "axes": 3, "interleaved": True, "dtype": "fp16", "far": 512},
        # a decoding step's pages: room for four guessed tokens, then back as none was right
        {"name": "arrange step b256", "op": "arrange", "what": "step", "rows": 256, "len": 8192, "Hkv": 8, "D": 128,
         "page": 64, "layers": 1, "beams": 1},
        # sixty-four answers to one prompt: its whole pages shared, the last one copied, of four layers
        {"name": "arrange fork 1 to 64", "op": "arrange", "what": "fork", "rows": 64, "len": 16400, "Hkv": 8, "D": 128,
         "page": 64, "layers": 4, "beams": 64},
        # a step of beam search over sixteen requests of four beams
        {"name": "arrange beams 16x4", "op": "arrange", "what": "beams", "rows": 64, "len": 2000, "Hkv": 8, "D": 128,
         "page": 32, "layers": 2, "beams": 4},
        # a pool that half of the requests have left
        {"name": "compact 6000 pages", "op": "compact", "rows": 96, "len": 4000, "Hkv": 8, "D": 128, "page": 64,
         "layers": 2},
        # a few answers to a short prompt: latency
        {"name": "shared b4 p1000", "op": "shared", "groups": 1, "B": 4, "T": 1, "prefix": 1000, "tail": 60, "Hq": 64,
         "Hkv": 8, "D": 128, "page": 64, "dtype": "bf16"},
        # several requests with several answers each, sizes that fit nothing
        {"name": "shared 6 groups fp16", "op": "shared", "groups": 6, "B": 45, "T": 1, "prefix": 5003, "tail": 700,
         "Hq": 28, "Hkv": 4, "D": 64, "page": 16, "dtype": "fp16"},
        # guessed tokens: four queries of each sequence
        {"name": "shared b16 t4 p8192", "op": "shared", "groups": 2, "B": 16, "T": 4, "prefix": 8192, "tail": 500,
         "Hq": 32, "Hkv": 8, "D": 128, "page": 32, "dtype": "bf16"},
        # a batch behind one long system prompt
        {"name": "shared b64 p16384", "op": "shared", "groups": 1, "B": 64, "T": 1, "prefix": 16384, "tail": 512,
         "Hq": 64, "Hkv": 8, "D": 128, "page": 64, "dtype": "bf16"},
        {"name": "shared b128 p32768", "op": "shared", "groups": 1, "B": 128, "T": 1, "prefix": 32768, "tail": 1024,
         "Hq": 64, "Hkv": 8, "D": 128, "page": 64, "dtype": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return min(max(int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))))), lo), hi)


def draw(rng):
    op = rng.choice(("rope", "arrange", "compact", "shared", "shared"))
    if op == "rope":
        D = rng.choice((64, 80, 96, 128, 256))
        Hk = rng.choice((1, 2, 4, 8, 24))
        Hq = Hk * rng.choice((1, 2, 4, 7, 8))
        dtype = rng.choice(("bf16", "bf16", "fp16", "fp32"))
        tokens = _log_int(rng, 1, min(32768, 16384 * 72 * 128 * 2 // ((Hq + Hk) * D * (4 if dtype == "fp32" else 2))))
        B = _log_int(rng, 1, tokens)
        return {"op": op, "B": B, "T": tokens // B, "Hq": Hq, "Hk": Hk, "D": D, "rot": rng.choice((D, D, D // 32 * 16)),
                "axes": rng.choice((1, 1, 2, 3)), "interleaved": rng.random() < 0.3, "dtype": dtype,
                "far": _log_int(rng, 64, 1 << 20)}
    D, page, Hkv = rng.choice((64, 128)), rng.choice((16, 32, 64, 128)), rng.choice((1, 2, 4, 8))
    if op == "arrange":
        rows, what = _log_int(rng, 2, 256), rng.choice(("step", "fork", "beams"))
        beams = 1 if what == "step" else min(rows, rng.choice((2, 4, 8, 64)))
        rows = rows // beams * beams
        length = _log_int(rng, 20, min(16384, (1 << 18) // rows * beams))
        return {"op": op, "what": what, "rows": rows, "len": length, "Hkv": Hkv, "D": D, "page": page,
                "layers": rng.choice((1, 2, 4)), "beams": beams}
    if op == "compact":
        rows = _log_int(rng, 2, 128)
        length = _log_int(rng, 20, min(8192, 96 * 4000 // rows))
        return {"op": op, "rows": rows, "len": length, "Hkv": Hkv, "D": D, "page": page, "layers": rng.choice((1, 2))}
    group, T = rng.choice((1, 2, 4, 7, 8)), rng.choice((1, 1, 1, 2, 5))
    B = _log_int(rng, 2, 128)
    groups = min(rng.choice((1, 1, 2, 5)), B)
    prefix = _log_int(rng, 100, 65536)
    while B * T * group * Hkv * prefix * D > 128 * 64 * 32768 * 128 or groups * prefix > 65536:
        prefix = -(-prefix // 2)
    return {"op": op, "groups": groups, "B": B, "T": T, "prefix": prefix, "tail": max(T, _log_int(rng, 1, 131072 // B)),
            "Hq": Hkv * group, "Hkv": Hkv, "D": D, "page": page, "dtype": rng.choice(("bf16", "bf16", "fp16"))}


# ------------------------------------------------------------------ inputs --

def _generator(seed):
    return torch.Generator(device="cuda").manual_seed(int(seed))


def _pool(g, pages, Hkv, page, D):
    """Pages of an 8-bit cache as earlier appends left them: codes and a power of two for each page and head."""
    codes = torch.empty(pages, Hkv, page, D, dtype=torch.uint8, device="cuda")
    scales = torch.empty(pages, Hkv, dtype=torch.float32, device="cuda")
    step = max(1, (1 << 26) // (Hkv * page * D))
    for p in range(0, pages, step):
        n = min(step, pages - p)
        x = torch.randn(n, Hkv, page, D, generator=g, device="cuda", dtype=torch.float32)
        x *= 0.5 + torch.rand(n, Hkv, 1, 1, generator=g, device="cuda")
        m, e = torch.frexp(x.abs().amax((2, 3)))
        s = torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875))
        codes[p:p + n] = (x / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
        scales[p:p + n] = s
    return codes, scales


def _caches(g, layers, pages, Hkv, page, D):
    return [(*_pool(g, pages, Hkv, page, D), *_pool(g, pages, Hkv, page, D)) for _ in range(layers)]


def _i32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_rope(case, g):
    B, T, Hq, Hk, D, axes = (case[k] for k in ("B", "T", "Hq", "Hk", "D", "axes"))
    dtype = _DTYPE[case["dtype"]]
    fused = torch.randn(B, T, Hq + 2 * Hk, D, generator=g, device="cuda")       # a projection's queries, keys and values
    fused = (fused * (1.0 + 7.0 * (torch.rand(D, generator=g, device="cuda") < 0.02))).to(dtype)
    half = case["rot"] // 2
    inv_freq = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
    start = torch.randint(0, case["far"], (axes, B, 1), generator=g, device="cuda")
    if axes == 1:
        positions = (start + torch.arange(T, device="cuda")).to(torch.int32)[0]
    else:
        positions = torch.randint(0, case["far"], (axes, B, T), generator=g, device="cuda").to(torch.int32)
    sections = [half // axes] * (axes - 1)
    sections.append(half - sum(sections))
    axis = torch.tensor([a for a, n in enumerate(sections) for _ in range(n)], device="cuda")
    weight = lambda: (1.0 + 0.2 * torch.randn(D, generator=g, device="cuda")).to(dtype)  # noqa: E731
    return {"case": case, "q": fused[:, :, :Hq], "k": fused[:, :, Hq:Hq + Hk], "positions": positions, "sections": sections, "axis": axis,
            "inv_freq": inv_freq.float(), "q_weight": weight(), "k_weight": weight()}


def _prepare_arrange(case, g):
    rows, length, page, beams, what = (case[k] for k in ("rows", "len", "page", "beams", "what"))
    width = -(-(length + 8) // page) + 1
    requests = rows // beams
    lens = (length * (0.5 + 0.5 * torch.rand(requests, generator=g, device="cuda"))).int().clamp(min=1).tolist()
    held = [0] * rows
    next_page, table = 0, [[0] * width for _ in range(rows)]
    refs_of = []
    for r in range(requests):
        n = -(-lens[r] // page)
        shared = n - 1 if what == "beams" else 0        # (beams share all but their last page)
        for b in range(beams):
            row = r * beams + b
            if what == "fork" and b > 0:
                continue                                 # (an answer that is not begun)
            held[row] = lens[r]
            for s in range(n):
                if b > 0 and s < shared:
                    table[row][s] = table[r * beams][s]
                    refs_of[table[row][s]] += 1
                else:
                    table[row][s] = next_page
                    refs_of.append(1)
                    next_page += 1
    pages = requests * (-(-length // page) + (beams if what == "beams" else 0)) + rows * 3 + 5
    place = torch.randperm(pages, generator=g, device="cuda")
    order = place.cpu()
    live = torch.arange(width)[None, :] < torch.tensor([-(-h // page) for h in held])[:, None]
    table = torch.where(live, order[torch.tensor(table)].int(), 0).cuda()
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[place[:next_page]] = _i32(refs_of)
    old = _i32(held)
    state = {"case": case, "refs": refs, "table": table, "held": old,
             "caches": _caches(g, case["layers"], pages, case["Hkv"], page, case["D"]) if what != "step" else []}
    index = torch.arange(rows, device="cuda", dtype=torch.int32)
    if what == "step":
        state.update(keep=old.clone(), room=old + 4, after=old.clone())
    elif what == "fork":
        parents = index // beams * beams
        keep = old[parents.long()]                       # (a new tensor: the pool's own changes)
        state.update(keep=keep, room=keep + 1, parents=parents, after=torch.where(index == parents, old, 0))
    else:
        parents = index // beams * beams + torch.randint(0, beams, (rows,), generator=g, device="cuda").int()
        state.update(keep=old.clone(), room=old + 1, parents=parents.int())
        state["kept"] = tuple(t.clone() for t in (refs, table, old))
    return state


def _prepare_compact(case, g):
    rows, length, page = case["rows"], case["len"], case["page"]
    width = -(-length // page)
    pages = rows * width + 3
    lens = (length * (0.25 + 0.75 * torch.rand(rows, generator=g, device="cuda"))).int().clamp(min=1)
    lens = torch.where(torch.arange(rows, device="cuda") % 2 == 1, lens, 0)          # every other request has left
    lens[rows // 2] = length
    slots = torch.arange(width, device="cuda")
    live = slots < (lens[:, None] + page - 1) // page
    table = torch.randperm(pages, generator=g, device="cuda")[: rows * width].view(rows, width).int()
    refs = torch.zeros(pages, dtype=torch.int32, device="cuda")
    refs[table[live].long()] = 1
    state = {"case": case, "refs": refs, "table": table, "held": lens.int(),
             "caches": _caches(g, case["layers"], pages, case["Hkv"], page, case["D"])}
    state["kept"] = tuple(state[k].clone() for k in ("refs", "table", "held"))
    return state


def _prepare_shared(case, g):
    B, T, Hkv, D, page, G = (case[k] for k in ("B", "T", "Hkv", "D", "page", "groups"))
    prefix, tail = case["prefix"], case["tail"]
    cuts = torch.randperm(B - 1, generator=g, device="cuda")[: G - 1].sort()[0].tolist() if G > 1 else []
    offsets = [0] + [c + 1 for c in cuts] + [B]
    of = [i for i in range(G) for _ in range(offsets[i], offsets[i + 1])]
    spread = torch.rand(G, generator=g, device="cuda")
    spread[0] = 1.0
    shared = (prefix * (0.5 + 0.5 * spread)).int().clamp(min=1).tolist()
    own_tokens = (tail * (0.1 + 0.9 * torch.rand(B, generator=g, device="cuda"))).int().clamp(min=T).tolist()
    lengths = [shared[of[b]] + own_tokens[b] for b in range(B)]
    width = max(-(-n // page) for n in lengths)
    table, count = torch.zeros(B, width, dtype=torch.int32), 0
    for b in range(B):
        first = offsets[of[b]]
        whole = shared[of[b]] // page if b != first else 0       # pages that are all prefix are the first sequence's
        n = -(-lengths[b] // page)
        table[b, :whole] = table[first, :whole]
        table[b, whole:n] = torch.arange(count, count + n - whole)
        count += n - whole
    pages = count + 3
    table = torch.randperm(pages, generator=g, device="cuda").int()[table.cuda().long()]
    kc, ks = _pool(g, pages, Hkv, page, D)
    vc, vs = _pool(g, pages, Hkv, page, D)
    for b in range(B):           # the tokens of a page that is part prefix are the same in each sequence's own copy
        first = offsets[of[b]]
        if shared[of[b]] % page and b != first:
            a, z = table[first, shared[of[b]] // page].long(), table[b, shared[of[b]] // page].long()
            n = shared[of[b]] % page
            for codes, scale in ((kc, ks), (vc, vs)):
                codes[z, :, :n] = codes[a, :, :n]
                scale[z] = scale[a]
    q = torch.randn(B, T, case["Hq"], D, generator=g, device="cuda").to(_DTYPE[case["dtype"]])
    return {"case": case, "q": q, "k_codes": kc, "k_scale": ks, "v_codes": vc, "v_scale": vs, "table": table,
            "lengths": _i32(lengths), "offsets": _i32(offsets), "shared": _i32(shared),
            "most": max(offsets[i + 1] - offsets[i] for i in range(G)), "prefix_pages": -(-max(shared) // page),
            "tail_pages": max(-(-lengths[b] // page) - shared[of[b]] // page for b in range(B))}


def prepare(case, seed):
    return {"rope": _prepare_rope, "arrange": _prepare_arrange, "compact": _prepare_compact,
            "shared": _prepare_shared}[case["op"]](case, _generator(seed))


# -------------------------------------------------------------- plain forms --

def _turned(x, weight, cos, sin, interleaved):
    """One operand normalised and turned, in 32 bits."""
    y = x.float()
    y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + 1e-6) * weight.float()
    rot = 2 * cos.shape[-1]
    part = y[..., :rot]
    a, b = (part[..., 0::2], part[..., 1::2]) if interleaved else (part[..., :rot // 2], part[..., rot // 2:])
    c, d = a * cos - b * sin, a * sin + b * cos
    part = torch.stack((c, d), -1).flatten(-2) if interleaved else torch.cat((c, d), -1)
    return torch.cat((part, y[..., rot:]), -1).to(x.dtype)


def _plain_rope(state):
    positions = state["positions"]
    if positions.dim() == 2:
        positions = positions[None]
    angle = positions.permute(1, 2, 0)[..., state["axis"]].double() * state["inv_freq"].double()      # (far positions: 64 bits)
    angle = angle.remainder(2 * math.pi)
    cos, sin = angle.cos().float()[:, :, None], angle.sin().float()[:, :, None]
    il = state["case"]["interleaved"]
    return {"q": _turned(state["q"], state["q_weight"], cos, sin, il), "k": _turned(state["k"], state["k_weight"], cos, sin, il)}


def _plain_arrange_once(state, keep, room, parents):
    refs, table, held, page = state["refs"], state["table"], state["held"], state["case"]["page"]
    R, M = table.shape
    index = torch.arange(R, device=table.device)
    par = index if parents is None else parents.long()
    slots = torch.arange(M, device=table.device)
    had = (held.long() + page - 1) // page
    whole = (slots + 1) * page <= keep[:, None]
    need = slots * page < room[:, None]
    first = torch.full_like(index, R).scatter_reduce(0, par, index, "amin")
    heir = torch.where(par == index, index, first)                     # who goes on writing in a row's last page
    cand = table[par].long()
    there = slots < had[par][:, None]
    mine = there & (heir[par] == index)[:, None] & (refs[torch.where(there, cand, 0)] == 1)
    fresh = need & ~whole & ~mine
    free = torch.argsort((refs != 0).to(torch.uint8), stable=True)      # free pages first, the lowest before the others
    order = (fresh.flatten().cumsum(0) - 1).view(R, M).clamp(0, len(refs) - 1)
    missing = (fresh.sum() - (refs == 0).sum()).clamp(min=0)
    new = torch.where(need, torch.where(fresh, free[order], cand), table.long())
    part = (slots * page < keep[:, None]) & fresh & ~whole
    src, dst = cand[part], new[part]
    ok = missing == 0
    delta = torch.zeros_like(refs)
    delta.index_add_(0, torch.where(need, new, 0).flatten(), need.flatten().int())
    live = slots < had[:, None]
    delta.index_add_(0, torch.where(live, table.long(), 0).flatten(), -live.flatten().int())
    refs.add_(torch.where(ok, delta, 0))
    table.copy_(torch.where(ok, new, table))
    held.copy_(torch.where(ok, room, held))
    return src, dst, missing.int()


def _restore(state):
    """The page tables as a snapshot has them (a pass begins where the last one did)."""
    for name, t in zip(("refs", "table", "held"), state["kept"]):
        state[name].copy_(t)


def _pool_outputs(state, **more):
    e4m3 = torch.float8_e4m3fn
    return {"refs": state["refs"], "table": state["table"], "held": state["held"],
            "caches": [(k.view(e4m3), ks, v.view(e4m3), vs) for k, ks, v, vs in state["caches"]], **more}


def _copy_pages(caches, src, dst):
    return [t.index_copy_(0, dst, t[src]) for c in caches for t in c]


def _plain_arrange(state):
    what = state["case"]["what"]
    if what == "beams":
        _restore(state)
    src, dst, missing = _plain_arrange_once(state, state["keep"], state["room"], state.get("parents"))
    _copy_pages(state["caches"], src, dst)
    if what != "beams":
        _plain_arrange_once(state, state["keep"] if what == "step" else state["after"], state["after"], None)
    return _pool_outputs(state, missing=missing)


def _plain_compact(state):
    _restore(state)
    refs, table, held, page = state["refs"], state["table"], state["held"], state["case"]["page"]
    used = refs > 0
    index = torch.arange(len(refs), device=refs.device)
    count = used.sum()
    movers, holes = index[used & (index >= count)], index[~used & (index < count)]
    _copy_pages(state["caches"], movers, holes)
    moved = torch.where(used, index, -1)
    moved[movers] = holes
    live = torch.arange(table.shape[1], device=refs.device) < (held[:, None] + page - 1) // page
    table.copy_(torch.where(live, moved[torch.where(live, table, 0).long()], table))
    refs[holes] = refs[movers]
    refs[movers] = 0
    return _pool_outputs(state, moved=moved.int())


def _page_values(codes, scales, ids):
    """[rows, Hkv, tokens, D] in 32 bits of the pages ids [rows, n]."""
    x = codes[ids].view(torch.float8_e4m3fn).float() * scales[ids][..., None, None]
    n, m, Hkv, page, D = x.shape
    return x.permute(0, 2, 1, 3, 4).reshape(n, Hkv, m * page, D)


def _plain_shared(state):
    q, page, table = state["q"], state["case"]["page"], state["table"].long()
    B, T, Hq, D = q.shape
    Hkv = state["k_codes"].shape[1]
    group = Hq // Hkv
    offsets, shared, lengths = (state[k].long() for k in ("offsets", "shared", "lengths"))
    seq = torch.arange(B, device=q.device)
    of = torch.searchsorted(offsets, seq, right=True) - 1             # each sequence's group
    rows = q.float().view(B, T, Hkv, group, D).transpose(1, 2).reshape(B, Hkv, T * group, D)
    at = (lengths[:, None] - T + torch.arange(T, device=q.device)).repeat_interleave(group, 1)     # position of each row

    # the prefixes, once for each group: its sequences' rows side by side, padded to the largest group's
    member = offsets[:-1, None] + torch.arange(state["most"], device=q.device)
    present = member < offsets[1:, None]
    member = member.clamp(max=B - 1)
    stacked = rows[member].transpose(1, 2).reshape(len(member), Hkv, -1, D)
    ids = table[offsets[:-1], : state["prefix_pages"]]
    k = _page_values(state["k_codes"], state["k_scale"], ids)
    s = stacked @ k.transpose(2, 3) * D ** -0.5
    del k
    place = torch.arange(s.shape[-1], device=q.device)
    hidden = place >= torch.minimum(shared[:, None], at[member].flatten(1) + 1)[:, :, None]
    s.masked_fill_(hidden[:, None], float("-inf"))
    m1 = s.amax(-1, keepdim=True)
    s = torch.exp_(s.sub_(torch.where(m1 > float("-inf"), m1, 0.0)))
    l1 = s.sum(-1, keepdim=True)
    o1 = s @ _page_values(state["v_codes"], state["v_scale"], ids)
    del s
    pick = present.flatten().nonzero().flatten()
    m1, l1, o1 = (x.view(len(member), Hkv, state["most"], T * group, -1).transpose(1, 2).flatten(0, 1)[pick]
                  for x in (m1, l1, o1))

    # each sequence's own tokens
    first = shared[of] // page
    slots = (first[:, None] + torch.arange(state["tail_pages"], device=q.device))
    ids = table.gather(1, slots.clamp(max=table.shape[1] - 1))
    s = rows @ _page_values(state["k_codes"], state["k_scale"], ids).transpose(2, 3) * D ** -0.5
    place = (slots[:, :, None] * page + torch.arange(page, device=q.device)).flatten(1)
    hidden = (place[:, None] < shared[of][:, None, None]) | (place[:, None] > at[:, :, None])
    s.masked_fill_(hidden[:, None], float("-inf"))
    m2 = s.amax(-1, keepdim=True)
    s = torch.exp(s - torch.where(m2 > float("-inf"), m2, 0.0))
    l2 = s.sum(-1, keepdim=True)
    o2 = s @ _page_values(state["v_codes"], state["v_scale"], ids)

    m = torch.maximum(m1, m2)
    w1, w2 = torch.exp(m1 - m), torch.exp(m2 - m)
    l = l1 * w1 + l2 * w2
    o = (o1 * w1 + o2 * w2) / l
    back = lambda x: x.view(B, Hkv, T, group, -1).transpose(1, 2).reshape(B, T, Hq, -1)  # noqa: E731
    return {"o": back(o).to(q.dtype), "lse": back(m + torch.log(l))[..., 0]}


# ---------------------------------------------------------------------- run --

def run(state):
    op = state["case"]["op"]
    if own:
        return _OWN[op](state)
    return {"rope": _plain_rope, "arrange": _plain_arrange, "compact": _plain_compact, "shared": _plain_shared}[op](state)


def _own_rope(state):
    import dense_bf16_gemm_02_gb300 as hk
    q, k = hk.qk_norm_rope(state["q"], state["k"], state["positions"], state["inv_freq"], q_weight=state["q_weight"],
                           k_weight=state["k_weight"], eps=1e-6, sections=state["sections"],
                           interleaved=state["case"]["interleaved"])
    return {"q": q, "k": k}


def _own_pool(state):
    import dense_bf16_gemm_02_gb300 as hk
    return (hk.Kv8Pool(state["refs"], state["table"], state["held"], state["case"]["page"]),
            [hk.Kv8Cache(k, v, ks, vs) for k, ks, v, vs in state["caches"]])


def _own_arrange(state):
    import dense_bf16_gemm_02_gb300 as hk
    what = state["case"]["what"]
    if what == "beams":
        _restore(state)
    pool, caches = _own_pool(state)
    missing = hk.kv8_arrange(pool, state["keep"], state["room"], parents=state.get("parents"), caches=caches)
    if what != "beams":
        hk.kv8_arrange(pool, state["keep"] if what == "step" else state["after"], state["after"])
    return _pool_outputs(state, missing=missing)


def _own_compact(state):
    import dense_bf16_gemm_02_gb300 as hk
    _restore(state)
    pool, caches = _own_pool(state)
    return _pool_outputs(state, moved=hk.kv8_compact(pool, caches=caches))


def _own_shared(state):
    import dense_bf16_gemm_02_gb300 as hk
    cache = hk.Kv8Cache(state["k_codes"], state["v_codes"], state["k_scale"], state["v_scale"])
    o, lse = hk.attention_kv8_shared(state["q"], cache, state["table"], state["lengths"], state["offsets"], state["shared"],
                                     causal=True, return_lse=True)
    return {"o": o, "lse": lse}


_OWN = {"rope": _own_rope, "arrange": _own_arrange, "compact": _own_compact, "shared": _own_shared}


# --------------------------------------------------------------------- work --

def work(case):
    op = case["op"]
    if op == "rope":
        n = case["B"] * case["T"] * (case["Hq"] + case["Hk"]) * case["D"]
        return {"bytes": 2 * n * (4 if case["dtype"] == "fp32" else 2), "flops": 7 * n}
    page_bytes = 2 * case["Hkv"] * case["page"] * case["D"] + 8 * case["Hkv"]
    if op == "arrange":
        rows, beams = case["rows"], case["beams"]
        entries = rows * 0.75 * case["len"] / case["page"]
        copied = {"step": 0, "fork": rows - rows // beams, "beams": rows * (1 - 1 / beams) ** beams}[case["what"]]
        return {"bytes": 8 * entries + 2 * copied * page_bytes * case["layers"], "flops": entries}
    if op == "compact":
        width = -(-case["len"] // case["page"])
        live = case["rows"] / 2 * 0.625 * width
        moved = live * (1 - live / (case["rows"] * width))
        return {"bytes": 2 * moved * page_bytes * case["layers"] + 8 * live, "flops": live}
    B, T, D, Hkv, Hq = (case[k] for k in ("B", "T", "D", "Hkv", "Hq"))
    prefix = case["prefix"] * (1.0 if case["groups"] == 1 else 1 / case["groups"] + (1 - 1 / case["groups"]) * 0.75)
    tail = max(T, 0.55 * case["tail"])
    return {"bytes": 2 * Hkv * D * (case["groups"] * prefix + B * tail) + 4 * B * T * Hq * D,
            "flops": 4 * B * T * Hq * D * (prefix + tail)}


# -------------------------------------------------------------------- exact --

def _exact_rope(state):
    pos = state["positions"].double()
    pos = pos[None] if pos.dim() == 2 else pos
    freq = state["inv_freq"].double()
    starts = [sum(state["sections"][:a]) for a in range(len(state["sections"]) + 1)]
    angle = torch.cat([pos[a][..., None] * freq[starts[a]:starts[a + 1]] for a in range(len(state["sections"]))], -1)
    turn = torch.polar(torch.ones_like(angle), angle)[:, :, None]
    out = {}
    for name in ("q", "k"):
        x = state[name].double()
        x = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + 1e-6).sqrt() * state[name + "_weight"].double()
        n = angle.shape[-1]
        for i in range(n):
            a, b = (2 * i, 2 * i + 1) if state["case"]["interleaved"] else (i, i + n)
            z = torch.complex(x[..., a], x[..., b]) * turn[..., i]
            x[..., a], x[..., b] = z.real, z.imag
        out[name] = x
    return out


def _exact_arrange_once(pool, keep, room, parents, page):
    """The rows one after the other; the pages to copy."""
    refs, table, held = pool
    R = len(table)
    parents = list(range(R)) if parents is None else parents
    before, old, had = list(refs), [list(r) for r in table], [-(-h // page) for h in held]
    free, copies = [p for p, n in enumerate(before) if n == 0], []
    for i in range(R):
        p = parents[i]
        heir = p if parents[p] == p else min(j for j in range(R) if parents[j] == p)
        for s in range(-(-room[i] // page)):
            from_parent = old[p][s] if s < had[p] else None
            if (s + 1) * page <= keep[i] or (from_parent is not None and heir == i and before[from_parent] == 1):
                table[i][s] = from_parent
            else:
                table[i][s] = free.pop(0)
                if s * page < keep[i]:
                    copies.append((from_parent, table[i][s]))
            refs[table[i][s]] += 1
        for s in range(had[i]):
            refs[old[i][s]] -= 1
        held[i] = room[i]
    return copies


def _exact_caches(state, copies):
    out = []
    for k, ks, v, vs in state["caches"]:
        layer = [k.view(torch.float8_e4m3fn).double(), ks.double(), v.view(torch.float8_e4m3fn).double(), vs.double()]
        for t in layer:
            source = t[[a for a, _ in copies]]
            for (_, b), x in zip(copies, source):
                t[b] = x
        out.append(tuple(layer))
    return out


def _exact_pool(pool, caches, **more):
    refs, table, held = (torch.tensor(x, dtype=torch.int32) for x in pool)
    return {"refs": refs, "table": table, "held": held, "caches": caches, **more}


def _exact_arrange(state):
    pool = [state[k].tolist() for k in ("refs", "table", "held")]
    page, what = state["case"]["page"], state["case"]["what"]
    parents = state["parents"].tolist() if "parents" in state else None
    copies = _exact_arrange_once(pool, state["keep"].tolist(), state["room"].tolist(), parents, page)
    if what != "beams":
        after = state["after"].tolist()
        _exact_arrange_once(pool, state["keep"].tolist() if what == "step" else after, after, None, page)
    return _exact_pool(pool, _exact_caches(state, copies), missing=torch.tensor(0, dtype=torch.int32))


def _exact_compact(state):
    refs, table, held = (state[k].tolist() for k in ("refs", "table", "held"))
    page, count = state["case"]["page"], sum(n > 0 for n in refs)
    movers = [p for p in range(count, len(refs)) if refs[p] > 0]
    holes = [p for p in range(count) if refs[p] == 0]
    goes = dict(zip(movers, holes))
    for row, h in zip(table, held):
        for s in range(-(-h // page)):
            row[s] = goes.get(row[s], row[s])
    moved = torch.tensor([goes.get(p, p) if n > 0 else -1 for p, n in enumerate(refs)], dtype=torch.int32)
    for a, b in goes.items():
        refs[b], refs[a] = refs[a], 0
    return _exact_pool((refs, table, held), _exact_caches(state, list(goes.items())), moved=moved)


def _exact_shared(state):
    c = state["case"]
    if c["B"] * c["T"] * c["Hq"] * (c["prefix"] + c["tail"]) * c["D"] > 1 << 36:
        return None
    q, page = state["q"].double(), c["page"]
    B, T, Hq, D = q.shape
    Hkv = c["Hkv"]
    out, lse = torch.zeros_like(q), torch.zeros(B, T, Hq, dtype=torch.float64, device=q.device)
    for b, n in enumerate(state["lengths"].tolist()):
        ids = state["table"][b, : -(-n // page)].long()
        k, v = ((state[x + "_codes"][ids].view(torch.float8_e4m3fn).double() * state[x + "_scale"][ids].double()[:, :, None, None])
                .transpose(0, 1).reshape(Hkv, -1, D)[:, :n] for x in "kv")
        s = torch.einsum("thgd,hld->thgl", q[b].view(T, Hkv, Hq // Hkv, D), k) / math.sqrt(D)
        seen = torch.arange(n, device=q.device)[None, :] <= (n - T + torch.arange(T, device=q.device))[:, None]
        s = s.masked_fill(~seen[:, None, None], float("-inf"))
        out[b] = torch.einsum("thgl,hld->thgd", torch.softmax(s, -1), v).reshape(T, Hq, D)
        lse[b] = torch.logsumexp(s, -1).view(T, Hq)
    return {"o": out, "lse": lse}


def exact(case, seed):
    state = prepare(case, seed)
    return {"rope": _exact_rope, "arrange": _exact_arrange, "compact": _exact_compact, "shared": _exact_shared}[case["op"]](state)
