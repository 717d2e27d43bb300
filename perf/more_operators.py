"""Measured cases of the cache operators of a target layer whose keys are rotated and whose cache may be held in 4 bits:

  rotate  a chunk's keys and queries rotated by their positions, keys and values written into the pages (bf16, f32)
  store   the same into a 4-bit cache, and the chunk read back from it
  read    cached tokens read out of the pages into dense rows
  attend  attention of a chunk of new tokens per slot over a 4-bit cache

Layouts, shared by the plain forms and the library.  E = 16 bytes / element size, D = head_dim:
  K [layers, pages, kv_heads, D / E, page, E], V [layers, pages, kv_heads, page / E, D, E] (bf16, f32),
  4 bits: K, V uint8 [layers, pages, page_bytes], a page holds the codes of all heads, then the scales of all heads:
    K codes  [kv_heads, D / 32, page, 16]            byte i: elements 2 i (low four bits) and 2 i + 1 of a block of 32
    V codes  [kv_heads, page / 8, D / 64, 16, 2, 8]  byte (o, g, n, h, t): elements n D / 16 + 4 g + 2 h and the next
                                                      of token 8 o + t
    scales   [kv_heads, D / 32, page]                2 ^ (byte - 127), of a block of 32 elements of a token
    a code: sign bit, then the place among 0, 0.5, 1, 1.5, 2, 3, 4, 6
  table [slots, max_pages] int32 (-1: no page), lens, held [slots] int32 (tokens, pages), refs [pages] int32,
  free_bits [ceil(pages / 32)] int32 (bit p % 32 of word p / 32: page p is free), n_free [1] int32.
"""
import math

import torch

own = False

_T = {"f32": torch.float32, "bf16": torch.bfloat16}
_SIZE = {"f32": 4, "bf16": 2}
_LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one stream's decoded token, 32 query heads on 8: latency
        {"name": "rotate_one", "op": "rotate", "dtype": "bf16", "slots": 1, "ctx": 1000, "chunk": 1, "ragged": 0,
         "page": 16, "heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128, "interleaved": False},
        # the smallest workload's verify chunk in binary32; neighbouring pairs, half of the dimensions rotated
        {"name": "rotate_tiny_f32", "op": "rotate", "dtype": "f32", "slots": 4, "ctx": 300, "chunk": 9, "ragged": 1,
         "page": 16, "heads": 8, "kv_heads": 8, "head_dim": 64, "rot": 32, "interleaved": True},
        # the verify chunk of 256 requests, all 17 tokens
        {"name": "rotate_verify_large", "op": "rotate", "dtype": "bf16", "slots": 256, "ctx": 4096, "chunk": 17,
         "ragged": 0, "page": 64, "heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128, "interleaved": False},
        # one decoded token of 32 requests into a 4-bit cache: latency
        {"name": "store_decode", "op": "store", "dtype": "bf16", "slots": 32, "ctx": 2100, "chunk": 1, "ragged": 0,
         "page": 32, "heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128, "interleaved": False},
        # two prompts' chunks into a 4-bit cache
        {"name": "store_prompt", "op": "store", "dtype": "bf16", "slots": 2, "ctx": 8192, "chunk": 2048, "ragged": 0,
         "page": 64, "heads": 32, "kv_heads": 8, "head_dim": 128, "rot": 128, "interleaved": False},
        # the smallest workload's cached tokens, binary32
        {"name": "read_tiny_f32", "op": "read", "pool": "f32", "dtype": "f32", "slots": 4, "ctx": 300, "page": 16,
         "kv_heads": 8, "head_dim": 64},
        # eight requests' prefixes of up to 20,000 tokens taken out of a 4-bit cache
        {"name": "read_prefix", "op": "read", "pool": "4bit", "dtype": "bf16", "slots": 8, "ctx": 20000, "page": 64,
         "kv_heads": 8, "head_dim": 128},
        # one stream decoding a token over a long context: few rows, a long axis
        {"name": "attend_one", "op": "attend", "dtype": "bf16", "slots": 1, "ctx": 30000, "chunk": 1, "ragged": 0,
         "page": 16, "heads": 32, "kv_heads": 8, "head_dim": 128},
        # the smallest workload's verify chunk (8 drafts and the anchor) in binary32, a head per query head
        {"name": "attend_tiny_f32", "op": "attend", "dtype": "f32", "slots": 4, "ctx": 300, "chunk": 9, "ragged": 1,
         "page": 16, "heads": 8, "kv_heads": 8, "head_dim": 64},
        # the verify chunk of 32 requests with scheduled lengths (1 to 17 tokens)
        {"name": "attend_verify", "op": "attend", "dtype": "bf16", "slots": 32, "ctx": 2100, "chunk": 17, "ragged": 1,
         "page": 32, "heads": 32, "kv_heads": 8, "head_dim": 128},
        # the verify chunk of 256 requests, all 17 tokens
        {"name": "attend_verify_large", "op": "attend", "dtype": "bf16", "slots": 256, "ctx": 4096, "chunk": 17,
         "ragged": 0, "page": 64, "heads": 32, "kv_heads": 8, "head_dim": 128},
        # two prompts' prefill chunks over what they have cached: the matrix products bound it
        {"name": "attend_prefill", "op": "attend", "dtype": "bf16", "slots": 2, "ctx": 8192, "chunk": 2048,
         "ragged": 0, "page": 64, "heads": 32, "kv_heads": 8, "head_dim": 128},
    ]


def _spread(rng, low, high):
    """A whole number whose logarithm is uniform over [low, high]."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["rotate", "rotate", "store", "store", "read", "attend", "attend", "attend"])
    heads, kv_heads, head_dim = rng.choice([(32, 8, 128), (16, 16, 64), (8, 1, 128), (28, 4, 128), (16, 2, 256),
                                            (24, 8, 64), (64, 8, 128), (5, 5, 128)])
    page, dtype = rng.choice([16, 32, 64, 128]), rng.choice(["bf16", "bf16", "bf16", "f32"])
    kind = rng.choice(["one", "verify", "verify", "prefill"])
    if kind == "prefill":
        slots, chunk, most = rng.randrange(1, 5), _spread(rng, 64, 512), 8000
    else:
        slots, chunk = _spread(rng, 1, 200), 1 if kind == "one" else rng.randrange(2, 18)
        most = min(30000, 400_000 // slots)
    case = {"op": op, "dtype": dtype, "slots": slots, "ctx": _spread(rng, 1, most), "chunk": chunk,
            "ragged": rng.randrange(2), "page": page, "heads": heads, "kv_heads": kv_heads, "head_dim": head_dim}
    if op == "attend":
        if dtype == "f32":
            case["ctx"] = max(1, case["ctx"] // 4)
        return case
    if op == "read":
        pool = rng.choice(["4bit", "4bit", "bf16", "f32"])
        return {"op": op, "pool": pool, "dtype": dtype if pool == "4bit" else pool, "slots": slots,
                "ctx": _spread(rng, 1, min(20000, 120_000 // slots)), "page": page, "kv_heads": kv_heads,
                "head_dim": head_dim}
    return {**case, "rot": rng.choice([head_dim, head_dim, head_dim // 2, 16]), "interleaved": rng.random() < 0.3}


# ---------------------------------------------------------------------------
# sizes that follow from a case (the seed only permutes slots and pages)
# ---------------------------------------------------------------------------
def _lengths(case):
    """(cached tokens, chunk tokens) of every slot."""
    n, ctx, chunk = case["slots"], case["ctx"], case.get("chunk", 1)
    if n == 1:
        return [(ctx, chunk)]
    lens = [max(0, ctx * (n + 3 * i) // (4 * n - 3) - i % 3) for i in range(n)]
    return [(ln, 1 + (5 * i) % chunk if case.get("ragged") else chunk) for i, ln in enumerate(lens)]


def _token_bytes(case, kind):
    """Bytes of a token's keys and values as `kind` holds them."""
    n = 2 * case["kv_heads"] * case["head_dim"]
    return n * 17 // 32 if kind == "4bit" else n * _SIZE[kind]


def work(case):
    at = _lengths(case)
    if case["op"] == "read":
        cached = sum(ln for ln, _ in at)
        return {"bytes": cached * (_token_bytes(case, case["pool"]) + _token_bytes(case, case["dtype"])), "flops": 0}
    h, g, d = case["heads"], case["kv_heads"], case["head_dim"]
    new, query = sum(c for _, c in at), 2 * h * d * _SIZE[case["dtype"]]
    if case["op"] == "attend":
        return {"bytes": sum(ln + c for ln, c in at) * _token_bytes(case, "4bit") + new * query,
                "flops": sum(4 * h * d * (c * ln + c * (c + 1) // 2) for ln, c in at)}
    token = _token_bytes(case, case["dtype"])
    # into 4 bits: the chunk comes out as codes and, read back, as values
    moved = 2 * token if case["op"] == "rotate" else 2 * token + _token_bytes(case, "4bit")
    return {"bytes": new * (query + moved), "flops": new * (h + g) * case["rot"] * 3}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _gains(d):
    """Keys have a few dimensions that are much larger than the others."""
    return torch.where(torch.arange(d, device="cuda") % 16 == 5, 4.0, 1.0)


def _pool(case, kind, pages, gen):
    """One layer's pages, filled with keys and values."""
    d, page, heads = case["head_dim"], case["page"], case["kv_heads"]
    if kind != "4bit":
        e, dt = 16 // _SIZE[kind], _T[kind]
        return {"K": torch.randn((1, pages, heads, d // e, page, e), generator=gen, device="cuda", dtype=dt),
                "V": torch.randn((1, pages, heads, page // e, d, e), generator=gen, device="cuda", dtype=dt)}
    pool = {n: torch.empty((1, pages, heads * page * d * 17 // 32), dtype=torch.uint8, device="cuda") for n in "KV"}
    some = max(1, (1 << 26) // (heads * page * d))
    for p in range(0, pages, some):
        n = min(some, pages - p)
        for name in "KV":
            x = torch.randn((n, page, heads, d), generator=gen, device="cuda")
            codes, scales = _quantise(x * _gains(d) if name == "K" else x)
            pool[name][0, p:p + n] = _pack(name, codes, scales)
    return pool


def _pack(name, codes, scales):
    """Bytes of pages from codes [pages, page, heads, d] and scale bytes [pages, page, heads, d / 32]."""
    n, page, heads, d = codes.shape
    pairs = codes[..., 0::2] | codes[..., 1::2] << 4
    if name == "K":
        pairs = pairs.view(n, page, heads, d // 32, 16).permute(0, 2, 3, 1, 4)
    else:
        pairs = pairs.view(n, page // 8, 8, heads, 16, d // 64, 2).permute(0, 3, 1, 5, 4, 6, 2)
    return torch.cat([pairs.reshape(n, -1), scales.permute(0, 2, 3, 1).reshape(n, -1)], 1)


def _pack_bits(refs):
    """free_bits of reference counts."""
    n = refs.numel()
    free = torch.zeros(-(-n // 32) * 32, dtype=torch.int64)
    free[:n] = refs == 0
    words = (free.view(-1, 32) << torch.arange(32)).sum(1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def _tables(lens, rows, pages):
    """Cache tables in which slot s holds the listed pages."""
    table = torch.full((len(rows), max(len(r) for r in rows)), -1, dtype=torch.int32)
    for s, r in enumerate(rows):
        table[s, :len(r)] = r
    refs = torch.bincount(torch.cat(list(rows)), minlength=pages).to(torch.int32)
    held = torch.tensor([len(r) for r in rows], dtype=torch.int32)
    t = {"table": table, "lens": torch.tensor(lens, dtype=torch.int32), "held": held, "refs": refs,
         "free_bits": _pack_bits(refs), "n_free": (refs == 0).sum().to(torch.int32).view(1)}
    return {k: v.cuda() for k, v in t.items()}


def prepare(case, seed):
    gen = _generator(seed)
    cpu = torch.Generator()
    cpu.manual_seed(seed)
    op, page, slots = case["op"], case["page"], case["slots"]
    g, d = case["kv_heads"], case["head_dim"]
    at = _lengths(case)
    at = [at[i] for i in torch.randperm(len(at), generator=cpu).tolist()]
    counts = [max(1, -(-(ln + (c if op != "read" else 0)) // page)) for ln, c in at]
    # requests that append share the whole pages of a prompt; the others have their own
    common = [ln // page if op in ("rotate", "store") else 0 for ln, _ in at]
    mine = [n - m for n, m in zip(counts, common)]
    pages = max(common) + sum(mine) + 5
    order = torch.randperm(pages, generator=cpu).to(torch.int32)
    prompt, rest = order[:max(common)], order[max(common):max(common) + sum(mine)].split(mine)
    rows = [torch.cat([prompt[:m], r]) for m, r in zip(common, rest)]
    kind = case["pool"] if op == "read" else ("4bit" if op in ("store", "attend") else case["dtype"])
    state = {"op": op, "kind": kind, "page": page, "kv_heads": g, "head_dim": d,
             "tables": _tables([ln for ln, _ in at], rows, pages), **_pool(case, kind, pages, gen)}
    dt = _T[case["dtype"]]
    if own:
        from draft_sampling_verification_w1_amd import cache
        shape = {"shape": (page, g, d)} if kind == "4bit" else {}
        state["cache"] = cache.PagedCache.of(state["K"], state["V"], **state["tables"], **shape)
    if op == "read":
        n = sum(ln for ln, _ in at)
        state["offsets"] = torch.tensor([0] + [ln for ln, _ in at]).cumsum(0).to(torch.int32).cuda()
        state["first"] = torch.zeros(slots, dtype=torch.int32, device="cuda")
        state["out"] = tuple(torch.zeros((n, g, d), dtype=dt, device="cuda") for _ in range(2))
        return state
    n, heads = slots * case["chunk"], case["heads"]
    state["chunk"] = case["chunk"]
    state["offsets"] = torch.tensor([0] + [c for _, c in at]).cumsum(0).to(torch.int32).cuda()
    state["q"] = torch.randn((n, heads, d), generator=gen, device="cuda", dtype=dt).mul_(2)
    state["q_out"] = torch.zeros_like(state["q"])
    if op == "attend":
        if own:
            state["ws"] = state["cache"].attend_workspace(n, heads)
        return state
    state["k"] = (torch.randn((n, g, d), generator=gen, device="cuda") * _gains(d)).to(dt)
    state["v"] = torch.randn((n, g, d), generator=gen, device="cuda", dtype=dt)
    # what 4 bits stand for is a bf16 value
    state["out"] = tuple(torch.zeros((n, g, d), dtype=torch.bfloat16, device="cuda") for _ in range(2))
    # radians per position of each pair
    state["freqs"] = 1e6 ** (torch.arange(0, case["rot"], 2, device="cuda", dtype=torch.float64) / -case["rot"])
    state["interleaved"] = case["interleaved"]
    if own:
        state["rotation"] = cache.Rotation(state["freqs"], interleaved=case["interleaved"])
    return state


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------
def _chunk(t, off, n):
    """Token rows in use, their slots and positions."""
    i = torch.arange(n, device=off.device)
    tokens = torch.nonzero(i < off[-1]).view(-1)
    slot = torch.searchsorted(off, tokens, right=True) - 1
    return tokens, slot, t["lens"][slot].long() + tokens - off[slot]


def _rotate(x, pos, freqs, interleaved):
    """Rows x [n, heads, d] rotated by their positions, in binary32."""
    angle = (pos.double().view(-1, 1) * freqs).unsqueeze(1)
    c, s = angle.cos().float(), angle.sin().float()
    x, rot = x.float(), 2 * freqs.numel()
    if interleaved:
        a, b = x[..., :rot:2], x[..., 1:rot:2]
    else:
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
    a, b = a * c - b * s, b * c + a * s
    turned = torch.stack([a, b], -1).flatten(-2) if interleaved else torch.cat([a, b], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _quantise(x):
    """Codes and scale bytes of blocks of 32 elements: the scale is the smallest power of two of which the largest
    element is at most 7 (what saturates is then off by no more than what is rounded next to it)."""
    blocks = x.float().unflatten(-1, (-1, 32))
    m, e = torch.frexp(blocks.abs().amax(-1))  # largest = m 2^e, 0.5 <= m < 1
    e = torch.where(m > 0.875, e - 2, e - 3).masked_fill(m == 0, -120).clamp(-120, 125)
    y = torch.ldexp(blocks.abs(), -e.unsqueeze(-1))
    step = torch.where(y < 2, 0.5, torch.where(y < 4, 1.0, 2.0))
    y = (torch.round(y / step) * step).clamp(max=6)
    code = torch.where(y <= 2, 2 * y, torch.where(y < 6, y + 2, y + 1)).to(torch.uint8)
    return (code | (blocks < 0).to(torch.uint8) << 3).flatten(-2), (e + 127).to(torch.uint8)


def _values(s, name, pages):
    """Pages [...] of a pool as tokens [..., page, kv_heads, d] in binary32."""
    g, d, page, lead = s["kv_heads"], s["head_dim"], s["page"], tuple(pages.shape)
    raw = s[name][0][pages.long()]
    n = len(lead)
    if s["kind"] != "4bit":
        to = (n + 2, n, n + 1, n + 3) if name == "K" else (n + 1, n + 3, n, n + 2)
        return raw.permute(*range(n), *to).reshape(*lead, page, g, d).float()
    code = torch.arange(256, device=raw.device)
    code = torch.stack([code & 15, code >> 4], 1)
    pair = torch.tensor(_LEVELS, device=raw.device)[code & 7] * torch.where(code > 7, -1.0, 1.0)
    size = g * page * d // 2
    x = pair[raw[..., :size].long()]
    if name == "K":
        x = x.view(*lead, g, d // 32, page, 32).permute(*range(n), n + 2, n, n + 1, n + 3)
    else:
        x = x.view(*lead, g, page // 8, d // 64, 16, 2, 8, 2)
        x = x.permute(*range(n), n + 1, n + 5, n, n + 3, n + 2, n + 4, n + 6)
    x = x.reshape(*lead, page, g, d // 32, 32)
    scale = (raw[..., size:].to(torch.int32) << 23).view(torch.float32).view(*lead, g, d // 32, page)
    return (x * scale.permute(*range(n), n + 2, n, n + 1).unsqueeze(-1)).flatten(-2)


def _append(s):
    t, off, page = s["tables"], s["offsets"].long(), s["page"]
    tokens, slot, pos = _chunk(t, off, len(s["k"]))
    dt, g, d = s["q"].dtype, s["kv_heads"], s["head_dim"]
    s["q_out"][tokens] = _rotate(s["q"][tokens], pos, s["freqs"], s["interleaved"]).to(dt)
    k, v = _rotate(s["k"][tokens], pos, s["freqs"], s["interleaved"]), s["v"][tokens]
    to, row = t["table"][slot, pos // page].long(), pos % page
    if s["kind"] != "4bit":
        e = s["K"].shape[-1]
        s["K"][0][to, :, :, row, :] = k.to(dt).view(-1, g, d // e, e)
        s["V"][0][to, :, row // e, :, row % e] = v
        return {"q": s["q_out"], "K": s["K"], "V": s["V"]}
    size, h, b = g * page * d // 2, torch.arange(g, device=pos.device).view(1, -1, 1), torch.arange(d // 32, device=pos.device)
    for name, x in (("K", k), ("V", v)):
        codes, scales = _quantise(x)
        pairs = codes[..., 0::2] | codes[..., 1::2] << 4
        blobs = s[name][0]
        there, row_ = to.view(-1, 1, 1), row.view(-1, 1, 1)
        blobs[there, size + (h * (d // 32) + b) * page + row_] = scales
        i = torch.arange(d // 2, device=pos.device)
        if name == "K":
            at = ((h * (d // 32) + i // 16) * page + row_) * 16 + i % 16
        else:
            n, i = i // (d // 32), i % (d // 32)
            at = (((h * (page // 8) + row_ // 8) * (d // 64) + i // 2) * 16 + n) * 16 + i % 2 * 8 + row_ % 8
        blobs[there, at] = pairs
    for name, out in zip("KV", s["out"]):
        out[tokens] = _values(s, name, to)[torch.arange(len(to), device=to.device), row].to(out.dtype)
    return {"q": s["q_out"], "k": s["out"][0], "v": s["out"][1]}


def _read(s):
    t, off, page = s["tables"], s["offsets"].long(), s["page"]
    for name, out in zip("KV", s["out"]):
        x = _values(s, name, t["table"].clamp(min=0)).flatten(1, 2)
        there = torch.arange(x.shape[1], device=off.device) < off.diff().view(-1, 1)
        out.copy_(x[there])
    return {"k": s["out"][0], "v": s["out"][1]}


def _attend(s):
    t, page, off, q = s["tables"], s["page"], s["offsets"].long(), s["q"]
    n, heads, d = q.shape
    g = s["kv_heads"]
    slots, width = t["table"].shape
    pages = t["table"].clamp(min=0)
    total = t["lens"].long() + off.diff()
    key = torch.arange(width * page, device=q.device)
    kt = _values(s, "K", pages).flatten(1, 2).permute(0, 2, 3, 1).contiguous()
    vt = _values(s, "V", pages).flatten(1, 2).transpose(1, 2).contiguous()
    vt.masked_fill_((key >= total.view(-1, 1)).view(slots, 1, -1, 1), 0)
    c = torch.arange(s["chunk"], device=q.device)
    there = c < off.diff().view(-1, 1)
    at = (off[:-1].view(-1, 1) + c).clamp(max=n - 1)
    qp = q[at].float().view(slots, -1, g, heads // g, d).permute(0, 2, 1, 3, 4).reshape(slots, g, -1, d)
    p = torch.matmul(qp, kt).mul_(1 / math.sqrt(d)).view(slots, g, -1, heads // g, width * page)
    p.masked_fill_((key > (t["lens"].view(-1, 1) + c).unsqueeze(-1)).view(slots, 1, -1, 1, width * page), -math.inf)
    p.sub_(p.amax(-1, keepdim=True)).exp_()
    p.div_(p.sum(-1, keepdim=True))
    o = torch.matmul(p.view(slots, g, -1, width * page), vt).view(slots, g, -1, heads // g, d)
    o = o.permute(0, 2, 1, 3, 4).reshape(slots, -1, heads, d)
    s["q_out"][at[there]] = o[there].to(q.dtype)
    return s["q_out"]


def run(state):
    s, op = state, state["op"]
    if own:
        c = s["cache"]
        if op == "read":
            c.read(0, s["offsets"], first=s["first"], out=s["out"])
            return {"k": s["out"][0], "v": s["out"][1]}
        if op == "attend":
            return c.attend(0, s["q"], s["offsets"], max_chunk=s["chunk"], out=s["q_out"], ws=s["ws"])
        c.append(0, s["k"], s["v"], s["offsets"], rotation=s["rotation"], q=s["q"], q_out=s["q_out"])
        if op == "rotate":
            return {"q": s["q_out"], "K": s["K"], "V": s["V"]}
        c.read(0, s["offsets"], out=s["out"])
        return {"q": s["q_out"], "k": s["out"][0], "v": s["out"][1]}
    return {"read": _read, "attend": _attend}.get(op, _append)(s)


# ---------------------------------------------------------------------------
# the definitions in 64 bits, token by token position and byte by byte address
# ---------------------------------------------------------------------------
def _exact_tokens(s, name, slot, n):
    """Tokens 0 .. n - 1 of a slot as [n, kv_heads, d]."""
    g, d, page = s["kv_heads"], s["head_dim"], s["page"]
    p = torch.arange(n, device="cuda")
    pages, row = s["tables"]["table"][slot].long()[p // page], p % page
    pool = s[name][0]
    h, e = torch.arange(g, device="cuda").view(-1, 1), torch.arange(d, device="cuda")
    pages, row = pages.view(-1, 1, 1), row.view(-1, 1, 1)
    if s["kind"] != "4bit":
        w = pool.shape[-1]
        if name == "K":
            return pool[pages, h, e // w, row, e % w].double()
        return pool[pages, h, row // w, e, row % w].double()
    if name == "K":
        byte = ((h * (d // 32) + e // 32) * page + row) * 16 + e % 32 // 2
    else:
        n16, rest = e // (d // 16), e % (d // 16)
        byte = (((h * (page // 8) + row // 8) * (d // 64) + rest // 4) * 16 + n16) * 16 + rest % 4 // 2 * 8 + row % 8
    code = pool[pages, byte].to(torch.int64) >> e % 2 * 4 & 15
    exponent, low = code >> 1 & 3, (code & 1).double()
    size = torch.where(exponent == 0, low / 2, (1 + low / 2) * torch.exp2((exponent - 1).double()))
    scale = pool[pages, g * page * d // 2 + (h * (d // 32) + e // 32) * page + row].double() - 127
    return torch.where(code > 7, -size, size) * torch.exp2(scale)


def _exact_rotate(s, name, out):
    """Rows of q or k turned as complex numbers, for the tokens that belong to a slot."""
    x, rot = s[name].double(), 2 * s["freqs"].numel()
    off, lens = s["offsets"].tolist(), s["tables"]["lens"].tolist()
    at = torch.cat([torch.arange(ln, ln + b - a, device="cuda") for ln, a, b in zip(lens, off, off[1:])])
    x = x[:off[-1]]
    pairs = x[..., :rot].unflatten(-1, (-1, 2) if s["interleaved"] else (2, -1))
    if not s["interleaved"]:
        pairs = pairs.transpose(-1, -2)
    angle = at.double().view(-1, 1, 1) * s["freqs"]
    z = torch.complex(pairs[..., 0].contiguous(), pairs[..., 1].contiguous()) * torch.polar(torch.ones_like(angle), angle)
    z = torch.stack([z.real, z.imag], -1 if s["interleaved"] else -2).flatten(-2)
    out = out.double().clone()
    out[:off[-1]] = torch.cat([z, x[..., rot:]], -1)
    return out, at


def _exact_nearest(x):
    """The 4-bit values nearest to x [..., d]."""
    b = x.unflatten(-1, (-1, 32))
    top = b.abs().amax(-1, keepdim=True)
    scale = torch.exp2(torch.ceil(torch.log2(top / 7)).clamp(-120, 125)).where(top > 0, 1.0)
    scale = torch.where(top > 7 * scale, 2 * scale, torch.where(top <= 3.5 * scale, scale / 2, scale)).where(top > 0, 1.0)
    y, best = b.abs() / scale, torch.zeros_like(b)
    for low, high, even_low in zip(_LEVELS, _LEVELS[1:], (True, False) * 4):
        mid = (low + high) / 2
        best = torch.where(y >= mid if not even_low else y > mid, high, best)
    return (best * b.sign() * scale).flatten(-2)


def exact(case, seed):
    s = prepare(case, seed)
    g, d, off = s["kv_heads"], s["head_dim"], s["offsets"].tolist()
    if s["op"] == "read":
        every = {n: [_exact_tokens(s, n, i, b - a) for i, (a, b) in enumerate(zip(off, off[1:]))] for n in "KV"}
        return {"k": torch.cat(every["K"]), "v": torch.cat(every["V"])}
    if s["op"] in ("rotate", "store"):
        q, at = _exact_rotate(s, "q", s["q_out"])
        k, _ = _exact_rotate(s, "k", s["out"][0])
        if s["op"] == "store":
            v = s["out"][1].double().clone()
            v[:off[-1]] = _exact_nearest(s["v"][:off[-1]].double())
            k[:off[-1]] = _exact_nearest(k[:off[-1]])
            return {"q": q, "k": k, "v": v}
        K, e, page = s["K"].double(), s["K"].shape[-1], s["page"]
        slot = torch.cat([torch.full((b - a,), i, device="cuda") for i, (a, b) in enumerate(zip(off, off[1:]))])
        for c in range(d // e):
            K[0, s["tables"]["table"][slot, at // page].long(), :, c, at % page] = k[:off[-1], :, c * e:c * e + e]
        return {"q": q, "K": K, "V": None}
    n, heads, _ = s["q"].shape
    out = torch.zeros((n, heads, d), dtype=torch.float64, device="cuda")
    for slot, ln in enumerate(s["tables"]["lens"].tolist()):
        a, b = off[slot], off[slot + 1]
        keys, vals = (_exact_tokens(s, name, slot, ln + b - a) for name in "KV")
        last = ln + torch.arange(b - a, device="cuda").repeat_interleave(heads // g)
        hidden = torch.arange(ln + b - a, device="cuda") > last.view(-1, 1)
        for h in range(g):
            span = slice(h * (heads // g), (h + 1) * (heads // g))
            score = s["q"][a:b, span].double().reshape(-1, d) @ keys[:, h].t().contiguous() / math.sqrt(d)
            o = torch.softmax(score.masked_fill(hidden, -math.inf), -1) @ vals[:, h].contiguous()
            out[a:b, span] = o.view(b - a, heads // g, d)
    return out
