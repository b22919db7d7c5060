"""The cases that the 8-bit paged KV cache's operators are measured on: appending rotated keys and
values (read back as the values the cache then holds), attention over the cache, and attention with a
sliding window and sink tokens. `run` computes them in elementary torch operations, or through the
package where `own` is true."""

import math

import torch

own = False

BLOCK = 16                 # tokens that share one scale
FLOOR = 2.0 ** -60         # smallest scale
DTYPES = {"fp16": torch.float16, "bf16": torch.bfloat16}
TOP = {"int8": 127.0, "e4m3": 448.0}


# --------------------------------------------------------------------------- cases
def _append(name, seqs, new, past, heads, kv_heads, dim, dtype, fmt, page, rot=0, inter=False):
    """seqs sequences; each appends `new` tokens at most (ragged below it) after `past` at most."""
    return {"name": name, "op": "append", "seqs": seqs, "new": new, "past": past, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "format": fmt, "page": page, "rot": rot or dim, "interleaved": inter}


def _attend(name, seqs, new, past, heads, kv_heads, dim, dtype, fmt, page, window=0, sinks=0):
    return {"name": name, "op": "attend", "seqs": seqs, "new": new, "past": past, "heads": heads, "kv_heads": kv_heads,
            "dim": dim, "dtype": dtype, "format": fmt, "page": page, "window": window, "sinks": sinks}


def listed():
    return [
        # one token of one request joins the cache (Llama-3-8B's heads): latency
        _append("append_one", 1, 1, 1000, 32, 8, 128, "fp16", "int8", 64),
        # a decode batch: one token each, most blocks partly filled
        _append("append_decode_batch", 64, 1, 8000, 32, 8, 128, "bf16", "int8", 16),
        # ragged prompts of a batch, new sequences
        _append("append_prompts", 5, 2048, 0, 32, 8, 128, "fp16", "e4m3", 64),
        # the next chunk of two long prompts; small heads, part of each rotated in neighbouring pairs
        _append("append_chunk_small_heads", 2, 2049, 4099, 16, 16, 64, "bf16", "int8", 32, rot=32, inter=True),
        # one request's decode step: latency
        _attend("decode_one", 1, 1, 776, 32, 8, 128, "fp16", "int8", 64),
        # a decode batch of ragged requests
        _attend("decode_batch", 32, 1, 8191, 32, 8, 128, "bf16", "int8", 16),
        # two requests with long histories (Llama-3-70B's heads)
        _attend("decode_long", 2, 1, 131000, 64, 8, 128, "fp16", "e4m3", 64),
        # checking a few drafted tokens of each request, a key head for every query head
        _attend("decode_drafts_small_heads", 48, 5, 4001, 16, 16, 64, "fp16", "int8", 32),
        # a whole prompt
        _attend("prompt", 1, 2048, 0, 32, 8, 128, "fp16", "int8", 64),
        # chunks of prompts over their histories
        _attend("prompt_chunks", 3, 509, 6001, 64, 8, 128, "bf16", "e4m3", 64),
        # a decode batch whose layer sees the last 2048 tokens and the first 4
        _attend("window_decode_batch", 64, 1, 32767, 32, 8, 128, "bf16", "int8", 64, window=2048, sinks=4),
        # a whole prompt through such a layer
        _attend("window_prompt", 1, 4096, 0, 32, 8, 128, "fp16", "int8", 64, window=1024, sinks=4),
    ]


def _spread(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    dim = rng.choice((64, 128))
    kv_heads = rng.choice((1, 2, 4, 8) if dim == 128 else (2, 5, 8, 16))
    heads = kv_heads * rng.choice((1, 2, 3, 4, 7, 8))
    how = dict(heads=heads, kv_heads=kv_heads, dim=dim, dtype=rng.choice(("fp16", "bf16")),
               fmt=rng.choice(("int8", "e4m3")), page=rng.choice((16, 32, 48, 64, 128)))
    kind = rng.choice(("append_decode", "append", "decode", "decode", "drafts", "prompt", "window", "window_prompt"))
    if kind == "append_decode":
        c = _append("", _spread(rng, 1, 256), 1, _spread(rng, 1, 8000), **how)
    elif kind == "append":
        new = _spread(rng, 2, 4096)
        c = _append("", rng.randint(1, max(1, min(16, 4096 // new))), new, rng.choice((0, _spread(rng, 1, 4096))),
                    rot=rng.choice((dim, dim // 2)), inter=rng.random() < 0.5, **how)
    elif kind == "decode":
        past = _spread(rng, 1, 65536)
        c = _attend("", _spread(rng, 1, max(1, min(128, 200_000 // past))), 1, past, **how)
    elif kind == "drafts":
        past = _spread(rng, 1, 16384)
        c = _attend("", _spread(rng, 1, max(1, min(64, 100_000 // past))), rng.randint(2, 8), past, **how)
    elif kind == "prompt":
        new = _spread(rng, 9, 2048)
        c = _attend("", rng.randint(1, max(1, 2048 // new)), new, rng.choice((0, _spread(rng, 1, 2048))), **how)
    elif kind == "window":
        past = _spread(rng, 16, 32768)
        c = _attend("", _spread(rng, 1, max(1, min(64, 200_000 // past))), rng.choice((1, 1, 3)), past,
                    window=_spread(rng, 1, 4096), sinks=rng.choice((0, 1, 4, 33)), **how)
    else:
        c = _attend("", 1, _spread(rng, 9, 2048), rng.choice((0, _spread(rng, 1, 2048))),
                    window=_spread(rng, 1, 1024), sinks=rng.choice((0, 4, 17)), **how)
    del c["name"]
    return c


# --------------------------------------------------------------------------- inputs
def _lengths(case):
    """(new tokens, earlier tokens) of each sequence: the largest first, the others ragged below
    them. They go by the case alone, so that `work` knows them."""
    g = torch.Generator().manual_seed(977 + case["seqs"])
    n, new, past = case["seqs"], case["new"], case["past"]
    a = (new * (0.5 + 0.5 * torch.rand(n, generator=g, dtype=torch.float64))).round().long().clamp_(1, new)
    p = (past * torch.rand(n, generator=g, dtype=torch.float64)).round().long() if past else torch.zeros(n, dtype=torch.long)
    a[0], p[0] = new, past
    return a.tolist(), p.tolist()


def _encode(x, s, fmt):
    """The 8-bit codes of x over the scale s, as bytes (int8: offset by 128)."""
    t = x / s
    if fmt == "int8":
        return (t.round().clamp_(-127, 127) + 128).to(torch.uint8)
    return t.clamp(-448, 448).to(torch.float32).to(torch.float8_e4m3fn).view(torch.uint8)


def _decode(code, fmt, dtype=torch.float32):
    """The numbers that codes stand for, before their scale."""
    if fmt == "int8":
        return code.to(dtype) - 128
    return code.view(torch.float8_e4m3fn).to(dtype)


def _held(case, total_pages, gen, dev):
    """Pages of a cache as earlier steps left them: normal values, a few channels of the keys
    larger than the others, 16 tokens of a head to a scale."""
    page, hk, dim, fmt = case["page"], case["kv_heads"], case["dim"], case["format"]
    loud = torch.ones(hk, 1, dim, device=dev)
    loud[:, :, :: 17] = 3.0
    got = []
    for part in (loud, torch.full_like(loud, 0.5)):
        codes = torch.empty(total_pages, hk, page, dim, dtype=torch.uint8, device=dev)
        scales = torch.empty(total_pages, hk, page // BLOCK, device=dev)
        for at in range(0, total_pages, 1 + (1 << 26) // (hk * page * dim)):
            to = min(total_pages, at + 1 + (1 << 26) // (hk * page * dim))
            x = torch.randn(to - at, hk, page, dim, generator=gen, device=dev) * part
            x = x.view(to - at, hk, page // BLOCK, BLOCK, dim)
            s = x.abs().amax((3, 4), keepdim=True) / TOP[fmt]
            codes[at:to] = _encode(x, s, fmt).view(to - at, hk, page, dim)
            scales[at:to] = s.view(to - at, hk, page // BLOCK)
        got += [codes, scales]
    return got


def prepare(case, seed):
    dev = torch.device("cuda")
    gen = torch.Generator(dev).manual_seed(seed)
    new, past = _lengths(case)
    n, page, dim, dt = case["seqs"], case["page"], case["dim"], DTYPES[case["dtype"]]
    lens = [a + p for a, p in zip(new, past)]
    pages = [-(-m // page) for m in lens]
    spare = 3
    order = torch.randperm(sum(pages) + spare, generator=gen, device=dev).to(torch.int32)
    table = torch.zeros(n, max(pages), dtype=torch.int32, device=dev)
    at = 0
    for b, k in enumerate(pages):
        table[b, :k] = order[at:at + k]
        at += k
    state = {"case": dict(case), "table": table, "max_new": max(new), "max_len": max(lens)}
    state["k_pages"], state["k_scales"], state["v_pages"], state["v_scales"] = _held(case, sum(pages) + spare, gen, dev)
    state["lens"] = torch.tensor(lens, dtype=torch.int32, device=dev)
    state["indptr"] = torch.tensor([0] + new, device=dev).cumsum(0).to(torch.int32)
    tokens, hq, hk = sum(new), case["heads"], case["kv_heads"]
    if case["op"] == "append":
        # q, k and v as one product with their joined weights leaves them
        qkv = torch.randn(tokens, (hq + 2 * hk) * dim, generator=gen, device=dev)
        qkv[:, :: 23] *= 3.0
        state["qkv"] = qkv.to(dt)
        half = case["rot"] // 2
        f = 500000.0 ** (-torch.arange(half, device=dev, dtype=torch.float64) / half)
        a = torch.arange(max(lens), device=dev, dtype=torch.float64)[:, None] * f
        state["rope"] = torch.cat((a.cos(), a.sin()), 1).float()
        # what is read back: each sequence from the first block that it wrote to
        back = [m - p // BLOCK * BLOCK for m, p in zip(lens, past)]
        state["back"] = torch.tensor([0] + back, device=dev).cumsum(0).to(torch.int32)
        state["back_tokens"], state["max_back"] = sum(back), max(back)
    else:
        state["q"] = (1.5 * torch.randn(tokens, hq, dim, generator=gen, device=dev)).to(dt)
    return state


# --------------------------------------------------------------------------- plain forms
def _turn(x, cos, sin, inter):
    """x [T, heads, dim] with its first channels turned by the angles of cos, sin [T, half]."""
    half = cos.shape[1]
    c, s = cos[:, None], sin[:, None]
    head, rest = x[..., :2 * half], x[..., 2 * half:]
    a, b = (head[..., 0::2], head[..., 1::2]) if inter else (head[..., :half], head[..., half:])
    pair = (a * c - b * s, b * c + a * s)
    head = torch.stack(pair, -1).flatten(-2) if inter else torch.cat(pair, -1)
    return torch.cat((head, rest), -1)


def _owner(indptr, tokens):
    """The sequence of each token, and its place among that sequence's."""
    t = torch.arange(tokens, device=indptr.device)
    b = torch.searchsorted(indptr[1:].long(), t, right=True)
    return b, t - indptr.long()[b]


def _put(pages, scales, x, slot, first, fmt):
    """Tokens x [T, heads, dim] into the pages. slot: their (page, place in it, block of it, whether
    the block has earlier tokens of the sequence); first: for each sequence the same of its first
    block, with the count of its earlier tokens."""
    page, off, blk, older = slot
    nb = scales.shape[2]
    top = torch.zeros(scales.shape[0] * nb, x.shape[1], dtype=x.dtype, device=x.device)
    key = page * nb + blk
    top.scatter_reduce_(0, key[:, None].expand(-1, x.shape[1]), x.abs().amax(-1), "amax")
    was = scales[page, :, blk]
    s = torch.maximum((top[key] / TOP[fmt]).float().clamp_min(FLOOR), torch.where(older[:, None], was, 0.0))
    fpage, fblk, kept = first
    at = (fblk * BLOCK)[:, None] + torch.arange(BLOCK, device=x.device)
    codes = pages[fpage[:, None], :, at]
    was = scales[fpage, :, fblk]
    scales[page, :, blk] = s
    now = torch.where(kept[:, None] > 0, scales[fpage, :, fblk], was)
    again = _encode(_decode(codes, fmt, torch.float64) * was[:, None, :, None].double(), now[:, None, :, None].double(), fmt)
    keep = (torch.arange(BLOCK, device=x.device)[None] < kept[:, None])[:, :, None, None]
    pages[fpage[:, None], :, at] = torch.where(keep, again, codes)
    pages[page, :, off] = _encode(x, s[..., None].double(), fmt)


def _plain_append(s):
    c, page = s["case"], s["case"]["page"]
    tokens, hq, hk, dim = s["qkv"].shape[0], c["heads"], c["kv_heads"], c["dim"]
    q, k, v = s["qkv"].view(tokens, hq + 2 * hk, dim).split((hq, hk, hk), 1)
    b, i = _owner(s["indptr"], tokens)
    lens, n = s["lens"].long(), s["indptr"].long().diff()
    past = lens - n
    pos = past[b] + i
    cos, sin = s["rope"][pos].double().chunk(2, 1)
    table = s["table"].long()
    slot = (table[b, pos // page], pos % page, pos % page // BLOCK, past[b] > pos // BLOCK * BLOCK)
    start = past // BLOCK * BLOCK
    start_page = table.gather(1, (start // page).clamp_max(table.shape[1] - 1)[:, None])[:, 0]
    first = (start_page, start % page // BLOCK, past - start)
    _put(s["k_pages"], s["k_scales"], _turn(k.double(), cos, sin, c["interleaved"]), slot, first, c["format"])
    _put(s["v_pages"], s["v_scales"], v.double(), slot, first, c["format"])
    rb, ri = _owner(s["back"], s["back_tokens"])
    at = start[rb] + ri
    pg, off = table[rb, at // page], at % page
    values = [(_decode(p[pg, :, off], c["format"]) * f[pg, :, off // BLOCK][..., None]).to(q.dtype)
              for p, f in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"]))]
    return {"q": _turn(q.double(), cos, sin, c["interleaved"]).to(q.dtype), "k": values[0], "v": values[1]}


def _plain_attend(s):
    c, page, fmt = s["case"], s["case"]["page"], s["case"]["format"]
    hq, hk, dim, n = c["heads"], c["kv_heads"], c["dim"], c["seqs"]
    tokens, most, window, sinks = s["q"].shape[0], s["max_new"], c["window"], c["sinks"]
    dev = s["q"].device
    lens, indptr = s["lens"].long(), s["indptr"].long()
    past = lens - indptr.diff()
    # the positions that some query of the sequence may see: all, or the window's and the sinks
    if window and sinks + window + most < s["max_len"]:
        begin = (past - window + 1).clamp_min(sinks)
        pos = torch.cat((torch.arange(sinks, device=dev).expand(n, -1), begin[:, None] + torch.arange(window + most, device=dev)), 1)
    else:
        pos = torch.arange(s["max_len"], device=dev).expand(n, -1)
    there = pos < lens[:, None]
    pos = torch.where(there, pos, 0)
    pg = s["table"].long().gather(1, pos // page)
    off = pos % page
    k, v = (_decode(p[pg, :, off], fmt) * f[pg, :, off // BLOCK][..., None]
            for p, f in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])))
    i = torch.arange(most, device=dev)
    q = s["q"][(indptr[:-1, None] + i).clamp_max(tokens - 1)].float()                       # [n, most, hq, dim]
    q = q.view(n, most, hk, hq // hk, dim).permute(0, 2, 3, 1, 4).reshape(n, hk, -1, dim)
    score = torch.matmul(q, k.permute(0, 2, 3, 1)) * dim ** -0.5
    at = past[:, None, None] + i[None, :, None]                                             # [n, most, 1]
    see = there[:, None] & (pos[:, None] <= at)
    if window:
        see = see & ((pos[:, None] > at - window) | (pos[:, None] < sinks))
    score = score.view(n, hk, hq // hk, most, -1).masked_fill(~see[:, None, None], -math.inf)
    score = score - score.amax(-1, keepdim=True).clamp_min(-1e30)
    p = score.exp()
    total = p.sum(-1, keepdim=True)
    p = (p / torch.where(total > 0, total, 1.0)).view(n, hk, -1, p.shape[-1])
    y = torch.matmul(p, v.permute(0, 2, 1, 3)).view(n, hq, most, dim)
    b, j = _owner(s["indptr"], tokens)
    return y[b, :, j].to(s["q"].dtype)


# --------------------------------------------------------------------------- one pass
def run(state):
    c = state["case"]
    if not own:
        return _plain_append(state) if c["op"] == "append" else _plain_attend(state)
    import weight_only_int4_gemv_b200 as awq
    if "cache" not in state:   # the handles that a program keeps for a layer's cache and a batch
        state["cache"] = awq.KvCache(state["k_pages"], state["v_pages"], state["k_scales"], state["v_scales"], c["format"])
        state["batch"] = awq.KvBatch(state["table"], state["lens"], state["indptr"], state["max_new"])
        if c["op"] == "append":
            state["behind"] = awq.KvBatch(state["table"], state["lens"], state["back"], state["max_back"])
    cache, batch = state["cache"], state["batch"]
    if c["op"] == "attend":
        return awq.awq_kv_attention(state["q"], cache, batch, window=c["window"], sinks=c["sinks"])
    hq, hk, dim = c["heads"], c["kv_heads"], c["dim"]
    q, k, v = state["qkv"].view(-1, hq + 2 * hk, dim).split((hq, hk, hk), 1)
    q = awq.awq_kv_append(k, v, cache, batch, q=q, rope=state["rope"], interleaved=c["interleaved"])
    k, v = awq.awq_kv_dequant(cache, state["behind"], state["back_tokens"], q.dtype)
    return {"q": q, "k": k, "v": v}


def _visible(case):
    """(query, key) pairs that attention computes, and keys of all sequences that some query sees."""
    pairs = keys = 0
    w, sinks = case["window"], case["sinks"]
    for a, p in zip(*_lengths(case)):
        for m in ((p + i + 1) for i in range(a)):
            pairs += m if not w else min(m, w + min(sinks, max(0, m - w)))
        low = max(0, p - w + 1) if w else 0
        keys += a + p - max(0, low - sinks)
    return pairs, keys


def work(case):
    new, past = _lengths(case)
    tokens, hq, hk, dim = sum(new), case["heads"], case["kv_heads"], case["dim"]
    scales = 2 * hk * 4 / BLOCK                      # bytes a token, keys and values
    if case["op"] == "append":
        back = sum(a + p % BLOCK for a, p in zip(new, past))
        held = 2 * hk * dim * (back + back - tokens) + scales * back     # codes written, the older ones read too
        return {"bytes": tokens * dim * 2 * (2 * hq + 2 * hk) + tokens * case["rot"] * 4 + held + back * 2 * hk * dim * 2,
                "flops": 6 * tokens * (hq + hk) * case["rot"] // 2 + 8 * back * hk * dim}
    pairs, keys = _visible(case)
    return {"bytes": 2 * tokens * hq * dim * 2 + keys * (2 * hk * dim + scales), "flops": 4 * pairs * hq * dim}


# --------------------------------------------------------------------------- the definition in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    new, past = _lengths(case)
    f64, page, fmt, hk, dim = torch.float64, case["page"], case["format"], case["kv_heads"], case["dim"]
    group = case["heads"] // hk

    def row(b, lo, hi):
        """Keys and values (numbers, scales) of positions lo .. hi of a sequence: [heads, count, dim]."""
        ids = s["table"][b, lo // page:-(-hi // page)].long()
        cut = slice(lo - lo // page * page, hi - lo // page * page)
        got = []
        for p, f in ((s["k_pages"], s["k_scales"]), (s["v_pages"], s["v_scales"])):
            codes = p[ids].transpose(0, 1).reshape(hk, -1, dim)[:, cut]
            number = codes.to(f64) - 128 if fmt == "int8" else codes.view(torch.float8_e4m3fn).to(f64)
            got.append((number, f[ids].transpose(0, 1).reshape(hk, -1).repeat_interleave(BLOCK, 1)[:, cut].to(f64)))
        return got

    if case["op"] == "attend":
        outs, at = [], 0
        for b, (a, p) in enumerate(zip(new, past)):
            lo = max(0, p - case["window"] + 1) if case["window"] else 0
            (k, ks), (v, vs) = row(b, 0, a + p)
            seen = torch.ones(a + p, dtype=torch.bool, device=k.device)
            if case["window"]:
                seen[min(case["sinks"], lo):lo] = False
            j = seen.nonzero()[:, 0]
            q = s["q"][at:at + a].to(f64)
            at += a
            qp = torch.arange(p, p + a, device=k.device)[:, None]
            hide = j[None] > qp
            if case["window"]:
                hide |= (j[None] <= qp - case["window"]) & (j[None] >= case["sinks"])
            y = torch.zeros(a, hk * group, dim, dtype=f64, device=k.device)
            for h in range(hk):
                kh, vh = k[h, j] * ks[h, j, None], v[h, j] * vs[h, j, None]
                for g in range(h * group, (h + 1) * group):
                    z = (q[:, g] @ kh.T / math.sqrt(dim)).masked_fill(hide, -math.inf)
                    y[:, g] = torch.softmax(z, 1) @ vh
            outs.append(y)
        return torch.cat(outs)

    tokens, hq = sum(new), case["heads"]
    x = s["qkv"].view(tokens, hq + 2 * hk, dim).to(f64)
    half = case["rot"] // 2
    every = torch.cat([torch.arange(p, p + a) for a, p in zip(new, past)]).to(x.device)
    turn = torch.complex(s["rope"][every, :half].to(f64), s["rope"][every, half:].to(f64))[:, None]
    lead = torch.arange(half, device=x.device) * (2 if case["interleaved"] else 1)
    mate = lead + (1 if case["interleaved"] else half)
    turned = x[:, :hq + hk].clone()
    z = torch.complex(turned[..., lead], turned[..., mate]) * turn
    turned[..., lead], turned[..., mate] = z.real, z.imag
    fresh = (turned[:, hq:], x[:, hq + hk:])
    back, at = ([], []), 0
    top = 127.0 if fmt == "int8" else 448.0
    for b, (a, p) in enumerate(zip(new, past)):
        start = p // BLOCK * BLOCK
        older = row(b, start, p) if p > start else None
        for w in (0, 1):
            add = fresh[w][at:at + a].transpose(0, 1)
            pad = -(a + p - start) % BLOCK
            grid = torch.cat((torch.zeros(hk, p - start, dim, dtype=f64, device=x.device), add,
                              torch.zeros(hk, pad, dim, dtype=f64, device=x.device)), 1).view(hk, -1, BLOCK, dim)
            scale = (grid.abs().amax((2, 3)) / top).float().clamp_min(2.0 ** -60)
            if older is not None:
                scale[:, 0] = torch.maximum(scale[:, 0], older[w][1][:, 0].float())
                grid.view(hk, -1, dim)[:, :p - start] = older[w][0] * older[w][1][..., None]
            scale = scale.to(f64)[..., None, None]
            t = grid / scale
            t = t.round() if fmt == "int8" else t.float().to(torch.float8_e4m3fn).to(f64)
            back[w].append((t * scale).view(hk, -1, dim)[:, :a + p - start].transpose(0, 1))
        at += a
    return {"q": turned[:, :hq], "k": torch.cat(back[0]), "v": torch.cat(back[1])}
