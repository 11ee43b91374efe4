"""Cases that measure the 4-bit paged KV cache and what feeds it: the per-head norm with
the position rotation, the quantised write and read-back of the cache, and the attention
over it.

`run` computes an operator in its plain form (elementary torch operations, fp32, rounded
once at the end) or, where `own` is true, through the framework's entry points.  Both take
the same state: the packed pages as they lie in device memory, and bf16 rows.
"""
import math
import random

import torch

own = False

DEV = "cuda"
THETA = 500000.0      # the rotary base of the repository's workloads
LIMIT = 61440.0       # magnitudes above this are stored as this

# ---------------------------------------------------------------- cases


def listed():
    return [
        # one sequence decodes one token: q and k of the new position, nothing but latency
        dict(name="norm_rope 1 token", op="norm_rope", tokens=1, hq=32, hk=8, d=128, rot=128, axes=1, inter=False),
        # image and video prompts: three position axes, partial rotation of interleaved pairs, odd length
        dict(name="norm_rope 3 axes odd", op="norm_rope", tokens=1237, hq=28, hk=4, d=128, rot=96, axes=3, inter=True),
        # the prefill of a batch of 4096-token prompts
        dict(name="norm_rope prefill", op="norm_rope", tokens=16384, hq=32, hk=8, d=128, rot=128, axes=1, inter=False),
        # one decode step of 16 sequences from the qkv projection: norm, rotate, quantise, write
        dict(name="append_qkv decode", op="append_qkv", batch=16, t=1, ragged=False, ctx=8192, hq=32, hk=8, d=128, page=64, axes=1),
        # a chunk of ragged prompts from the qkv projection, positions on three axes
        dict(name="append_qkv ragged", op="append_qkv", batch=5, t=1531, ragged=True, ctx=4096, hq=28, hk=4, d=128, page=16, axes=3),
        # a prefilled batch whose keys are already rotated enters the cache
        dict(name="append prefill", op="append", batch=4, t=4096, ragged=False, ctx=4096, hq=32, hk=8, d=128, page=64, axes=1),
        # a short shared prefix is read back as bf16 rows
        dict(name="read ragged d64", op="read", batch=3, t=517, ragged=True, ctx=777, hq=16, hk=4, d=64, page=32, axes=1),
        # a long document's cache read back
        dict(name="read long", op="read", batch=2, t=32768, ragged=False, ctx=32768, hq=32, hk=8, d=128, page=128, axes=1),
        # one short conversation decodes one token
        dict(name="attention short", op="attention", batch=1, t=1, ragged=False, ctx=777, hq=32, hk=8, d=128, page=16, axes=1),
        # sixteen 32K contexts decode one token each
        dict(name="attention decode 32k", op="attention", batch=16, t=1, ragged=False, ctx=32768, hq=32, hk=8, d=128, page=64, axes=1),
        # drafted tokens of ragged sequences are verified at once
        dict(name="attention verify", op="attention", batch=8, t=5, ragged=True, ctx=8192, hq=28, hk=4, d=128, page=32, axes=1),
        # a chunk of new tokens behind a cached context
        dict(name="attention chunk", op="attention", batch=2, t=1024, ragged=False, ctx=8192, hq=32, hk=8, d=128, page=64, axes=1),
    ]


def _between(rng, a, b):
    """A whole number between a and b, spread over its logarithm."""
    return min(b, max(a, int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))))


def draw(rng):
    op = rng.choice(["norm_rope", "append_qkv", "append", "read", "attention", "attention"])
    d = rng.choice([64, 128, 128])
    hk = rng.choice([1, 2, 4, 8])
    g = rng.choice([g for g in (1, 3, 4, 7, 8) if g * hk <= 32])
    axes = rng.choice([1, 1, 3])
    if op == "norm_rope":
        rot = rng.choice([d, d, d // 2, d - 16])
        return dict(op=op, tokens=_between(rng, 1, 12000), hq=hk * g, hk=hk, d=d, rot=rot, axes=axes, inter=rng.random() < 0.5)
    page = rng.choice([16, 32, 64, 128])
    batch = _between(rng, 1, 16)
    ragged = rng.random() < 0.6
    if op == "attention":
        if rng.random() < 0.5:
            t, ctx = rng.randint(1, 8), _between(rng, 16, 16384)
        else:
            t, batch = _between(rng, 9, 1024), min(batch, 2)
            ctx = t + _between(rng, 1, 6000)
        ctx = max(ctx, t)
        return dict(op=op, batch=batch, t=t, ragged=ragged, ctx=ctx, hq=hk * g, hk=hk, d=d, page=page, axes=1)
    t = _between(rng, 1, max(1, 12000 // batch))
    ctx = t + _between(rng, 1, 4096)
    return dict(op=op, batch=batch, t=t, ragged=ragged, ctx=ctx, hq=hk * g, hk=hk, d=d, page=page, axes=axes)


# ---------------------------------------------------------------- inputs

def _inv_freq(rot):
    return torch.tensor([THETA ** (-2.0 * i / rot) for i in range(rot // 2)], dtype=torch.float32)


def _axis_of_pair(rot, axes):
    """Which position axis turns pair i: with three axes a quarter of the pairs follow the
    first (time) and the others split into the second and third (height, width)."""
    n = rot // 2
    if axes == 1:
        return [0] * n
    a = n // 4
    b = a + (n - a) // 2
    return [0 if i < a else 1 if i < b else 2 for i in range(n)]


def _positions(gen, case, last):
    """int32 [axes][tokens]; `last`: the position of each token in its sequence."""
    if case["axes"] == 1:
        return last.to(torch.int32)[None].contiguous()
    hw = torch.randint(0, 96, (2, last.numel()), generator=gen, device=DEV)
    return torch.cat([last[None], hw + last[None] // 2]).to(torch.int32).contiguous()


def _rows(gen, tokens, heads, d):
    """bf16 [tokens][heads][d]: normal, a few outlier channels in every head."""
    gain = torch.ones(heads, d, device=DEV)
    gain.scatter_(1, torch.randint(0, d, (heads, 4), generator=gen, device=DEV), 6.0)
    x = torch.randn(tokens, heads, d, generator=gen, device=DEV)
    return (x * gain).to(torch.bfloat16)


def _lengths(case):
    """(new tokens, cached tokens behind the call) of each sequence, from the case alone."""
    b, t, c = case["batch"], case["t"], case["ctx"]
    if not case["ragged"]:
        return [t] * b, [c] * b
    rng = random.Random(b * 1000003 + t * 1009 + c)
    fresh = [t] + [rng.randint(1, t) for _ in range(b - 1)]
    cached = [rng.randint(max(1, c // 2), c) for _ in range(b - 1)] + [c]
    return fresh, [max(x, y) for x, y in zip(fresh, cached)]


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(seed)
    op, hq, hk, d = case["op"], case["hq"], case["hk"], case["d"]
    s = dict(case=dict(case))
    if op == "norm_rope":
        n, rot = case["tokens"], case["rot"]
        first = torch.randint(0, 100000, (1,), generator=gen, device=DEV)
        s.update(qkv=_rows(gen, n, hq + 2 * hk, d), positions=_positions(gen, case, first + torch.arange(n, device=DEV)))
    else:
        rot = d
        fresh, cached = _lengths(case)
        t, c = torch.tensor(fresh, device=DEV), torch.tensor(cached, device=DEV)
        page = case["page"]
        per = -(-case["ctx"] // page)
        n_pages = case["batch"] * per + 3
        table = torch.randperm(n_pages, generator=gen, device=DEV)[: case["batch"] * per].to(torch.int32)
        start = torch.zeros(case["batch"] + 1, dtype=torch.int32, device=DEV)
        start[1:] = torch.cumsum(t, 0)
        n = sum(fresh)
        s.update(q_start=start, kv_len=c.to(torch.int32), page_table=table.view(case["batch"], per).contiguous(),
                 tokens=n, max_q=max(fresh), max_kv=max(cached), n_pages=n_pages,
                 # the pages, and behind them a line for the cache's error word
                 buffer=torch.zeros(n_pages * hk * page * 20 * d // 16 + 256, dtype=torch.uint8, device=DEV))
        if op in ("read", "attention"):
            # every cached token was written from such rows
            whole = dict(s, q_start=torch.cat([start[:1], torch.cumsum(c, 0)]).to(torch.int32), tokens=sum(cached))
            step = 1 << 17
            for i in range(0, whole["tokens"], step):
                m = min(step, whole["tokens"] - i)
                _write(whole, _rows(gen, m, hk, d), _rows(gen, m, hk, d), i)
            s["q"] = _rows(gen, n, hq, d)
        else:
            s.update(qkv=_rows(gen, n, hq + 2 * hk, d))
        if op == "append_qkv":
            _, where = _places(s, 0, n)
            s["positions"] = _positions(gen, case, where)
    if op in ("norm_rope", "append_qkv"):
        s.update(q_weight=(1 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(torch.bfloat16),
                 k_weight=(1 + 0.2 * torch.randn(d, generator=gen, device=DEV)).to(torch.bfloat16),
                 eps=1e-6, rot=rot, inv_freq=_inv_freq(rot), axis=_axis_of_pair(rot, case["axes"]),
                 inter=bool(case.get("inter", False)))
    return s


# ---------------------------------------------------------------- the plain forms

def _places(s, first, count):
    """(sequence, position in it) of the packed token rows [first, first + count)."""
    row = torch.arange(first, first + count, device=DEV)
    b = torch.searchsorted(s["q_start"][1:].long(), row, right=True)
    fresh = s["q_start"].long().diff()
    return b, s["kv_len"].long()[b] - fresh[b] + row - s["q_start"].long()[b]


def _pages(s):
    """The page bytes as [blocks of 16 tokens of one page and head][bytes]; page-major."""
    d = s["case"]["d"]
    return s["buffer"][:-256].view(-1, 20 * d)


def _blocks(s, b, pos):
    """(block, token in it) per head of position pos of sequence b: [tokens][heads], [tokens]."""
    hk, page = s["case"]["hk"], s["case"]["page"]
    p = s["page_table"].long()[b, pos // page]
    inside = pos % page
    head = torch.arange(hk, device=DEV)
    return (p[..., None] * hk + head) * (page // 16) + (inside // 16)[..., None], inside % 16


def _quantise(x):
    """fp32 [..., d] -> codes uint8 [..., d/32, 32], scale and zero fp16 [..., d/32]."""
    x = torch.nan_to_num(x, nan=0.0).clamp(-LIMIT, LIMIT).unflatten(-1, (-1, 32))
    lo, hi = x.amin(-1), x.amax(-1)
    scale, zero = ((hi - lo) / 15).half(), lo.half()
    y = (x.double() - zero.double()[..., None]) / scale.double().clamp_min(2.0 ** -24)[..., None]
    code = torch.where(scale[..., None] > 0, y.round().clamp(0, 15), 0)
    return code.to(torch.uint8), scale, zero


def _flip(tok, d):
    """Value rows of 64 bytes keep their 8-byte pieces crossed in every other token pair."""
    return ((tok >> 1) & 1) * 4 if d == 128 else torch.zeros_like(tok)


def _pack(code, scale, zero, tok, value):
    """One side of a token's row: (code bytes [tokens][heads][d/2], scale bytes)."""
    d = code.shape[-2] * 32
    if value:  # piece gq of 2 d/32 bytes: four channels of every group
        n = code.unflatten(-1, (8, 4)).transpose(-3, -2)                        # [gq][group][4]
        at = torch.arange(8, device=DEV) ^ _flip(tok, d)[:, None]
        n = n.gather(2, at[:, None, :, None, None].expand_as(n))
    else:      # piece tq of 4 d/32 bytes: eight channels of every group
        n = code.unflatten(-1, (4, 8)).transpose(-3, -2)
    n = n.reshape(*code.shape[:-2], d)
    return n[..., 0::2] | (n[..., 1::2] << 4), torch.stack([scale, zero], -1).flatten(-2).contiguous().view(torch.uint8)


def _write(s, k, v, first=0):
    """Quantises rows k, v [tokens][heads][d] into the places of the packed rows from `first` on."""
    d = s["case"]["d"]
    block, tok = _blocks(s, *_places(s, first, k.shape[0]))
    pages = _pages(s)
    base = (block * (20 * d))[..., None]
    at = 0
    for x, value in ((k, False), (v, True)):
        codes, scales = _pack(*_quantise(x.float()), tok, value)
        pages.view(-1)[base + at + (tok * (d // 2))[:, None, None] + torch.arange(d // 2, device=DEV)] = codes
        at += 8 * d
        pages.view(-1)[base + at + (tok * (d // 8))[:, None, None] + torch.arange(d // 8, device=DEV)] = scales
        at += 2 * d


def _fetch(s, b, pos):
    """(k, v) fp32 [..., heads, d] of positions pos of sequences b."""
    d = s["case"]["d"]
    block, tok = _blocks(s, b, pos)
    rows = _pages(s).view(-1, 20, d)
    got = []
    for value in (False, True):
        at = 10 if value else 0
        codes = rows[:, at:at + 8].reshape(-1, 16, d // 2)[block, tok[..., None]]
        sz = rows[:, at + 8:at + 10].reshape(-1, 16, d // 8)[block, tok[..., None]].view(torch.float16).float()
        n = torch.stack([codes & 15, codes >> 4], -1).flatten(-2)
        if value:
            n = n.unflatten(-1, (8, d // 32, 4))
            piece = torch.arange(8, device=DEV) ^ _flip(tok, d)[..., None]
            n = n.gather(-3, piece[..., None, :, None, None].expand_as(n))
        else:
            n = n.unflatten(-1, (4, d // 32, 8))
        n = n.transpose(-3, -2).flatten(-2).float()                              # [group][32]
        got.append((n * sz[..., 0::2, None] + sz[..., 1::2, None]).flatten(-2))
    return got


def _norm_rope(s, x, weight):
    x = x.float()
    x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + s["eps"]) * weight.float()
    rot, inter = s["rot"], s["inter"]
    pos = s["positions"][torch.tensor(s["axis"], device=DEV)].double().T           # [tokens][pairs]
    angle = pos * s["inv_freq"].to(DEV).double()
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]
    r = x[..., :rot]
    a, b = (r[..., 0::2], r[..., 1::2]) if inter else (r[..., : rot // 2], r[..., rot // 2:])
    a, b = a * cos - b * sin, b * cos + a * sin
    r = torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)
    return torch.cat([r, x[..., rot:]], -1).to(torch.bfloat16)


def _attention(s):
    """Causal attention of the packed query rows over every sequence's pages."""
    case = s["case"]
    hq, hk, d, g = case["hq"], case["hk"], case["d"], case["hq"] // case["hk"]
    nb, tm, cm = case["batch"], s["max_q"], s["max_kv"]
    start, ln = s["q_start"].long(), s["kv_len"].long()
    fresh = start.diff()
    seq = torch.arange(nb, device=DEV)[:, None]
    pos = torch.arange(cm, device=DEV)[None].expand(nb, cm)
    k, v = _fetch(s, seq.expand(nb, cm), torch.minimum(pos, ln[:, None] - 1))
    j = torch.arange(tm, device=DEV)[None]
    q = s["q"][torch.minimum(start[:-1, None] + j, start[1:, None] - 1)].float()  # [b][t][hq][d]
    q = q.view(nb, tm, hk, g, d).permute(0, 2, 3, 1, 4).reshape(nb, hk, g * tm, d)
    logit = q @ k.permute(0, 2, 3, 1) / math.sqrt(d)
    seen = (ln - fresh)[:, None] + j + 1                                           # tokens that query j sees
    hidden = pos[:, None] >= seen[..., None]
    logit = logit.view(nb, hk, g, tm, cm).masked_fill_(hidden[:, None, None], -math.inf)
    p = torch.exp(logit - logit.amax(-1, keepdim=True))
    p = (p / p.sum(-1, keepdim=True)).view(nb, hk, g * tm, cm)
    o = (p @ v.permute(0, 2, 1, 3)).view(nb, hk, g, tm, d).permute(0, 3, 1, 2, 4).reshape(nb, tm, hq, d)
    row = torch.arange(s["tokens"], device=DEV)
    b = torch.searchsorted(start[1:], row, right=True)
    return o[b, row - start[b]].to(torch.bfloat16)


def _plain(s):
    case = s["case"]
    op, hq, hk = case["op"], case["hq"], case["hk"]
    if op == "attention":
        return _attention(s)
    if op == "read":
        return [x.to(torch.bfloat16) for x in _fetch(s, *_places(s, 0, s["tokens"]))]
    q, k, v = s["qkv"].split([hq, hk, hk], 1)
    if op == "append":
        _write(s, k, v)
        return [x.to(torch.bfloat16) for x in _fetch(s, *_places(s, 0, s["tokens"]))]
    q, k = _norm_rope(s, q, s["q_weight"]), _norm_rope(s, k, s["k_weight"])
    if op == "norm_rope":
        return q, k
    _write(s, k, v)
    return [q, *(x.to(torch.bfloat16) for x in _fetch(s, *_places(s, 0, s["tokens"])))]


# ---------------------------------------------------------------- the framework's calls

def _handles(s):
    """The rotation, the cache and the batch that a user's program makes once and keeps."""
    if "rope" not in s:
        import decode_attention_prefill_b200 as pm
        case = s["case"]
        s["pm"] = pm
        s["rope"] = pm.Rope.make(case["d"], inv_freq=s["inv_freq"].tolist(), axes=s["axis"], interleaved=s["inter"],
                                 eps=s["eps"]) if "inv_freq" in s else None
        if "buffer" in s:
            cfg = pm.KV4Config.make(case["hq"], case["hk"], case["d"], page_tokens=case["page"])
            s["cache"] = pm.KV4Cache(cfg, s["n_pages"], buffer=s["buffer"])
            s["batch"] = pm.KV4Batch(s["kv_len"], s["page_table"], s["q_start"], n_tokens=s["tokens"],
                                     max_q=s["max_q"])
    return s["pm"], s["rope"], s.get("cache"), s.get("batch")


def _own(s):
    pm, rope, cache, batch = _handles(s)
    case = s["case"]
    op, hq, hk = case["op"], case["hq"], case["hk"]
    if op == "attention":
        return cache.attend(batch, s["q"])
    if op == "read":
        return cache.read(batch)
    q, k, v = s["qkv"].split([hq, hk, hk], 1)
    if op == "norm_rope":
        return pm.norm_rope(rope, q, k, s["positions"], s["q_weight"], s["k_weight"])
    if op == "append":
        cache.append(batch, k, v)
        return cache.read(batch)
    q = cache.append_qkv(batch, rope, q, k, v, s["positions"], s["q_weight"], s["k_weight"])
    return [q, *cache.read(batch)]


def run(state):
    return _own(state) if own else _plain(state)


# ---------------------------------------------------------------- floors

def work(case):
    op, hq, hk, d = case["op"], case["hq"], case["hk"], case["d"]
    if op == "norm_rope":
        n = case["tokens"]
        return {"bytes": n * ((hq + hk) * d * 4 + 4 * case["axes"]) + 4 * d, "flops": n * (hq + hk) * d * 10}
    fresh, whole = _lengths(case)
    n = sum(fresh)
    cached = 2.5 * d / 2                                # bytes of a token's k and v in one head
    rows = 4 * d
    if op == "attention":
        seen = sum(t * c - t * (t - 1) / 2 for t, c in zip(fresh, whole))
        return {"bytes": sum(whole) * hk * cached + n * hq * rows, "flops": 4 * hq * d * seen}
    if op == "read":
        return {"bytes": n * hk * (cached + rows), "flops": n * hk * d * 4}
    both = 2 * n * hk * (cached + rows)                 # the write, and the read-back
    if op == "append_qkv":
        return {"bytes": both + n * hq * rows, "flops": n * (hq + 3 * hk) * d * 10}
    return {"bytes": both, "flops": n * hk * d * 20}


# ---------------------------------------------------------------- the definition in 64 bits

def _exact_norm_rope(s, x, weight):
    x = x.double()
    x = x / torch.sqrt((x * x).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]) * weight.double()
    y = x.clone()
    half = s["rot"] // 2
    for i in range(half):
        a, b = (2 * i, 2 * i + 1) if s["inter"] else (i, i + half)
        turn = s["positions"][s["axis"][i]].double() * float(s["inv_freq"][i])
        c, n = torch.cos(turn)[:, None], torch.sin(turn)[:, None]
        y[..., a] = c * x[..., a] - n * x[..., b]
        y[..., b] = n * x[..., a] + c * x[..., b]
    return y


def _exact_stored(x):
    """The values that the cache stands for after rows x were written."""
    x = torch.where(torch.isnan(x.double()), 0.0, x.double())
    x = torch.clamp(x, -LIMIT, LIMIT)
    y = torch.empty_like(x)
    for g in range(0, x.shape[-1], 32):
        part = x[..., g:g + 32]
        low = part.min(-1, keepdim=True).values
        scale = ((part.max(-1, keepdim=True).values - low) / 15).to(torch.float16).double()
        low = low.to(torch.float16).double()
        code = torch.round((part - low) / torch.where(scale > 0, scale, 1.0))
        y[..., g:g + 32] = torch.where(scale > 0, code.clamp(0, 15), 0.0) * scale + low
    return y


def _exact_cached(s, b, n):
    """(k, v) float64 [n][heads][d] of the first n tokens of sequence b, from the page bytes."""
    case = s["case"]
    hk, d, page = case["hk"], case["d"], case["page"]
    t = torch.arange(n, device=DEV)
    blk = s["page_table"][b].long()[t // page] * hk * (page // 16) + (t % page) // 16
    base = (blk[:, None] + torch.arange(hk, device=DEV) * (page // 16)) * (20 * d)     # [n][hk]
    r = t % 16
    c = torch.arange(d, device=DEV)
    g, e = c // 32, c % 32
    raw = s["buffer"]
    found = []
    for side in (0, 1):
        if side == 0:
            off = (r * (d // 2))[:, None] + (e // 8) * (d // 8) + g * 4 + (e % 8) // 2
        else:
            piece = (e // 4)[None] ^ (4 * ((r // 2) % 2) if d == 128 else 0 * r)[:, None]
            off = (r * (d // 2))[:, None] + piece * (d // 16) + g * 2 + (e % 4) // 2
        byte = raw[base[..., None] + side * 10 * d + off[:, None]].long()
        code = torch.where(c % 2 == 1, byte // 16, byte % 16).double()
        at = base[..., None] + side * 10 * d + 8 * d + (r * (d // 8))[:, None, None] + 4 * torch.arange(d // 32, device=DEV)
        num = raw[at[..., None] + torch.arange(4, device=DEV)].contiguous().view(torch.float16).double()
        found.append(code * num[..., 0][..., g] + num[..., 1][..., g])
    return found


def exact(case, seed):
    s = prepare(case, seed)
    op, hq, hk, d = case["op"], case["hq"], case["hk"], case["d"]
    if op == "attention":
        out = torch.empty(s["tokens"], hq, d, dtype=torch.float64, device=DEV)
        first = s["q_start"].tolist()
        for b in range(case["batch"]):
            n, t = int(s["kv_len"][b]), first[b + 1] - first[b]
            k, v = _exact_cached(s, b, n)
            hide = torch.arange(n, device=DEV)[None] > (n - t + torch.arange(t, device=DEV))[:, None]
            for h in range(hq):
                kv = h // (hq // hk)
                a = s["q"][first[b]:first[b + 1], h].double() @ k[:, kv].T * d ** -0.5
                out[first[b]:first[b + 1], h] = torch.softmax(a.masked_fill(hide, -math.inf), -1) @ v[:, kv]
        return out
    if op == "read":
        first, parts = s["q_start"].tolist(), []
        for b in range(case["batch"]):
            n = int(s["kv_len"][b])
            k, v = _exact_cached(s, b, n)
            parts.append((k[n - first[b + 1] + first[b]:], v[n - first[b + 1] + first[b]:]))
        return [torch.cat([p[i] for p in parts]) for i in (0, 1)]
    q, k, v = s["qkv"][:, :hq], s["qkv"][:, hq:hq + hk], s["qkv"][:, hq + hk:]
    if op == "append":
        return [_exact_stored(k), _exact_stored(v)]
    q, k = _exact_norm_rope(s, q, s["q_weight"]), _exact_norm_rope(s, k, s["k_weight"])
    if op == "norm_rope":
        return q, k
    # keys enter the cache as the bf16 rows that the rotation gives
    return [q, _exact_stored(k.to(torch.bfloat16)), _exact_stored(v)]
