"""Work of a paged KV cache held in 4 bits, for measuring.

Four operators, each in its plain form (elementary torch operations) and, with
``own`` set, as calls of the framework:

pages   block tables and slot maps of a batch of requests, from their lengths
store   bf16 K/V rows into the 4-bit cache at given slots, and read back (what
        4 bits hold is only seen through a load)
load    the rows of given slots back as bf16
attend  attention of new tokens over the 4-bit cache through block tables, with
        or without a sliding window and first tokens that stay visible

Cache format. Each (token, head) row of D channels is cut into groups of G
channels; a group keeps lo (its minimum) and s = bf16((max - lo) / 15) as bf16
and 4-bit codes n = min(15, round((x - lo) / s)) (0 where s is 0), rounded half to
even; it stands for lo + s n. The
cache is [layers][pages][heads][page tokens / 16] blobs of 16 tokens, each
blob: K codes, K parameters, V codes, V parameters.
  K codes   byte (c % 32) / 8 * D/8 + c / 32 * 4 + c % 8 / 2 of the token's D/2
  V codes   the tokens 2p and 2p + 1 share D bytes: byte
            c % 32 / 4 * D/8 + c / 32 * 4 + token % 2 * 2 + c % 4 / 2
  (the even channel of a byte in its low half), parameters [token][group] (s, lo).
"""
import math

import torch

own = False
DEVICE = "cuda"


# ---------------------------------------------------------------- the cases

def listed():
    return [
        # one decode step of a serving batch: every request gets one token
        dict(name="pages, decode step", op="pages", requests=64, len=4096, count=1, page=16),
        # many prompts and running requests mixed, ragged
        dict(name="pages, mixed batch", op="pages", requests=4096, len=4096, count=257, page=16),
        # the new tokens of one decode step, one layer
        dict(name="store, decode step", op="store", layers=1, tokens=64, heads=8, dim=128, group=32, page=16),
        # a 16K-token cache of 32 layers restored from its compressed form
        dict(name="store, restored cache", op="store", layers=32, tokens=16384, heads=8, dim=128, group=32, page=16),
        # one 256-token object of all layers, read back to be compressed
        dict(name="load, one object", op="load", layers=32, tokens=256, heads=8, dim=128, group=32, page=16),
        # a 32K-token cache of 40 layers with 2 KV heads swapped out
        dict(name="load, whole cache", op="load", layers=40, tokens=32768, heads=2, dim=128, group=64, page=64),
        # the first answers of a single short chat, as many KV heads as query heads
        dict(name="attend, one short", op="attend", requests=1, queries=1, kv=129, spread=0.0, q_heads=12, heads=12, dim=64,
             group=32, page=16, window=0, sinks=0),
        # a serving batch at ragged lengths
        dict(name="attend, batch", op="attend", requests=64, queries=1, kv=8192, spread=0.5, q_heads=32, heads=8, dim=128,
             group=32, page=16, window=0, sinks=0),
        # a few drafted tokens of long contexts verified at once
        dict(name="attend, drafts at 128K", op="attend", requests=4, queries=4, kv=131072, spread=0.1, q_heads=32, heads=2,
             dim=128, group=64, page=64, window=0, sinks=0),
        # a whole prompt
        dict(name="attend, prompt 8K", op="attend", requests=1, queries=8192, kv=8192, spread=0.0, q_heads=32, heads=8,
             dim=128, group=32, page=16, window=0, sinks=0),
        # long streams that see their last 4096 tokens and the first 4
        dict(name="window, batch at 32K", op="attend", requests=32, queries=1, kv=32768, spread=0.3, q_heads=32, heads=8,
             dim=128, group=32, page=16, window=4096, sinks=4),
        # one chunk of a long prompt under a window
        dict(name="window, chunk at 32K", op="attend", requests=1, queries=2048, kv=32768, spread=0.0, q_heads=32, heads=8,
             dim=128, group=128, page=32, window=4096, sinks=4),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("pages", "store", "load", "attend", "attend", "prompt"))
    page = rng.choice((16, 16, 32, 48, 64, 128))
    if kind == "pages":
        n = _log(rng, 1, 4096)
        return dict(op="pages", requests=n, len=_log(rng, 16, 4096), count=_log(rng, 1, 300), page=page)
    heads, dim = rng.choice(((8, 128), (2, 128), (12, 64), (1, 128), (4, 64), (5, 128)))
    group = rng.choice([g for g in (32, 64, 128) if g <= dim])
    if kind in ("store", "load"):
        layers = rng.choice((1, 1, 12, 32, 40))
        most = max(1, 16384 * 32 * 8 * 128 // (layers * heads * dim))
        return dict(op=kind, layers=layers, tokens=_log(rng, 1, min(most, 32768)), heads=heads, dim=dim, group=group, page=page)
    ratio = rng.choice((1, 2, 4, 4, 7, 8, 16)) if heads <= 2 else rng.choice((1, 2, 3, 4, 4))
    window = rng.choice((0, 0, _log(rng, 16, 8192)))
    sinks = rng.choice((0, 1, 4, 37)) if window else 0
    if kind == "attend":
        queries = rng.choice((1, 1, 1, 2, 4, 5))
        requests = _log(rng, 1, 64)
        kv = max(queries, _log(rng, 1, min(131072, 400000 // requests)))
        spread = rng.choice((0.0, 0.3, 0.9))
    else:
        queries = _log(rng, 6, 4096)
        requests = rng.choice((1, 1, 2, 5))
        kv = min(queries * rng.choice((1, 1, 2, 5)) + rng.randrange(64), 16384)
        requests = max(1, min(requests, 8192 * 8192 * 32 // (4 * queries * kv * heads * ratio)))
        spread = rng.choice((0.0, 0.2))
    return dict(op="attend", requests=requests, queries=queries, kv=kv, spread=spread, q_heads=heads * ratio, heads=heads,
                dim=dim, group=group, page=page, window=window, sinks=sinks)


def _spread(n, high, spread):
    """n lengths from high down to (1 - spread) high, in no order, by the case alone."""
    return [max(1, high - int(((i * 0.6180339887) % 1.0) * spread * high)) for i in range(n)]


def _lengths(case):
    """(query tokens, cache tokens) of each request of an attend case."""
    kv = _spread(case["requests"], case["kv"], case["spread"])
    return [min(case["queries"], k) for k in kv], kv


# --------------------------------------------------------------- the inputs

def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    ints = dict(dtype=torch.int32, device=DEVICE)
    if case["op"] == "pages":
        n, page = case["requests"], case["page"]
        # work() goes by the lengths: they are the case's, their order is the seed's
        turn = torch.randperm(n, generator=g, device=DEVICE)
        lens = torch.tensor(_spread(n, case["len"], 0.9), **ints)[turn]
        counts = torch.tensor(_spread(n, case["count"], 1.0), **ints)[turn]
        tokens = sum(_spread(n, case["count"], 1.0))
        width = -(-(case["len"] + case["count"]) // page)
        held = (lens + page - 1) // page
        need = int(((lens + counts + page - 1) // page - held).sum())
        pages = int(held.sum()) + need + 33
        ids = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
        at = torch.arange(width, **ints)[None, :]
        first = torch.cumsum(held, 0) - held
        table = torch.where(at < held[:, None], ids[(first[:, None] + at).clamp(max=pages - 1)], -1).to(torch.int32).contiguous()
        free = ids[int(held.sum()):].contiguous()
        return dict(case=case, table=table, lens=lens, counts=counts, free=free,
                    free_count=torch.tensor([free.numel()], **ints), tokens=tokens + 7)
    heads, dim, group, page = case["heads"], case["dim"], case["group"], case["page"]
    # channels of very different size, as keys have them
    sigma = torch.exp(0.5 * torch.randn(heads, dim, generator=g, device=DEVICE))
    sigma[:, :2] *= 8.0
    bf = dict(dtype=torch.bfloat16, device=DEVICE)
    if case["op"] in ("store", "load"):
        layers, n = case["layers"], case["tokens"]
        pages = -(-n // page) + 1
        ids = torch.randperm(pages, generator=g, device=DEVICE)
        at = torch.arange(n, device=DEVICE)
        slots = (ids[at // page] * page + at % page).to(torch.int32)
        data = torch.zeros(layers, pages, heads, page // 16, 16 * (dim + 8 * (dim // group)), dtype=torch.uint8, device=DEVICE)
        kv = torch.empty(layers, 2, n, heads, dim, **bf)
        for layer in range(layers):
            x = torch.randn(2, n, heads, dim, generator=g, device=DEVICE)
            x[0] *= sigma
            kv[layer] = x
        s = dict(case=case, data=data, slots=slots)
        if case["op"] == "store":
            return dict(s, k=kv[:, 0], v=kv[:, 1])
        for layer in range(layers):
            _write(data[layer:layer + 1], kv[layer:layer + 1, 0], kv[layer:layer + 1, 1], slots, page, group)
        return s
    nq, nkv = _lengths(case)
    requests = len(nq)
    held = [-(-k // page) for k in nkv]
    pages = sum(held) + 1
    ids = torch.randperm(pages, generator=g, device=DEVICE).to(torch.int32)
    first = torch.tensor([0] + held, **ints).cumsum(0)[:-1]
    width = max(held)
    at = torch.arange(width, **ints)[None, :]
    table = torch.where(at < torch.tensor(held, **ints)[:, None], ids[(first[:, None] + at).clamp(max=pages - 1)], -1)
    # places that hold no token keep what was there before (here bytes that are no numbers)
    data = torch.full((1, pages, heads, page // 16, 16 * (dim + 8 * (dim // group))), 255, dtype=torch.uint8, device=DEVICE)
    lens = torch.tensor(nkv, **ints)
    pos = torch.arange(width * page, **ints)
    slots = (table[:, (pos // page).long()] * page + pos % page)[pos[None, :] < lens[:, None]]
    step = 65536
    for a in range(0, slots.numel(), step):
        part = slots[a:a + step]
        k = (torch.randn(1, part.numel(), heads, dim, generator=g, device=DEVICE) * sigma).to(torch.bfloat16)
        v = torch.randn(1, part.numel(), heads, dim, generator=g, device=DEVICE).to(torch.bfloat16)
        _write(data, k, v, part, page, group)
    tokens = sum(nq)
    ratio = case["q_heads"] // heads
    q = 1.5 * torch.randn(tokens, heads, ratio, dim, generator=g, device=DEVICE) / sigma[:, None, :]
    cu = torch.tensor([0] + nq, **ints).cumsum(0).to(torch.int32)
    return dict(case=case, data=data, table=table.to(torch.int32).contiguous(), lens=lens, cu=cu,
                q=q.reshape(tokens, heads * ratio, dim).to(torch.bfloat16))


# ----------------------------------------------------------- the plain forms

def _views(data, dim, group):
    """K codes, K parameters, V codes, V parameters of the cache's bytes."""
    a, b = 16 * dim // 2, 16 * 4 * (dim // group)
    kc = data[..., :a].unflatten(-1, (16, 4, dim // 32, 4))                       # token, c%32/8, c/32, byte
    kp = data[..., a:a + b].view(torch.bfloat16).unflatten(-1, (16, dim // group, 2))
    vc = data[..., a + b:2 * a + b].unflatten(-1, (8, 8, dim // 32, 2, 2))        # pair, c%32/4, c/32, token%2, byte
    vp = data[..., 2 * a + b:].view(torch.bfloat16).unflatten(-1, (16, dim // group, 2))
    return kc, kp, vc, vp


def _quantise(x, group):
    """x [..., dim] -> codes (whole numbers in 8 bits) [..., dim], (s, lo) [..., groups, 2] in bf16."""
    x = x.float().unflatten(-1, (-1, group))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    s = ((hi - lo) / 15.0).to(torch.bfloat16).float()
    n = torch.where(s > 0.0, torch.round((x - lo) / s).clamp(max=15.0), 0.0).to(torch.uint8).flatten(-2)
    return n, torch.cat((s, lo), -1).to(torch.bfloat16)


def _write(data, k, v, slots, page, group):
    """The rows k, v [layers, tokens, heads, dim] at slots."""
    dim = k.shape[-1]
    kc, kp, vc, vp = _views(data, dim, group)
    slots = slots.long()
    pg, blob, tok = slots // page, slots % page // 16, slots % 16
    n, par = _quantise(k, group)
    n = n.unflatten(-1, (dim // 32, 4, 4, 2)).transpose(-4, -3)
    kc[:, pg, :, blob, tok] = (n[..., 0] | (n[..., 1] << 4)).transpose(0, 1)
    kp[:, pg, :, blob, tok] = par.transpose(0, 1)
    n, par = _quantise(v, group)
    n = n.unflatten(-1, (dim // 32, 8, 2, 2)).transpose(-4, -3)
    vc[:, pg, :, blob, tok // 2, :, :, tok % 2] = (n[..., 0] | (n[..., 1] << 4)).transpose(0, 1)
    vp[:, pg, :, blob, tok] = par.transpose(0, 1)


def _values(codes, par, group):
    """lo + s n in fp32."""
    par = par.float()
    return (codes.float().unflatten(-1, (-1, group)) * par[..., 0:1] + par[..., 1:2]).flatten(-2)


def _k_of(c, p, group):
    c = torch.stack((c & 15, c >> 4), -1).transpose(-4, -3)
    return _values(c.flatten(-4), p, group)


_v_of = _k_of  # both keep [c%32 part][c/32] bytes of two channels, once the token is picked


def _read(data, slots, page, group, dim):
    kc, kp, vc, vp = _views(data, dim, group)
    slots = slots.long()
    pg, blob, tok = slots // page, slots % page // 16, slots % 16
    k = _k_of(kc[:, pg, :, blob, tok], kp[:, pg, :, blob, tok], group)
    v = _v_of(vc[:, pg, :, blob, tok // 2, :, :, tok % 2], vp[:, pg, :, blob, tok], group)
    return k.to(torch.bfloat16).transpose(0, 1), v.to(torch.bfloat16).transpose(0, 1)


def _plain_pages(s):
    page, table, lens, counts = s["case"]["page"], s["table"], s["lens"], s["counts"]
    held = (lens + page - 1) // page
    need = (lens + counts + page - 1) // page - held
    base = torch.cumsum(need, 0) - need
    at = torch.arange(table.shape[1], device=DEVICE)[None, :]
    new = (at >= held[:, None]) & (at < (held + need)[:, None])
    take = s["free_count"] - 1 - (base[:, None] + at - held[:, None])
    table.copy_(torch.where(new, s["free"][take.clamp(0, s["free"].numel() - 1)], table))
    end = torch.cumsum(counts, 0)
    cu = torch.cat((torch.zeros_like(end[:1]), end)).to(torch.int32)
    t = torch.arange(s["tokens"], device=DEVICE)
    r = torch.searchsorted(end, t, right=True).clamp(max=lens.numel() - 1)
    pos = t - cu[r] + lens[r]
    slots = table[r, (pos // page).clamp(max=table.shape[1] - 1)] * page + pos % page
    slots = torch.where(t < end[-1], slots, -1).to(torch.int32)
    return dict(table=table, slots=slots, cu=cu, lens=lens + counts, free_count=(s["free_count"] - need.sum()).to(torch.int32))


def _plain_attend(s):
    case, q, table, lens, cu = s["case"], s["q"], s["table"], s["lens"], s["cu"]
    heads, dim, group, page = case["heads"], case["dim"], case["group"], case["page"]
    requests, width = table.shape
    most, ratio = case["queries"], case["q_heads"] // heads
    got = s["data"][0][table.clamp(min=0).long()]                      # requests, width, heads, blobs, bytes
    kc, kp, vc, vp = _views(got, dim, group)
    tokens = width * page
    seen = (torch.arange(tokens, device=DEVICE)[None, :] < lens[:, None])[:, None, :, None]
    k = _k_of(kc, kp, group).transpose(1, 2).reshape(requests, heads, tokens, dim)
    v = _v_of(vc.movedim(-2, -4).flatten(-5, -4), vp, group).transpose(1, 2).reshape(requests, heads, tokens, dim)
    k, v = torch.where(seen, k, 0.0), torch.where(seen, v, 0.0)
    row = torch.arange(most, device=DEVICE)
    n = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + torch.minimum(row[None, :], n[:, None] - 1)).long()
    qp = q.float()[at].unflatten(2, (heads, ratio)).permute(0, 2, 3, 1, 4).reshape(requests, heads, ratio * most, dim)
    scores = torch.matmul(qp, k.transpose(-1, -2)).mul_(1.0 / math.sqrt(dim)).unflatten(2, (ratio, most))
    pos = (lens - n)[:, None, None] + row[None, :, None]
    j = torch.arange(tokens, device=DEVICE)[None, None, :]
    hide = (j > pos) | (j >= lens[:, None, None])
    if case["window"]:
        hide = hide | ((pos - j >= case["window"]) & (j >= case["sinks"]))
    scores.masked_fill_(hide[:, None, None], -math.inf)
    scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    total = scores.sum(-1, keepdim=True)
    out = torch.matmul(scores.flatten(2, 3), v).unflatten(2, (ratio, most)) / total
    out = out.permute(0, 3, 1, 2, 4).reshape(requests, most, heads * ratio, dim)
    t = torch.arange(q.shape[0], device=DEVICE)
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return out[r, t - cu[r]].to(torch.bfloat16)


# ------------------------------------------------------------------ one pass

def _cache(s):
    """The handle that a user's program keeps for its cache."""
    if "cache" not in s:
        from kv_cache_compression_03_gb300 import cachegen as cg
        case, d = s["case"], s["data"]
        s["cache"] = cg.Int4Cache(d.shape[0], d.shape[1], case["page"], case["heads"], case["dim"], case["group"], data=d)
    return s["cache"]


def run(state):
    s, case = state, state["case"]
    op, page, group = case["op"], case["page"], case.get("group")
    if own:
        if op == "pages":
            from kv_cache_compression_03_gb300 import cachegen as cg
            p = cg.grow_pages(s["table"], s["lens"], s["counts"], s["free"], s["free_count"], page, s["tokens"])
            return dict(table=s["table"], slots=p.slots, cu=p.cu, lens=p.lens, free_count=p.free_count)
        cache = _cache(s)
        if op == "attend":
            return dict(out=cache.attention(s["q"], s["cu"], s["lens"], s["table"], window=case["window"], sinks=case["sinks"],
                                            max_q_len=case["queries"]))
        if op == "store":
            cache.store(s["k"], s["v"], s["slots"])
        k, v = cache.load(s["slots"], layers=case["layers"])
        return dict(k=k, v=v)
    if op == "pages":
        return _plain_pages(s)
    if op == "attend":
        return dict(out=_plain_attend(s))
    if op == "store":
        _write(s["data"], s["k"], s["v"], s["slots"], page, group)
    k, v = _read(s["data"], s["slots"], page, group, case["dim"])
    return dict(k=k, v=v)


# ------------------------------------------------------- what a pass has to do

def work(case):
    if case["op"] == "pages":
        n, page = case["requests"], case["page"]
        lens, counts = _spread(n, case["len"], 0.9), _spread(n, case["count"], 1.0)
        pairs = sorted(zip(lens, counts))
        need = sum(-(-(a + b) // page) + (-a // page) for a, b in pairs)
        shared = sum(1 for a in lens if a % page)
        return dict(bytes=8 * n + 4 * shared + 8 * need + 4 * sum(counts) + 8 * n + 12, flops=0)
    heads, dim = case["heads"], case["dim"]
    held = dim + 8 * (dim // case["group"])                            # bytes of one token and head in the cache
    if case["op"] in ("store", "load"):
        rows = case["layers"] * case["tokens"] * heads
        there = rows * (4 * dim + held)
        return dict(bytes=there * (2 if case["op"] == "store" else 1) + 4 * case["tokens"], flops=0)
    nq, nkv = _lengths(case)
    window, sinks = case["window"] or 1 << 40, case["sinks"]
    pairs = tokens = 0
    for n, k in zip(nq, nkv):
        p0 = k - n
        # the last min(window, position + 1) tokens, and the first ones before those
        for p in range(p0, k):
            low = max(0, p + 1 - window)
            pairs += p + 1 - low + min(low, sinks)
        low = max(0, p0 + 1 - window)
        tokens += k - low + min(low, sinks)
    return dict(bytes=tokens * heads * held + 4 * sum(nq) * case["q_heads"] * dim, flops=4 * dim * case["q_heads"] * pairs)


# ------------------------------------------------- the definition in 64 bits

def _places(dim, device):
    """Byte and shift of each channel in a token's K codes and in a pair's V codes (token 0 of the pair)."""
    c = torch.arange(dim, device=device)
    kb = (c % 32) // 8 * (dim // 8) + c // 32 * 4 + c % 8 // 2
    vb = (c % 32) // 4 * (dim // 8) + c // 32 * 4 + c % 4 // 2
    return kb, vb, c % 2 * 4


def _exact_rows(case, data, slots):
    """The values of slots in one layer's bytes [pages, heads, blobs, bytes]: k, v [tokens, heads, dim] in 64 bits."""
    dim, group, page = case["dim"], case["group"], case["page"]
    groups = dim // group
    kb, vb, shift = _places(dim, data.device)
    rows = data[slots // page, :, slots % page // 16]                  # tokens, heads, bytes of the blob
    tok = (slots % 16)[:, None, None]
    of = torch.arange(dim, device=data.device) // group
    a = 8 * dim + 64 * groups
    out = []
    for place, par in ((tok * (dim // 2) + kb, 8 * dim), (a + tok // 2 * dim + tok % 2 * 2 + vb, a + 8 * dim)):
        code = rows.gather(2, place.expand(-1, rows.shape[1], -1)) >> shift & 15
        at = (par + (tok * groups + of) * 4).expand(-1, rows.shape[1], -1)
        b = [rows.gather(2, at + i).int() for i in range(4)]
        s = ((b[1] << 24) | (b[0] << 16)).view(torch.float32).double()
        lo = ((b[3] << 24) | (b[2] << 16)).view(torch.float32).double()
        out.append(lo + s * code.double())
    return out


def _exact_stored(x, group):
    x = x.double()
    out = torch.empty_like(x)
    for a in range(0, x.shape[-1], group):
        y = x[..., a:a + group]
        lo = y.min(-1, keepdim=True).values
        s = ((y.max(-1, keepdim=True).values - lo) / 15).to(torch.bfloat16).double()
        out[..., a:a + group] = torch.where(s > 0, lo + s * torch.round((y - lo) / s).clamp(0, 15), lo)
    return out


def exact(case, seed):
    if case["op"] == "pages":
        return None                                                    # whole numbers
    s = prepare(case, seed)
    if case["op"] == "store":
        return dict(k=_exact_stored(s["k"], case["group"]), v=_exact_stored(s["v"], case["group"]))
    if case["op"] == "load":
        both = [_exact_rows(case, d, s["slots"].long()) for d in s["data"]]
        return dict(k=torch.stack([b[0] for b in both]), v=torch.stack([b[1] for b in both]))
    nq, nkv = _lengths(case)
    heads, dim, page = case["heads"], case["dim"], case["page"]
    ratio = case["q_heads"] // heads
    out = torch.empty(sum(nq), case["q_heads"], dim, dtype=torch.float64, device=DEVICE)
    row = 0
    for r, (n, m) in enumerate(zip(nq, nkv)):
        at = torch.arange(m, device=DEVICE)
        k, v = _exact_rows(case, s["data"][0], s["table"][r, at // page].long() * page + at % page)
        behind = torch.arange(m - n, m, device=DEVICE)[:, None] - at[None, :]
        visible = behind >= 0
        if case["window"]:
            visible &= (behind < case["window"]) | (at[None, :] < case["sinks"])
        for h in range(case["q_heads"]):
            score = s["q"][row:row + n, h].double() @ k[:, h // ratio].T / math.sqrt(dim)
            p = torch.softmax(torch.where(visible, score, -math.inf), -1)
            out[row:row + n, h] = p @ v[:, h // ratio]
        row += n
    return dict(out=out)
