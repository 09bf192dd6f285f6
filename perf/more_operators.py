"""Work of a paged 4-bit KV cache whose requests share a prefix, and whose tokens
are evicted by the attention that they got, for measuring.

Five operators, each in its plain form (elementary torch operations) and, with
``own`` set, as calls of the framework:

shared   attention of new tokens of a batch whose requests begin with the same
         cached tokens, read once for all of them
weigh    the attention weight that each cached token got from the new tokens'
         queries, summed per KV head and added to what it had
choose   the tokens of each head that stay: the first ones, the last ones and
         those with the greatest weights
compact  the tokens that stay moved to the front of their request's pages, their
         weights with them (what 4 bits hold is seen through a load)
release  the pages behind the shorter requests, back on the list of free pages

Cache format. Each (token, head) row of D channels is cut into groups of G
channels; a group keeps lo and s as bf16 and 4-bit codes n; it stands for
lo + s n. The cache is [layers][pages][heads][page tokens / 16] blobs of 16
tokens, each blob: K codes, K parameters, V codes, V parameters.
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
        # a few chats just begun on one short instruction, as many KV heads as query heads
        dict(name="shared, four short", op="shared", requests=4, queries=1, shared=1024, kv=65, spread=0.9, q_heads=12, heads=12,
             dim=64, group=32, page=16),
        # one decode step of a serving batch on a long instruction
        dict(name="shared, batch", op="shared", requests=64, queries=1, shared=16384, kv=1024, spread=0.9, q_heads=32, heads=8,
             dim=128, group=32, page=16),
        # questions of some hundred tokens about one document
        dict(name="shared, questions", op="shared", requests=8, queries=300, shared=32768, kv=300, spread=0.7, q_heads=32, heads=2,
             dim=128, group=64, page=64),
        # a decode step that keeps account of its attention
        dict(name="weigh, batch", op="weigh", requests=64, queries=1, kv=8192, spread=0.5, q_heads=32, heads=8, dim=128, group=32,
             page=16, window=0, sinks=0),
        # the last tokens of a long prompt say which of it is wanted
        dict(name="weigh, last of 32K", op="weigh", requests=1, queries=32, kv=32768, spread=0.0, q_heads=32, heads=8, dim=128,
             group=32, page=16, window=0, sinks=0),
        # whole prompts, each of whose queries counts
        dict(name="weigh, prompts", op="weigh", requests=2, queries=2048, kv=2048, spread=0.3, q_heads=32, heads=8, dim=128,
             group=128, page=32, window=0, sinks=0),
        # one layer of a serving batch that has filled its budget
        dict(name="choose, one layer", op="choose", layers=1, requests=64, heads=8, len=4608, spread=0.2, budget=4096, recent=256,
             sinks=4),
        # every layer of a long context cut to a few thousand tokens
        dict(name="choose, long context", op="choose", layers=32, requests=1, heads=8, len=65536, spread=0.0, budget=4096, recent=64,
             sinks=16),
        # one layer of a batch, an eighth of whose tokens goes
        dict(name="compact, one layer", op="compact", layers=1, requests=16, heads=8, len=2304, spread=0.2, budget=2048, recent=128,
             sinks=4, dim=128, group=32, page=16),
        # all layers of a long context, half of whose tokens go
        dict(name="compact, long context", op="compact", layers=32, requests=1, heads=8, len=16384, spread=0.0, budget=8192,
             recent=64, sinks=16, dim=128, group=32, page=16),
        # a serving batch cut to its budget
        dict(name="release, batch", op="release", requests=64, len=4608, spread=0.9, budget=4096, page=16),
        # thousands of requests that end or are cut
        dict(name="release, many", op="release", requests=4096, len=4096, spread=1.0, budget=300, page=16),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    kind = rng.choice(("shared", "shared", "weigh", "weigh", "choose", "compact", "release"))
    page = rng.choice((16, 16, 32, 48, 64, 128))
    spread = rng.choice((0.0, 0.3, 0.9))
    if kind == "release":
        length = _log(rng, 16, 4096)
        return dict(op=kind, requests=_log(rng, 1, 4096), len=length, spread=rng.choice((0.3, 0.9, 1.0)), budget=_log(rng, 1, length),
                    page=page)
    heads, dim = rng.choice(((8, 128), (2, 128), (12, 64), (1, 128), (4, 64), (5, 128)))
    group = rng.choice([g for g in (32, 64, 128) if g <= dim])
    ratio = rng.choice((1, 2, 4, 4, 7, 8, 16)) if heads <= 2 else rng.choice((1, 2, 3, 4, 4))
    if kind in ("choose", "compact"):
        most = 65536 if kind == "choose" else 32768
        layers, requests = rng.choice((1, 1, 2, 12, 32)), _log(rng, 1, 64)
        length = _log(rng, 1, max(2, min(most, (65536 * 256 if kind == "choose" else 16384 * 256) // (layers * requests * heads))))
        budget = max(1, int(length * rng.choice((0.1, 0.5, 0.9, 1.1)))) + rng.randrange(3)
        recent = int(budget * rng.choice((0.0, 0.1, 0.5)))
        sinks = min(rng.choice((0, 1, 4, 37)), budget - recent)
        c = dict(op=kind, layers=layers, requests=requests, heads=heads, len=length, spread=spread, budget=budget, recent=recent,
                 sinks=sinks)
        return c if kind == "choose" else dict(c, dim=dim, group=group, page=page)
    size = dict(q_heads=heads * ratio, heads=heads, dim=dim, group=group, page=page)
    if kind == "shared":
        requests = _log(rng, 1, 64)
        queries = rng.choice((1, 1, 1, 2, 4, _log(rng, 5, 300)))
        # no more pairs of a query and a token than the questions have
        most = 8 * 200 * 32768 * 32 // (requests * queries * heads * ratio)
        kv = max(queries, _log(rng, 1, max(2, min(4096, most))))
        return dict(op=kind, requests=requests, queries=queries, shared=max(1, _log(rng, 16, max(17, min(65536, most))) // page) * page,
                    kv=kv, spread=spread, **size)
    window = rng.choice((0, 0, 0, _log(rng, 16, 8192)))
    sinks = rng.choice((0, 1, 4, 37)) if window else 0
    queries = rng.choice((1, 1, 1, 2, 5, _log(rng, 6, 64), _log(rng, 64, 2048)))
    requests = _log(rng, 1, 64) if queries < 6 else rng.choice((1, 1, 2, 3))
    kv = max(queries, _log(rng, 1, min(65536, 400000 // requests)) if queries < 64 else queries * rng.choice((1, 1, 2)) + rng.randrange(64))
    requests = max(1, min(requests, 2 * 2048 * 2048 * 32 // (queries * kv * heads * ratio)))
    return dict(op=kind, requests=requests, queries=queries, kv=kv, spread=spread, window=window, sinks=sinks, **size)


def _spread(n, high, spread):
    """n lengths from high down to (1 - spread) high, in no order, by the case alone."""
    return [max(1, high - int(((i * 0.6180339887) % 1.0) * spread * high)) for i in range(n)]


def _lengths(case):
    """(query tokens, tokens behind the shared ones) of each request."""
    kv = _spread(case["requests"], case["kv"], case["spread"])
    return [min(case["queries"], k) for k in kv], kv


# --------------------------------------------------------------- the inputs

def _pages(held, gen, more):
    """A table of pages in no order for requests that hold so many each (a list), and the ids that are left."""
    ints = dict(dtype=torch.int32, device=DEVICE)
    ids = torch.randperm(sum(held) + more, generator=gen, device=DEVICE).to(torch.int32)
    n = torch.tensor(held, **ints)
    first = torch.cumsum(n, 0) - n
    at = torch.arange(max(held), **ints)[None, :]
    table = torch.where(at < n[:, None], ids[(first[:, None] + at).clamp(max=ids.numel() - 1)], -1)
    return table.to(torch.int32).contiguous(), ids[sum(held):].contiguous()


def _fill(data, slots, gen, heads, dim, group, page, sigma):
    """Random rows, as models have them, into the slots of every layer."""
    step = 65536
    for layer in range(data.shape[0]):
        for a in range(0, slots.numel(), step):
            part = slots[a:a + step]
            k = (torch.randn(1, part.numel(), heads, dim, generator=gen, device=DEVICE) * sigma).to(torch.bfloat16)
            v = torch.randn(1, part.numel(), heads, dim, generator=gen, device=DEVICE).to(torch.bfloat16)
            _write(data[layer:layer + 1], k, v, part, page, group)


def _weights(shape, length, lens, gen):
    """Sums of attention weights: a few large ones, many small, some that nothing ever came to; 0 behind the last token."""
    w = torch.exp(2.0 * torch.randn(*shape, length, generator=gen, device=DEVICE)) / length
    w = torch.where(torch.rand(*shape, length, generator=gen, device=DEVICE) < 0.02, 0.0, w)
    at = torch.arange(length, device=DEVICE)
    return torch.where(at < lens[:, None, None], w, 0.0)


def prepare(case, seed):
    g = torch.Generator(device=DEVICE).manual_seed(seed)
    ints = dict(dtype=torch.int32, device=DEVICE)
    op = case["op"]
    if op == "release":
        n, page = case["requests"], case["page"]
        lens = _spread(n, case["len"], case["spread"])
        table, free = _pages([-(-x // page) for x in lens], g, 17)
        room = torch.full((table.numel(),), -7, **ints)
        now = torch.tensor(lens, **ints)
        return dict(case=case, table=table, lens=now, new_lens=now.clamp(max=case["budget"]), free=torch.cat((free, room)),
                    free_count=torch.tensor([free.numel()], **ints))
    if op == "choose":
        lens = torch.tensor(_spread(case["requests"], case["len"], case["spread"]), **ints)
        return dict(case=case, lens=lens, weights=_weights((case["layers"], case["requests"], case["heads"]), case["len"], lens, g))
    heads, dim, group, page = case["heads"], case["dim"], case["group"], case["page"]
    # channels of very different size, as keys have them
    sigma = torch.exp(0.5 * torch.randn(heads, dim, generator=g, device=DEVICE))
    sigma[:, :2] *= 8.0
    blob = 16 * (dim + 8 * (dim // group))
    if op == "compact":
        layers, n = case["layers"], case["requests"]
        lens = _spread(n, case["len"], case["spread"])
        table, _ = _pages([-(-x // page) for x in lens], g, 1)
        data = torch.full((layers, sum(-(-x // page) for x in lens) + 1, heads, page // 16, blob), 255, dtype=torch.uint8, device=DEVICE)
        now = torch.tensor(lens, **ints)
        pos = torch.arange(table.shape[1] * page, **ints)
        places = table[:, (pos // page).long()] * page + pos % page
        _fill(data, places[pos[None, :] < now[:, None]], g, heads, dim, group, page, sigma)
        weights = _weights((layers, n, heads), pos.numel(), now, g)
        kept = _plain_choose(weights, now, case["budget"], case["recent"], case["sinks"])
        new = now.clamp(max=case["budget"])
        slots = places[pos[None, :] < new[:, None]].to(torch.int32)
        return dict(case=case, data=data, table=table, lens=now, new_lens=new, kept=kept["kept"], weights=weights, slots=slots)
    nq, nkv = _lengths(case)
    shared = case.get("shared", 0)
    first, _ = _pages([-(-shared // page)], g, 0) if shared else (torch.empty(1, 0, **ints), None)
    table, _ = _pages([-(-k // page) for k in nkv], g, 1)
    table = torch.where(table >= 0, table + first.shape[1], -1)
    table = torch.cat((first.expand(len(nq), -1), table), 1).to(torch.int32).contiguous()
    lens = torch.tensor(nkv, **ints) + shared
    # places that hold no token keep what was there before (here bytes that are no numbers)
    data = torch.full((1, sum(-(-k // page) for k in nkv) + 1 + first.shape[1], heads, page // 16, blob), 255, dtype=torch.uint8,
                      device=DEVICE)
    pos = torch.arange(table.shape[1] * page, **ints)
    places = table[:, (pos // page).long()] * page + pos % page
    there = pos[None, :] < lens[:, None]
    there[1:, :shared] = False
    _fill(data, places[there], g, heads, dim, group, page, sigma)
    tokens, ratio = sum(nq), case["q_heads"] // heads
    q = 1.5 * torch.randn(tokens, heads, ratio, dim, generator=g, device=DEVICE) / sigma[:, None, :]
    cu = torch.tensor([0] + nq, **ints).cumsum(0).to(torch.int32)
    s = dict(case=case, data=data, table=table, lens=lens, cu=cu, q=q.reshape(tokens, heads * ratio, dim).to(torch.bfloat16))
    if op == "weigh":
        before = lens - (cu[1:] - cu[:-1])
        s["weights"] = ratio * case["queries"] * _weights((len(nq), heads), pos.numel(), before, g)
        s["out"] = torch.zeros_like(s["weights"])
    return s


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


def _of(c, p, group):
    """The values of K or V codes [.., channel parts of 32, parts, bytes of two channels]."""
    c = torch.stack((c & 15, c >> 4), -1).transpose(-4, -3)
    return _values(c.flatten(-4), p, group)


def _read(data, slots, page, group, dim):
    kc, kp, vc, vp = _views(data, dim, group)
    slots = slots.long()
    pg, blob, tok = slots // page, slots % page // 16, slots % 16
    k = _of(kc[:, pg, :, blob, tok], kp[:, pg, :, blob, tok], group)
    v = _of(vc[:, pg, :, blob, tok // 2, :, :, tok % 2], vp[:, pg, :, blob, tok], group)
    return k.to(torch.bfloat16).transpose(0, 1), v.to(torch.bfloat16).transpose(0, 1)


def _gather(data, table, lens, dim, group, want_v=True):
    """K and V [requests, heads, tokens of a table row, dim] in fp32, 0 where a request holds none."""
    got = data[table.clamp(min=0).long()]                              # requests, pages, heads, blobs, bytes
    kc, kp, vc, vp = _views(got, dim, group)
    requests, width, heads, blobs = got.shape[:4]
    tokens = width * blobs * 16
    seen = (torch.arange(tokens, device=DEVICE)[None, :] < lens[:, None])[:, None, :, None]
    k = torch.where(seen, _of(kc, kp, group).transpose(1, 2).reshape(requests, heads, tokens, dim), 0.0)
    if not want_v:
        return k, None
    v = _of(vc.movedim(-2, -4).flatten(-5, -4), vp, group).transpose(1, 2).reshape(requests, heads, tokens, dim)
    return k, torch.where(seen, v, 0.0)


def _padded(s):
    """The queries as [requests, heads, ratio, most, dim] in fp32, which of them there are, and their positions [requests, most]."""
    case, cu, lens = s["case"], s["cu"], s["lens"]
    heads, ratio = case["heads"], case["q_heads"] // case["heads"]
    row = torch.arange(case["queries"], device=DEVICE)
    n = cu[1:] - cu[:-1]
    at = (cu[:-1, None] + torch.minimum(row[None, :], n[:, None] - 1)).long()
    q = s["q"].float()[at].unflatten(2, (heads, ratio)).permute(0, 2, 3, 1, 4)
    return q, row[None, :] < n[:, None], (lens - n)[:, None] + row[None, :]


def _plain_shared(s):
    case, shared, page, dim = s["case"], s["case"]["shared"], s["case"]["page"], s["case"]["dim"]
    table, lens, cu = s["table"], s["lens"], s["cu"]
    q, _, pos = _padded(s)
    requests, heads, ratio, most, _ = q.shape
    # the shared tokens: one product for the rows of all requests
    rows = q.movedim(1, 0).reshape(heads, requests * ratio * most, dim)
    k, v = _gather(s["data"][0], table[:1, :shared // page], lens[:1], dim, case["group"])
    before = torch.matmul(rows, k[0].transpose(-1, -2)).mul_(1.0 / math.sqrt(dim))
    k2, v2 = _gather(s["data"][0], table[:, shared // page:], lens - shared, dim, case["group"])
    scores = torch.matmul(q.flatten(2, 3), k2.transpose(-1, -2)).mul_(1.0 / math.sqrt(dim)).unflatten(2, (ratio, most))
    j = shared + torch.arange(scores.shape[-1], device=DEVICE)[None, None, :]
    scores.masked_fill_(((j > pos[:, :, None]) | (j >= lens[:, None, None]))[:, None, None], -math.inf)
    by_head = scores.movedim(1, 0).reshape(heads, requests * ratio * most, -1)
    top = torch.maximum(before.amax(-1, keepdim=True), by_head.amax(-1, keepdim=True))
    before.sub_(top).exp_()
    scores.sub_(top.reshape(heads, requests, ratio, most, 1).movedim(1, 0)).exp_()
    total = before.sum(-1).reshape(heads, requests, ratio, most).movedim(1, 0) + scores.sum(-1)
    out = torch.matmul(before, v[0]).reshape(heads, requests, ratio, most, dim).movedim(1, 0)
    out = (out + torch.matmul(scores.flatten(2, 3), v2).unflatten(2, (ratio, most))) / total[..., None]
    out = out.permute(0, 3, 1, 2, 4).reshape(requests, most, heads * ratio, dim)
    t = torch.arange(s["q"].shape[0], device=DEVICE)
    r = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    return dict(out=out[r, t - cu[r]].to(torch.bfloat16))


def _plain_weigh(s):
    case, lens = s["case"], s["lens"]
    q, there, pos = _padded(s)
    requests, heads, ratio, most, dim = q.shape
    k, _ = _gather(s["data"][0], s["table"], lens, dim, case["group"], False)
    scores = torch.matmul(q.flatten(2, 3), k.transpose(-1, -2)).mul_(1.0 / math.sqrt(dim)).unflatten(2, (ratio, most))
    at, j = pos[:, :, None], torch.arange(k.shape[2], device=DEVICE)[None, None, :]
    hide = (j > at) | (j >= lens[:, None, None])
    if case["window"]:
        hide = hide | ((at - j >= case["window"]) & (j >= case["sinks"]))
    scores.masked_fill_(hide[:, None, None], -math.inf)
    scores.sub_(scores.amax(-1, keepdim=True)).exp_()
    scores.div_(scores.sum(-1, keepdim=True)).mul_(there[:, None, None, :, None])
    got = s["weights"] + scores.sum((2, 3))
    s["out"].copy_(torch.where(j[0] < lens[:, None], got.movedim(1, 0), s["out"].movedim(1, 0)).movedim(0, 1))
    return dict(weights=s["out"])


def _plain_choose(weights, lens, budget, recent, sinks):
    """Of each row's first lens tokens, in order: the first `sinks`, the last `recent`, and the greatest of the others, `budget` in all."""
    n = weights.shape[-1]
    m = lens[:, None, None]
    at = torch.arange(n, device=DEVICE)
    rank = torch.where((at < sinks) | (at >= m - recent), math.inf, weights.to(torch.float64))
    rank = torch.where(at < m, rank, -math.inf)
    order = torch.sort(rank, dim=-1, descending=True, stable=True).indices[..., :budget]
    order = torch.where(torch.arange(order.shape[-1], device=DEVICE) < m, order, n)
    order = torch.sort(order, dim=-1).values
    kept = torch.full((*weights.shape[:-1], budget), -1, dtype=torch.int32, device=DEVICE)
    kept[..., :order.shape[-1]] = torch.where(order < n, order, -1).to(torch.int32)
    return dict(kept=kept, lens=lens.clamp(max=budget))


def _plain_compact(s):
    case, data, table, lens, new = s["case"], s["data"], s["table"], s["lens"], s["new_lens"]
    page, dim, group, kept = case["page"], case["dim"], case["group"], s["kept"]
    layers, requests, heads, budget = kept.shape
    stays = torch.arange(budget, device=DEVICE) < new[:, None]
    r, i = torch.nonzero(stays, as_tuple=True)                         # every token that stays, of every request
    layer, head = torch.arange(layers, device=DEVICE)[:, None, None], torch.arange(heads, device=DEVICE)[None, :, None]
    src = kept[:, r, :, i].permute(1, 2, 0).long()                     # layers, heads, tokens
    kc, kp, vc, vp = _views(data, dim, group)

    def place(at):
        return table[r, at // page].long(), at % page // 16, at % 16

    p, b, t = place(src)
    got = [x[layer, p, head, b, t].clone() for x in (kc, kp, vp)]
    gv = vc[layer, p, head, b, t // 2, :, :, t % 2].clone()
    p, b, t = place(i.expand(layers, heads, -1))
    for x, y in zip((kc, kp, vp), got):
        x[layer, p, head, b, t] = y
    vc[layer, p, head, b, t // 2, :, :, t % 2] = gv
    w = s["weights"]
    moved, most = w.gather(-1, kept.clamp(min=0).long()), min(budget, w.shape[-1])
    w.masked_fill_(torch.arange(w.shape[-1], device=DEVICE) < lens[:, None, None], 0.0)
    w[..., :most] = torch.where(stays[:, None, :most], moved[..., :most], w[..., :most])
    return w


def _plain_release(s):
    case, table, lens, new = s["case"], s["table"], s["lens"], s["new_lens"]
    page, free = case["page"], s["free"]
    held, stays = (lens + page - 1) // page, (new + page - 1) // page
    gone = held - stays
    end = torch.cumsum(gone, 0)
    cu = torch.cat((torch.zeros_like(end[:1]), end)).to(torch.int32)
    at = torch.arange(table.shape[1], device=DEVICE)[None, :]
    goes = (at >= stays[:, None]) & (at < held[:, None])
    free[s["free_count"] + (cu[:-1, None] + at - stays[:, None])[goes]] = table[goes]
    table.masked_fill_(goes, -1)
    return dict(table=table, free=free, free_count=(s["free_count"] + end[-1]).to(torch.int32), lens=new.clone(), cu=cu)


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
    op = case["op"]
    if own:
        if op in ("choose", "release"):
            from kv_cache_compression_03_gb300 import cachegen as cg
            if op == "choose":
                c = cg.choose_tokens(s["weights"], s["lens"], case["budget"], recent=case["recent"], sinks=case["sinks"])
                return dict(kept=c.kept, lens=c.lens)
            p = cg.release_pages(s["table"], s["lens"], s["new_lens"], s["free"], s["free_count"], case["page"])
            return dict(table=s["table"], free=s["free"], free_count=p.free_count, lens=p.lens, cu=p.cu)
        cache = _cache(s)
        if op == "shared":
            return dict(out=cache.attention(s["q"], s["cu"], s["lens"], s["table"], max_q_len=case["queries"], shared=case["shared"]))
        if op == "weigh":
            return dict(weights=cache.weigh(s["q"], s["cu"], s["lens"], s["table"], s["weights"], window=case["window"],
                                            sinks=case["sinks"], max_q_len=case["queries"], out=s["out"]))
        cache.compact(s["kept"], s["new_lens"], s["lens"], s["table"], weights=s["weights"])
        k, v = cache.load(s["slots"], layers=case["layers"])
        return dict(k=k, v=v, weights=s["weights"])
    if op == "shared":
        return _plain_shared(s)
    if op == "weigh":
        return _plain_weigh(s)
    if op == "choose":
        return _plain_choose(s["weights"], s["lens"], case["budget"], case["recent"], case["sinks"])
    if op == "release":
        return _plain_release(s)
    w = _plain_compact(s)
    k, v = _read(s["data"], s["slots"], case["page"], case["group"], case["dim"])
    return dict(k=k, v=v, weights=w)


# ------------------------------------------------------- what a pass has to do

def work(case):
    op = case["op"]
    if op == "release":
        n, page = case["requests"], case["page"]
        lens = _spread(n, case["len"], case["spread"])
        gone = sum(-(-x // page) + (-min(x, case["budget"]) // page) for x in lens)
        return dict(bytes=8 * n + 12 * gone + 8 * n + 12, flops=0)
    if op in ("choose", "compact"):
        rows = case["layers"] * case["heads"]
        lens = _spread(case["requests"], case["len"], case["spread"])
        stay = [min(x, case["budget"]) for x in lens]
        if op == "choose":
            return dict(bytes=4 * rows * (sum(lens) + case["budget"] * len(lens)) + 8 * len(lens), flops=0)
        held = case["dim"] + 8 * (case["dim"] // case["group"])        # bytes of one token and head in the cache
        # tokens read and written, their weights too, what is behind set to 0; then read and given as bf16
        return dict(bytes=rows * (sum(stay) * (2 * held + 12 + held + 4 * case["dim"]) + 4 * (sum(lens) - sum(stay))), flops=0)
    heads, dim = case["heads"], case["dim"]
    held = dim + 8 * (dim // case["group"])
    nq, nkv = _lengths(case)
    if op == "shared":
        tokens = case["shared"] + sum(nkv)
        pairs = sum(n * (case["shared"] + k - n) + n * (n + 1) // 2 for n, k in zip(nq, nkv))
        return dict(bytes=tokens * heads * held + 4 * sum(nq) * case["q_heads"] * dim, flops=4 * dim * case["q_heads"] * pairs)
    window, sinks = case["window"] or 1 << 40, case["sinks"]
    pairs = tokens = 0
    for n, k in zip(nq, nkv):
        for p in range(k - n, k):
            low = max(0, p + 1 - window)
            pairs += p + 1 - low + min(low, sinks)
        low = max(0, k - n + 1 - window)
        tokens += k - low + min(low, sinks)
    # half of what a token holds is K; the weights of all tokens are read and written
    return dict(bytes=tokens * heads * held // 2 + 8 * sum(nkv) * heads + 2 * sum(nq) * case["q_heads"] * dim,
                flops=2 * dim * case["q_heads"] * pairs)


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


def _exact_probabilities(s, k, row, n, m, h, ratio):
    """The probabilities of a request's n query rows of query head h over its m tokens, in 64 bits."""
    case = s["case"]
    at = torch.arange(m, device=DEVICE)
    behind = torch.arange(m - n, m, device=DEVICE)[:, None] - at[None, :]
    visible = behind >= 0
    if case.get("window"):
        visible &= (behind < case["window"]) | (at[None, :] < case["sinks"])
    score = s["q"][row:row + n, h].double() @ k[:, h // ratio].T / math.sqrt(case["dim"])
    return torch.softmax(torch.where(visible, score, -math.inf), -1)


def exact(case, seed):
    op = case["op"]
    if op in ("choose", "release"):
        return None                                                    # whole numbers
    s = prepare(case, seed)
    heads, dim, page = case["heads"], case["dim"], case["page"]
    if op == "compact":
        layers, requests = case["layers"], case["requests"]
        ks, vs, weights = [], [], s["weights"].double()
        for layer in range(layers):
            kk, vv = [], []
            for r in range(requests):
                n, m = int(s["new_lens"][r]), int(s["lens"][r])
                at = torch.arange(m, device=DEVICE)
                k, v = _exact_rows(case, s["data"][layer], s["table"][r, at // page].long() * page + at % page)
                stay = s["kept"][layer, r, :, :n].long()               # heads, tokens
                for x, y in ((kk, k), (vv, v)):
                    x.append(torch.stack([y[stay[h], h] for h in range(heads)], 1))
                for h in range(heads):
                    w = torch.zeros(m, dtype=torch.float64, device=DEVICE)
                    w[:n] = s["weights"][layer, r, h, stay[h]].double()
                    weights[layer, r, h, :m] = w
            ks.append(torch.cat(kk))
            vs.append(torch.cat(vv))
        return dict(k=torch.stack(ks), v=torch.stack(vs), weights=weights)
    nq, nkv = _lengths(case)
    ratio, shared = case["q_heads"] // heads, case.get("shared", 0)
    out = torch.empty(sum(nq), case["q_heads"], dim, dtype=torch.float64, device=DEVICE)
    sums = s["weights"].double() if op == "weigh" else None
    row = 0
    for r, (n, m) in enumerate(zip(nq, nkv)):
        m += shared
        at = torch.arange(m, device=DEVICE)
        k, v = _exact_rows(case, s["data"][0], s["table"][r, at // page].long() * page + at % page)
        for h in range(case["q_heads"]):
            p = _exact_probabilities(s, k, row, n, m, h, ratio)
            if op == "weigh":
                sums[r, h // ratio, :m] += p.sum(0)
            else:
                out[row:row + n, h] = p @ v[:, h // ratio]
        row += n
    return dict(weights=sums) if op == "weigh" else dict(out=out)
